// FP8 linear map with a weight scale per block of 128 x 128:
//   y[m][n] = sum over K blocks b of  ws[n / 128][b] * sx[m][b] * sum_{k in b} q[m][k] * W[n][k]
// W are E4M3 codes with fp32 block scales ws; q and sx are x quantised per
// row and 128 values: sx the least power of two with |x| <= 448 sx over the
// block, q = x / sx rounded to nearest-even E4M3.  An activation of the
// framework follows where asked for, and one rounding to bf16.
//
// A power-of-two sx costs no accuracy against an fp32 scale (E4M3 is a
// floating type: the scale only places its range, and the block's largest
// value lands in (224, 448]) and goes into the scale operand of
// v_mfma_scale_f32_16x16x128_f8f6f4 for free.  The instruction's K is exactly
// one block, so each MFMA starts from zero and its result is added to the
// fp32 accumulator times ws: 4 VALU multiply-adds per MFMA.
//
// Within an instruction a product is cut, towards zero, to a multiple of
// 2^-13 times the power of two of the largest of the 8 products it is added
// with first (measured; everything after that is fp32).  On normal data that
// is 2 to 3e-4 of the result, against 1.7e-3 from its rounding to bf16 and
// several per cent from the quantisation itself; the bf16 instructions, which
// would keep the products whole, run at half the rate.
//
// Operands: A = weights (16 rows), B = tokens (16), so that a lane's four
// accumulators are consecutive outputs of one token.  All scales of a row
// within an instruction are equal, so K may be laid out in any order as long
// as A and B agree: 16-byte group g = lane / 16 of each 64-byte half.
#include <hip/hip_runtime.h>

#include "act.h"
#include "block.h"
#include "decode.h"
#include "gemm_util.h"
#include "mxfp8.h"

namespace moe {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

// Scale byte of a block from its largest magnitude's fp32 bits: the least
// power of two with amax <= 448 scale (448 = 1.75 * 2^8), at least 2^-127;
// 255 (NaN) for a block with a NaN or an infinity.
__device__ __forceinline__ uint32_t block_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255u;
  const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)(e > 0 ? e : 0);
}

// ---- weight preparation: one thread per 16 prepared bytes

__global__ void __launch_bounds__(256)
    fp8_prepare_kernel(Fp8Shape s, const uint8_t* __restrict__ codes, const float* __restrict__ scales,
                       uint8_t* __restrict__ prepared) {
  const int kb = s.kblocks(), nb = (s.N + 127) / 128;
  const int64_t chunks = (int64_t)s.subtiles() * kb * 128;
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  float* const ps = (float*)(prepared + s.codes_bytes());
  for (int64_t it = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; it < chunks; it += stride) {
    const int lane = (int)(it & 63), half = (int)((it >> 6) & 1);
    const int64_t sb = it >> 7;
    const int b = (int)(sb % kb);
    const int sub = (int)(sb / kb);
    const int part = s.gated ? (sub & 1) : 0;  // up rows follow the N gate rows
    const int row = (s.gated ? sub >> 1 : sub) * 16 + (lane & 15);
    const int k0 = b * 128 + half * 64 + (lane >> 4) * 16;
    uint64_t v[2] = {0, 0};
    if (row < s.N) {
      const uint8_t* src = codes + ((int64_t)part * s.N + row) * s.K + k0;  // 8-byte aligned: K % 8 == 0
      if (k0 < s.K) v[0] = *(const uint64_t*)src;
      if (k0 + 8 < s.K) v[1] = *(const uint64_t*)(src + 8);
    }
    ((uint64_t*)prepared)[2 * it] = v[0];
    ((uint64_t*)prepared)[2 * it + 1] = v[1];
    if (lane == 0 && half == 0) ps[sb] = scales[((int64_t)part * nb + row / 128) * kb + b];
  }
}

// ---- activation quantisation: 16 consecutive lanes per 128 values

__global__ void __launch_bounds__(256)
    fp8_quantize_rows(const uint16_t* __restrict__ x, int64_t items, int K, int kb, uint8_t* __restrict__ codes,
                      uint8_t* __restrict__ scales, int sstride) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  // items is a multiple of 16 and so is the stride: a block's lanes stay together
  for (int64_t it = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; it < items; it += stride) {
    const int per = kb * 16;
    const int64_t row = it / per;
    const int c = (int)(it - row * per);
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (c * 8 < K) raw = *(const uint4*)(x + row * K + c * 8);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float v[8];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      amax = max(amax, (w[i] << 16) & 0x7FFFFFFFu);
      amax = max(amax, w[i] & 0x7FFF0000u);
    }
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, d));
    const uint32_t sb = block_scale_byte(amax);
    uint32_t lo = 0x7F7F7F7Fu, hi = 0x7F7F7F7Fu;
    if (sb != 255u) {
      const float inv = mx_inv_scale(sb);
      lo = hi = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo |= e4m3_code(v[i] * inv) << (8 * i);
        hi |= e4m3_code(v[4 + i] * inv) << (8 * i);
      }
    }
    *(uint2*)(codes + it * 8) = make_uint2(lo, hi);
    if ((c & 15) == 0) scales[row * sstride + (c >> 4)] = (uint8_t)sb;
  }
}

// ---- products: each wave takes every NW-th K block of FS subtiles x 16 TT
// tokens; the waves' sums are joined in LDS in wave order.

template <int FS, int TT, int NW, bool GATED>
__global__ void __launch_bounds__(NW * 64)
    fp8_rows_kernel(Fp8Shape s, const uint8_t* __restrict__ prepared, const uint8_t* __restrict__ codes,
                    const uint8_t* __restrict__ xscale, int M, uint16_t* __restrict__ out) {
  __shared__ f32x4_t part[NW][FS * TT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int kb = s.kblocks(), ns = s.subtiles(), srow = s.scale_row();
  const int sub0 = blockIdx.x * FS;
  const int64_t tok0 = (int64_t)blockIdx.y * (16 * TT);
  const int r = lane & 15, g = lane >> 4;
  const float* const ws = (const float*)(prepared + s.codes_bytes());
  f32x4_t acc[FS][TT];
#pragma unroll
  for (int f = 0; f < FS; ++f)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[f][t] = f32x4_t{};
  const uint8_t* xrow[TT];
  const uint8_t* srows[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int64_t m = min(tok0 + 16 * t + r, (int64_t)M - 1);  // rows past M repeat the last one and are not stored
    xrow[t] = codes + m * kb * 128 + g * 16;
    srows[t] = xscale + m * srow;
  }
  for (int b = wave; b < kb; b += NW) {
    i32x8_t bop[TT];
    int sx[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const i32x4_t lo = *(const i32x4_t*)(xrow[t] + b * 128), hi = *(const i32x4_t*)(xrow[t] + b * 128 + 64);
      bop[t] = i32x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      sx[t] = srows[t][b];
    }
#pragma unroll
    for (int f = 0; f < FS; ++f) {
      const int sub = min(sub0 + f, ns - 1);
      const uint8_t* a = prepared + ((int64_t)sub * kb + b) * 2048 + lane * 16;
      const i32x4_t lo = *(const i32x4_t*)a, hi = *(const i32x4_t*)(a + 1024);
      const i32x8_t aop = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      const float w = ws[(int64_t)sub * kb + b];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const f32x4_t p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(aop, bop[t], f32x4_t{}, 0, 0, 0, 127, 0, sx[t]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[f][t][i] = fmaf(w, p[i], acc[f][t][i]);
      }
    }
  }
#pragma unroll
  for (int f = 0; f < FS; ++f)
#pragma unroll
    for (int t = 0; t < TT; ++t) part[wave][f * TT + t][lane] = acc[f][t];
  __syncthreads();
  // output tiles of 16 features x 16 tokens, dealt to the waves
  constexpr int kTiles = (GATED ? FS / 2 : FS) * TT;
  for (int o = wave; o < kTiles; o += NW) {
    const int f = o / TT, t = o % TT;
    f32x4_t v{}, u{};
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      v += part[i][(GATED ? 2 * f : f) * TT + t][lane];
      if (GATED) u += part[i][(2 * f + 1) * TT + t][lane];
    }
    const int n = (GATED ? sub0 / 2 + f : sub0 + f) * 16 + 4 * g;
    const int64_t m = tok0 + 16 * t + r;
    if (n >= s.N || m >= M) continue;  // N % 8 == 0: the lane's four outputs are all in or all out
    uint32_t o16[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o16[i] = f32_to_bf16_rne(s.has_act ? gated_act(s.act, v[i], u[i]) : v[i]);
    *(uint2*)(out + m * s.N + n) = make_uint2(o16[0] | (o16[1] << 16), o16[2] | (o16[3] << 16));
  }
}

template <int FS, int TT, int NW>
hipError_t launch_rows(const Fp8Shape& s, const uint8_t* prepared, const uint8_t* codes, const uint8_t* xscale, int M,
                       uint16_t* out, hipStream_t st) {
  const dim3 grid((unsigned)((s.subtiles() + FS - 1) / FS), (unsigned)((M + 16 * TT - 1) / (16 * TT)));
  if (s.gated)
    hipLaunchKernelGGL((fp8_rows_kernel<FS, TT, NW, true>), grid, dim3(NW * 64), 0, st, s, prepared, codes, xscale, M,
                       out);
  else
    hipLaunchKernelGGL((fp8_rows_kernel<FS, TT, NW, false>), grid, dim3(NW * 64), 0, st, s, prepared, codes, xscale,
                       M, out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_prepare(const Fp8Shape& s, const uint8_t* codes, const float* scales, uint8_t* prepared,
                              hipStream_t st) {
  const int64_t blocks = ((int64_t)s.subtiles() * s.kblocks() * 128 + 255) / 256;
  hipLaunchKernelGGL(fp8_prepare_kernel, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st, s, codes,
                     scales, prepared);
  return hipGetLastError();
}

hipError_t launch_fp8_linear(const Fp8Shape& s, const uint8_t* prepared, const uint16_t* x, int M, uint16_t* out,
                             uint8_t* ws, hipStream_t st) {
  uint8_t* const codes = ws;
  uint8_t* const xscale = ws + s.code_bytes(M);
  const int64_t items = (int64_t)M * s.kblocks() * 16;
  const int64_t blocks = (items + 255) / 256;
  hipLaunchKernelGGL(fp8_quantize_rows, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st, x, items,
                     s.K, s.kblocks(), codes, xscale, s.scale_row());
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (M <= 16) return launch_rows<2, 1, 8>(s, prepared, codes, xscale, M, out, st);
  return launch_rows<4, 4, 4>(s, prepared, codes, xscale, M, out, st);
}

}  // namespace moe
