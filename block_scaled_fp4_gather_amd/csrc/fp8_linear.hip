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

// ---- activation quantisation

// Largest of 16 consecutive lanes, in all of them (rotations within a row).
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
#define MOE_STEP(CTRL) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true))
  MOE_STEP(0x121);  // row_ror:1
  MOE_STEP(0x122);
  MOE_STEP(0x124);
  MOE_STEP(0x128);
#undef MOE_STEP
  return v;
}

// 8 values of a 128-value block, whose other values 15 neighbouring lanes
// hold: codes and the block's scale byte.  v_cvt_pk_fp8_f32 rounds to
// nearest-even; no value exceeds 448.
__device__ __forceinline__ uint2 quantise8(const uint4& raw, uint32_t& byte) {
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
  byte = block_scale_byte(row_max_u32(amax));
  if (byte == 255u) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const float inv = mx_inv_scale(byte);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= inv;
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// One wave per row and 4 K blocks (a scale dword).
__global__ void __launch_bounds__(256)
    fp8_quantize_rows(const uint16_t* __restrict__ x, int M, int K, int kb, uint8_t* __restrict__ codes,
                      uint8_t* __restrict__ scales, int64_t scale_rows) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int q = blockIdx.y;
  if (row >= M) return;
  const int c = (q * 64 + lane) * 8;
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (c < K) raw = *(const uint4*)(x + row * K + c);
  uint32_t byte;
  const uint2 code = quantise8(raw, byte);
  if (c < kb * 128) *(uint2*)(codes + row * kb * 128 + c) = code;
  const uint32_t dword = __builtin_amdgcn_readlane(byte, 0) | __builtin_amdgcn_readlane(byte, 16) << 8 |
                         __builtin_amdgcn_readlane(byte, 32) << 16 | __builtin_amdgcn_readlane(byte, 48) << 24;
  if (lane == 0) *(uint32_t*)(scales + (q * scale_rows + row) * 4) = dword;
}

// ---- few tokens: FS subtiles x 16 TT tokens per workgroup, whose NW waves
// share K in runs of consecutive blocks and join their sums in LDS in wave
// order.  What bounds it is the time from a load to its use, so each wave
// loads U blocks' operands while it multiplies the U before.
//
// FUSED: x is quantised by each workgroup itself into LDS (up to kFusedUnits
// blocks of 128 values), while the first weights are on their way: for the
// fewest tokens that takes less than a launch of its own.

template <int NW>
constexpr int kFusedUnits = 4 * 4 * NW;  // 4 passes of the workgroup's 16-lane groups

template <int FS, int TT, int NW, int U, bool GATED, bool FUSED>
__global__ void __launch_bounds__(NW * 64)
    fp8_few_kernel(Fp8Shape s, const uint8_t* __restrict__ prepared, const uint8_t* __restrict__ codes,
                   const uint8_t* __restrict__ xscale, const uint16_t* __restrict__ x, int M,
                   uint16_t* __restrict__ out) {
  static_assert(!GATED || FS % 2 == 0, "whole gate and up pairs");
  static_assert(!FUSED || TT == 1, "few tokens");
  __shared__ f32x4_t part[NW][FS * TT][64];
  __shared__ uint8_t qcodes[FUSED ? kFusedUnits<NW> * 128 : 16], qscale[FUSED ? kFusedUnits<NW> : 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kb = s.kblocks(), ns = s.subtiles();
  const int64_t mp = s.scale_rows(M);
  const int sub0 = blockIdx.x * FS;
  const int64_t tok0 = (int64_t)blockIdx.y * (16 * TT);
  const int r = lane & 15, g = lane >> 4;
  const float* const ws = (const float*)(prepared + s.codes_bytes());
  const int per = (kb + NW - 1) / NW, b0 = wave * per, b1 = min(kb, b0 + per);

  struct Operands {
    i32x8_t a[U][FS], b[U][TT];
    int sx[U][TT];
    float w[U][FS];
  };
  const uint8_t* xrow[TT];
  const uint8_t* srow[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int64_t m = min(tok0 + 16 * t + r, (int64_t)M - 1);  // rows past M repeat the last one and are not stored
    xrow[t] = codes + m * kb * 128 + g * 16;
    srow[t] = xscale + m * 4;
  }
  auto load = [&](int b, Operands& o) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int bu = min(b + u, kb - 1);  // blocks past the run are loaded and not used
#pragma unroll
      for (int f = 0; f < FS; ++f) {
        const int64_t sub = min(sub0 + f, ns - 1);
        const uint8_t* const at = prepared + (sub * kb + bu) * 2048;
        const i32x4_t lo = *(const i32x4_t*)(at + lane * 16), hi = *(const i32x4_t*)(at + lane * 16 + 1024);
        o.a[u][f] = i32x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        o.w[u][f] = ws[sub * kb + bu];
      }
      if constexpr (!FUSED)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const i32x4_t lo = *(const i32x4_t*)(xrow[t] + bu * 128), hi = *(const i32x4_t*)(xrow[t] + bu * 128 + 64);
          o.b[u][t] = i32x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          o.sx[u][t] = srow[t][(bu >> 2) * mp * 4 + (bu & 3)];
        }
    }
  };
  f32x4_t acc[FS][TT];
#pragma unroll
  for (int f = 0; f < FS; ++f)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[f][t] = f32x4_t{};
  auto multiply = [&](int b, Operands& o) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u >= b1) break;
      if constexpr (FUSED) {
        const int unit = min(r, M - 1) * kb + b + u;
        const i32x4_t lo = *(const i32x4_t*)(qcodes + unit * 128 + g * 16);
        const i32x4_t hi = *(const i32x4_t*)(qcodes + unit * 128 + g * 16 + 64);
        o.b[u][0] = i32x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        o.sx[u][0] = qscale[unit];
      }
#pragma unroll
      for (int f = 0; f < FS; ++f)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const f32x4_t p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(o.a[u][f], o.b[u][t], f32x4_t{}, 0, 0, 0,
                                                                             127, 0, o.sx[u][t]);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[f][t][i] = fmaf(o.w[u][f], p[i], acc[f][t][i]);
        }
    }
  };

  Operands o0, o1;
  if constexpr (FUSED) {
    const int units = M * kb;
    uint4 raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int unit = (i * NW * 64 + (int)threadIdx.x) / 16, row = unit / kb;
      const int c = (unit - row * kb) * 128 + (lane & 15) * 8;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (unit < units && c < s.K) raw[i] = *(const uint4*)(x + (int64_t)row * s.K + c);
    }
    __builtin_amdgcn_sched_barrier(0);  // x first: it is needed first
    load(b0, o0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int unit = (i * NW * 64 + (int)threadIdx.x) / 16;
      uint32_t byte;
      const uint2 code = quantise8(raw[i], byte);
      if (unit < units) {
        *(uint2*)(qcodes + unit * 128 + (lane & 15) * 8) = code;
        if ((lane & 15) == 0) qscale[unit] = (uint8_t)byte;
      }
    }
    __syncthreads();
  } else {
    load(b0, o0);
  }
  for (int b = b0; b < b1; b += 2 * U) {
    load(b + U, o1);
    __builtin_amdgcn_sched_barrier(0);
    multiply(b, o0);
    load(b + 2 * U, o0);
    __builtin_amdgcn_sched_barrier(0);
    multiply(b + U, o1);
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
    if (s.has_act)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = gated_act(s.act, v[i], u[i]);
    *(uint2*)(out + m * s.N + n) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  }
}

// ---- many tokens: BM tokens x BN weight rows per workgroup of 8 waves
// (WT x WF), one K block per step.  Tokens (a row of 128 codes: the 16-byte
// chunk c of row r at position c ^ row_swz(r)) and weights (in the layout they
// were prepared in) go to LDS by direct copies, one step ahead in two slots.
// Every 4 steps the scale dwords of the tokens' next 4 K blocks follow.
template <int BM, int BN, int WT, int WF>
struct Fp8Tile {
  static constexpr int FS = BN / 16 / WF, TT = BM / 16 / WT;
  static constexpr int kTokens = BM * 128, kSlot = kTokens + BN * 128;
  static constexpr int kCopies = kTokens / 1024 / 8, kWCopies = BN / 64, kAllCopies = kCopies + kWCopies;
  static constexpr int kLds = 2 * kSlot + 2 * 4 * BM;
  static_assert(WT * WF == 8 && FS % 2 == 0 && BM % 64 == 0 && BN % 64 == 0,
                "8 waves, whole gate and up pairs, whole copies");
  static_assert(kAllCopies + 1 < FS * TT, "copies between the products");
};

template <int BM, int BN, int WT, int WF, bool GATED>
__global__ void __launch_bounds__(512, 2)
    fp8_tile_kernel(Fp8Shape s, const uint8_t* __restrict__ prepared, const uint8_t* __restrict__ codes,
                    const uint8_t* __restrict__ xscale, int M, int tiles_m, int tiles_n, uint16_t* __restrict__ out) {
  using T = Fp8Tile<BM, BN, WT, WF>;
  constexpr int FS = T::FS, TT = T::TT;
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* const sring = smem + 2 * T::kSlot;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  // Workgroups are dealt to the 8 XCDs in turn: give each XCD a contiguous
  // range of tiles, in bands of 4 token tiles, so that what runs together on
  // it shares token and weight tiles in its L2.
  const int per = gridDim.x / 8;
  const int logical = (blockIdx.x % 8) * per + blockIdx.x / 8;
  if (logical >= tiles_m * tiles_n) return;
  const int band = logical / (4 * tiles_n), in_band = logical - band * 4 * tiles_n;
  const int bm = min(4, tiles_m - 4 * band);
  const int tn = in_band / bm, tm = 4 * band + in_band % bm;

  const int kb = s.kblocks(), ns = s.subtiles();
  const int64_t mp = s.scale_rows(M), tok0 = (int64_t)tm * BM;
  const int wf = wave % WF, wt = wave / WF;
  const int sub0 = tn * (BN / 16) + wf * FS;
  const float* const ws = (const float*)(prepared + s.codes_bytes());

  // token copies of this wave: rows of the tile past the last token repeat it
  const uint8_t* const tile = codes + tok0 * kb * 128;
  const int rows = (int)min((int64_t)M - tok0, (int64_t)BM);
  uint32_t src[T::kCopies];  // at most 255 rows of 2^20 bytes
#pragma unroll
  for (int c = 0; c < T::kCopies; ++c) {
    const int row = (c * 8 + wave) * 8 + lane / 8;
    src[c] = (uint32_t)min(row, rows - 1) * (kb * 128u) + ((lane & 7) ^ row_swz<128>(row)) * 16;
  }
  // Scale dwords of K blocks 4q .. 4q + 3 (the scale rows are padded to whole
  // tiles).  In a step this repeats for 4 steps what the first of them did,
  // and every wave takes part: a branch in the middle of a step costs more.
  const uint32_t part = (wave % (BM / 64)) * 256;
  const uint8_t* const scales = xscale + tok0 * 4 + part;
  const int last_q = (kb - 1) / 4;
  auto copy_scales = [&](int q) {
    const int from = min(q, last_q);
    dma4_at(scales + from * mp * 4, lane * 4, lds_addr(sring) + (q & 1) * 4 * BM + part);
  };
  // weight copies of this wave: 1 KiB, half a subtile's block, each; subtiles past the last repeat it
  const uint8_t* wsrc[T::kWCopies];
#pragma unroll
  for (int c = 0; c < T::kWCopies; ++c) {
    const int kib = c * 8 + wave;
    wsrc[c] = prepared + (int64_t)min(tn * (BN / 16) + kib / 2, ns - 1) * kb * 2048 + (kib & 1) * 1024;
  }
  const uint32_t lds0 = lds_addr(smem) + wave * 1024;
  auto copy = [&](int b, int ring, int c) {  // copy c of K block b: tokens, then weights
    const uint32_t to = lds0 + ring * T::kSlot + c * 8192;
    if (c < T::kCopies)
      dma16_at(tile + (int64_t)b * 128, src[c], to);
    else
      dma16_at(wsrc[c - T::kCopies] + (int64_t)b * 2048, lane * 16, to);
  };
  const float* const wscale = ws + (int64_t)min(sub0 + lane % FS, ns - 1) * kb;
  f32x4_t acc[FS][TT];
#pragma unroll
  for (int f = 0; f < FS; ++f)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[f][t] = f32x4_t{};

  const int swz = row_swz<128>(r);  // the same for every 16th row: rows 16 t + r
  const int brow = (wt * TT * 16 + r) * 128, bs = (wt * TT * 16 + r) * 4;
  float w = wscale[0];
#pragma unroll
  for (int c = 0; c < T::kAllCopies; ++c) copy(0, 0, c);
  copy_scales(0);
#pragma unroll 1
  for (int b = 0; b < kb; ++b) {
    vm_wait<0>();     // this wave's copies for step b are here
    __syncthreads();  // everyone's are, and everyone is done with step b - 1
    const int next = min(b + 1, kb - 1);  // past the last block it is copied again, and not used
    float wf_[FS];
#pragma unroll
    for (int f = 0; f < FS; ++f) wf_[f] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), f));
    w = wscale[next];
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* const slot = smem + (b & 1) * T::kSlot + brow;
    const uint8_t* const wslot = smem + (b & 1) * T::kSlot + T::kTokens + wf * FS * 2048 + lane * 16;
    const uint8_t* const sc = sring + ((b >> 2) & 1) * 4 * BM + bs + (b & 3);
    auto read = [&](int t, i32x8_t& bop, int& sx) {
      const i32x4_t lo = *(const i32x4_t*)(slot + t * 2048 + (g ^ swz) * 16);
      const i32x4_t hi = *(const i32x4_t*)(slot + t * 2048 + ((4 + g) ^ swz) * 16);
      bop = i32x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      sx = sc[t * 64];
    };
    // The multiply-adds of a product come kLag products later: its result is
    // there by then, and they run in the shadow of the products in between.
    // The order is pinned: left alone, the compiler puts them right behind
    // their product and waits, or keeps so much in flight that registers spill.
    constexpr int kLag = 2, kRing = kLag + 1, kAll = FS * TT;
    i32x8_t a[FS], bop[2];
    int sx[2];
    f32x4_t p[kRing];
    read(0, bop[0], sx[0]);
#pragma unroll
    for (int f = 0; f < FS; ++f) {
      const i32x4_t lo = *(const i32x4_t*)(wslot + f * 2048), hi = *(const i32x4_t*)(wslot + f * 2048 + 1024);
      a[f] = i32x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
#pragma unroll
    for (int i = 0; i < kAll + kLag; ++i) {
      const int t = i / FS, f = i % FS;
      if (i < kAll) {
        if (f == 0 && t + 1 < TT) read(t + 1, bop[(t + 1) & 1], sx[(t + 1) & 1]);
        // the next step's copies go between the first products
        if (i >= 1 && i <= T::kAllCopies) copy(next, (b + 1) & 1, i - 1);
        if (i == T::kAllCopies + 1) copy_scales((b >> 2) + 1);
        p[i % kRing] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[f], bop[t & 1], f32x4_t{}, 0, 0, 0, 127, 0,
                                                                       sx[t & 1]);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (i >= kLag) {
        const int j = i - kLag;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[j % FS][j / FS][e] = fmaf(wf_[j % FS], p[j % kRing][e], acc[j % FS][j / FS][e]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  vm_wait<0>();  // no copy may land after the workgroup's LDS is released

  __syncthreads();

  // Each wave turns its outputs round in its own part of the LDS, so that it
  // stores whole rows of up to 128 bytes: 16-byte chunk c of token row i at
  // position c ^ (i % chunks of a row).
  constexpr int kRow = (GATED ? FS / 2 : FS) * 32, kPer = kRow / 16;
  static_assert(8 * TT * 16 * kRow <= 2 * T::kSlot, "the waves' parts");
  uint8_t* const mine = smem + wave * TT * 16 * kRow;
  auto put = [&](auto kind) {
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int f = 0; f < FS; f += GATED ? 2 : 1) {
        f32x4_t v = acc[f][t];
        if constexpr (decltype(kind)::value >= 0)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = act_of<decltype(kind)::value>(s.act, v[i], GATED ? acc[f + (GATED ? 1 : 0)][t][i] : 0.0f);
        const int c = (GATED ? f / 2 : f) * 2 + g / 2;
        *(uint2*)(mine + (16 * t + r) * kRow + (c ^ (r % kPer)) * 16 + g % 2 * 8) =
            make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
      }
  };
  if constexpr (GATED) {
    if (s.act.kind == kActGeluTanh) put(std::integral_constant<int, kActGeluTanh>{});
    else if (s.act.kind == kActSwigluOai) put(std::integral_constant<int, kActSwigluOai>{});
    else put(std::integral_constant<int, kActSilu>{});
  } else {
    if (s.has_act) put(std::integral_constant<int, kActRelu2>{});
    else put(std::integral_constant<int, -1>{});
  }
  wave_sync();
  const int n = (GATED ? sub0 / 2 : sub0) * 16 + lane % kPer * 8;
  const int64_t m0 = tok0 + wt * TT * 16;
#pragma unroll
  for (int i = 0; i < TT * 16 * kPer / 64; ++i) {
    const int row = i * (64 / kPer) + lane / kPer;
    const uint4 v = *(const uint4*)(mine + row * kRow + (lane % kPer ^ row % kPer) * 16);
    // N % 8 == 0: a chunk's eight outputs are all in or all out
    if (m0 + row < M && n < s.N) *(uint4*)(out + (m0 + row) * s.N + n) = v;
  }
}

template <int BM, int BN, int WT, int WF>
hipError_t launch_tile(const Fp8Shape& s, const uint8_t* prepared, const uint8_t* codes, const uint8_t* xscale, int M,
                       uint16_t* out, hipStream_t st) {
  using T = Fp8Tile<BM, BN, WT, WF>;
  const int tm = (M + BM - 1) / BM, tn = (s.subtiles() + BN / 16 - 1) / (BN / 16);
  const dim3 grid(grid8((int64_t)tm * tn));
  if (s.gated)
    hipLaunchKernelGGL((fp8_tile_kernel<BM, BN, WT, WF, true>), grid, dim3(512), T::kLds, st, s, prepared, codes,
                       xscale, M, tm, tn, out);
  else
    hipLaunchKernelGGL((fp8_tile_kernel<BM, BN, WT, WF, false>), grid, dim3(512), T::kLds, st, s, prepared, codes,
                       xscale, M, tm, tn, out);
  return hipGetLastError();
}

template <int FS, int TT, int NW, int U, bool FUSED>
hipError_t launch_few(const Fp8Shape& s, const uint8_t* prepared, const uint8_t* codes, const uint8_t* xscale,
                      const uint16_t* x, int M, uint16_t* out, hipStream_t st) {
  // a gated map takes its subtiles in pairs
  constexpr int GFS = FS % 2 ? 2 * FS : FS;
  const int fs = s.gated ? GFS : FS;
  const dim3 grid((unsigned)((s.subtiles() + fs - 1) / fs), (unsigned)((M + 16 * TT - 1) / (16 * TT)));
  if (s.gated)
    hipLaunchKernelGGL((fp8_few_kernel<GFS, TT, NW, U, true, FUSED>), grid, dim3(NW * 64), 0, st, s, prepared, codes,
                       xscale, x, M, out);
  else
    hipLaunchKernelGGL((fp8_few_kernel<FS, TT, NW, U, false, FUSED>), grid, dim3(NW * 64), 0, st, s, prepared, codes,
                       xscale, x, M, out);
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
  const bool deep = s.kblocks() > 16;  // enough blocks for 16 waves
  if (M <= 4 && M * s.kblocks() <= (deep ? kFusedUnits<16> : kFusedUnits<4>)) {
    if (deep) return launch_few<1, 1, 16, 2, true>(s, prepared, codes, xscale, x, M, out, st);
    return launch_few<1, 1, 4, 2, true>(s, prepared, codes, xscale, x, M, out, st);
  }
  hipLaunchKernelGGL(fp8_quantize_rows, dim3((unsigned)((M + 3) / 4), (unsigned)((s.kblocks() + 3) / 4)), dim3(256), 0,
                     st, x, M, s.K, s.kblocks(), codes, xscale, s.scale_rows(M));
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (M <= 16) {
    if (deep) return launch_few<1, 1, 16, 2, false>(s, prepared, codes, xscale, x, M, out, st);
    return launch_few<1, 1, 4, 2, false>(s, prepared, codes, xscale, x, M, out, st);
  }
  if (M <= 32) return launch_few<2, 2, 8, 1, false>(s, prepared, codes, xscale, x, M, out, st);
  if (M <= 128) return launch_few<2, 4, 8, 1, false>(s, prepared, codes, xscale, x, M, out, st);
  const int64_t big = (int64_t)((M + 255) / 256) * ((s.subtiles() + 15) / 16);
  if (big >= 192) return launch_tile<256, 256, 2, 4>(s, prepared, codes, xscale, M, out, st);
  return launch_tile<128, 128, 2, 4>(s, prepared, codes, xscale, M, out, st);
}

}  // namespace moe
