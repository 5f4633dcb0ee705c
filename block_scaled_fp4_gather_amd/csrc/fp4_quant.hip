// FP4 quantisation of bf16 or fp32 rows, and its inverse.
//
// MXFP4: blocks of 32, s = 2^(floor(log2 max|x|) - 2) as the OCP MX formats
// define it (2 = exponent of E2M1's largest power of two), at least 2^-127;
// codes = x / s rounded to nearest-even E2M1, magnitudes capped at 6.  The
// conversion instruction divides by the power of two and rounds; all of it is
// exact.
// NVFP4: g = max|x| / (6 * 448) over an expert, blocks of 16, s = max|block| /
// (6 g) rounded to nearest-even E4M3 (at most 448), codes = x / (s g) rounded
// to nearest-even E2M1, capped at 6.  Both roundings are those of the exact
// quotient: it is taken in fp32, within 2^-21 of itself, and where the two
// ends of a range of 2^-20 around that round differently, x is compared with
// the midpoint times the divisor in 64 bits, where that product (at most 32
// significant bits) is exact.
// A block with a NaN or an infinity gets the scale NaN and codes 7.
//
// Bound by memory: a thread takes 8 consecutive values (16 bytes of bf16) four
// times before it works on the first; the 4 or 2 threads of a block are
// consecutive lanes.  16384 x 7168 of bf16 to MXFP4 in 64 to 75 us (4.0 to 4.7
// TB/s) and back in 54 (5.5); 64 x 640 x 2560 of fp32 to NVFP4 in 112 (the
// maxima, 3.8) and 77, and back in 109 (4.4).
#include <hip/hip_runtime.h>

#include "decode.h"
#include "experts.h"
#include "fp4_codes.h"
#include "mxfp8.h"

namespace moe {
namespace {

constexpr int kU = 4;             // loads of a thread in flight
constexpr float kNear = 0x1p-20f; // half the width of the range that has to round alike, relative
constexpr int64_t kMaxBlocks = 8192;

// 8 values as they are read.
template <bool F32>
struct Raw {
  uint4 v[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ float raw_value(const Raw<F32>& r, int i) {
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[F32].x, r.v[F32].y, r.v[F32].z, r.v[F32].w};
  if (F32) return __uint_as_float(w[i]);
  return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
}

// Rows of c8 items of 8 values, ld values apart.
struct Rows {
  int c8;
  uint64_t inverse;  // 2^64 / c8, rounded up
  int64_t gap;       // values between two rows
};

// Item `it`.  Rows without gaps need no division; that of the others is a
// product, too large by one at most (it has fewer than 41 bits, c8 fewer than 18).
template <bool F32, bool STRIDED>
__device__ __forceinline__ Raw<F32> load_raw(const void* x, int64_t it, const Rows& rows) {
  int64_t at = it * 8;
  if (STRIDED) {
    int64_t row = (int64_t)__umul64hi((uint64_t)it, rows.inverse);
    row -= row * rows.c8 > it;
    at += row * rows.gap;
  }
  Raw<F32> r;
  const uint4* const p = (const uint4*)((const uint8_t*)x + at * (F32 ? 4 : 2));
  r.v[0] = p[0];
  if (F32) r.v[F32] = p[F32];
  return r;
}

// Largest magnitude of the 8 values, as bits: a NaN or an infinity compares
// above every number.
template <bool F32>
__device__ __forceinline__ uint32_t raw_amax(const Raw<F32>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(raw_value(r, i)) & 0x7FFFFFFFu);
  return m;
}

__device__ __forceinline__ bool finite_bits(uint32_t b) { return b < 0x7F800000u; }

// Code of v with |v| / unit rounded exactly, unit > 0: of the midpoints between
// the values 0 0.5 1 1.5 2 3 4 6, those that lie below it are counted, and one
// that it equals where the code below is odd.  (Their products with the unit are
// made from each other, exactly: as constants they would fill scalar registers.)
__device__ __forceinline__ uint32_t e2m1_exact(float v, double unit) {
  const double a = fabs((double)v), h = 0.5 * unit;
  const double t0 = 0.5 * h, t1 = t0 + h, t2 = t1 + h, t3 = t2 + h, t4 = 2.0 * t2, t5 = 2.0 * t3, t6 = 2.0 * t4;
  const int c = (a > t0) + (a >= t1) + (a > t2) + (a >= t3) + (a > t4) + (a >= t5) + (a > t6);
  return (uint32_t)c | (__float_as_uint(v) >> 31 << 3);
}

// Codes of 8 finite values over 1 / inv, unrounded by more than 2^-21 or not
// at all.
template <bool F32>
__device__ __forceinline__ uint32_t e2m1_codes(const Raw<F32>& r, float inv) {
  uint32_t w = 0;
#define MOE_PAIR(I) \
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, raw_value(r, 2 * I) * inv, raw_value(r, 2 * I + 1) * inv, 1.0f, I)
  MOE_PAIR(0);
  MOE_PAIR(1);
  MOE_PAIR(2);
  MOE_PAIR(3);
#undef MOE_PAIR
  return w;
}

// MXFP4: 8 values and their block's scale byte.
template <bool F32>
__device__ __forceinline__ uint32_t mxfp4_codes(const Raw<F32>& r, uint32_t byte) {
  if constexpr (!F32) return mxfp4_codes8(r.v[0], byte);
  if (byte == 255u) return 0x77777777u;
  const float s = mxfp4_scale(byte);
  uint32_t w = 0;
#define MOE_PAIR(I) w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, raw_value(r, 2 * I), raw_value(r, 2 * I + 1), s, I)
  MOE_PAIR(0);
  MOE_PAIR(1);
  MOE_PAIR(2);
  MOE_PAIR(3);
#undef MOE_PAIR
  return w;
}

// An expert's global scale and what the blocks need of it.
struct Global {
  double g;
  float g32, inv6;  // 1 / (6 g)
  bool plain;       // g and the quotients stay far from the ends of fp32
};

__device__ __forceinline__ Global global_of(float g) {
  Global o;
  o.g = g;
  o.g32 = g;
  o.inv6 = (float)(1.0 / (6.0 * (double)g));
  o.plain = g >= 0x1p-60f && g <= 0x1p60f;
  return o;
}

// E4M3 byte of a block's scale, amax / (6 g), from amax's bits (finite).
__device__ __forceinline__ uint32_t nvfp4_scale(uint32_t amax_bits, const Global& g) {
  const float amax = __uint_as_float(amax_bits);
  float q = amax * g.inv6;
  if (!g.plain) {
    const double d = (double)amax / (6.0 * g.g);
    q = (float)fmin(d, 512.0);
  }
  q = fminf(q, 448.0f);
  const uint32_t two = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q * (1.0f - kNear), fminf(q * (1.0f + kNear), 448.0f), 0, false);
  const uint32_t lo = two & 0xFFu, hi = (two >> 8) & 0xFFu;
  if (lo == hi) return lo;
  // hi = lo + 1: the midpoint of the two
  const double t = 0.5 * ((double)e4m3_value(lo) + (double)e4m3_value(hi)) * 6.0 * g.g;
  return ((lo & 1u) ? (double)amax >= t : (double)amax > t) ? hi : lo;
}

template <bool F32>
__device__ __forceinline__ uint32_t nvfp4_codes(const Raw<F32>& r, uint32_t byte, const Global& g) {
  if (byte == 0) return 0;
  const float s = e4m3_value(byte);
  const float inv = 1.0f / (s * g.g32);
  const uint32_t lo = e2m1_codes(r, inv * (1.0f - kNear)), hi = e2m1_codes(r, inv * (1.0f + kNear));
  if (lo == hi && g.plain) return lo;
  const double unit = (double)s * g.g;
  uint32_t w = 0;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    float v = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) v = i == j ? raw_value(r, j) : v;
    w |= e2m1_exact(v, unit) << (4 * i);
  }
  return w;
}

template <bool NV, bool F32, bool STRIDED>
__global__ void __launch_bounds__(256) fp4_quantize_kernel(QuantArgs a, Rows rows, int64_t items, int parts) {
  const int64_t step = (int64_t)gridDim.x * 256;
  // From the last expert back: the one that fp4_amax_kernel read last may still be
  // in the cache before HBM (64 x 640 x 2560 of fp32: 85 -> 78 us, and the inverse,
  // which starts at the first, 120 -> 112).
  for (int64_t e = a.experts - 1 - blockIdx.y; e >= 0; e -= gridDim.y) {
    const uint8_t* const x = (const uint8_t*)a.x + e * a.rows * a.ld * (F32 ? 4 : 2);
    uint32_t* const codes = (uint32_t*)(a.codes + e * a.rows * (a.K / 2));
    uint8_t* const scales = a.scales + e * a.rows * (a.K / (NV ? 16 : 32));
    Global g{};
    float g32 = 0.0f;
    if (NV) {
      if (a.partial) {
        // the expert's largest finite magnitude over the workgroups that looked for it
        __shared__ uint32_t wmax[4];
        uint32_t m = threadIdx.x < (unsigned)parts ? a.partial[e * kQuantParts + threadIdx.x] : 0u;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
        __syncthreads();  // an earlier expert's maxima have been read
        if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
        __syncthreads();
        m = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
        g32 = __uint_as_float(m) / 2688.0f;
        if (blockIdx.x == 0 && threadIdx.x == 0) a.g_out[e] = g32;
      } else {
        g32 = a.global[e];
      }
      g = global_of(g32);
    }
    for (int64_t it0 = (int64_t)blockIdx.x * 256 + threadIdx.x; it0 < items; it0 += kU * step) {
      Raw<F32> r[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (it0 + u * step < items) r[u] = load_raw<F32, STRIDED>(x, it0 + u * step, rows);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t it = it0 + u * step;
        if (it >= items) break;  // the lanes of a block leave together: items are whole blocks
        uint32_t m = raw_amax(r[u]);
        m = max(m, (uint32_t)__shfl_xor((int)m, 1));
        if (!NV) m = max(m, (uint32_t)__shfl_xor((int)m, 2));
        uint32_t byte, w;
        if (NV) {
          // a scale of zero holds zeros; one that is negative, infinite or NaN holds nothing
          const bool ok = finite_bits(m) && g32 >= 0.0f && finite_bits(__float_as_uint(g32) & 0x7FFFFFFFu);
          byte = !ok ? 0x7Fu : g32 > 0.0f ? nvfp4_scale(m, g) : 0u;
          w = ok ? nvfp4_codes(r[u], byte, g) : 0x77777777u;
        } else {
          byte = mxfp4_scale_byte(m);
          w = mxfp4_codes(r[u], byte);
        }
        codes[it] = w;
        if (NV ? (it & 1) == 0 : (it & 3) == 0) scales[it / (NV ? 2 : 4)] = (uint8_t)byte;
      }
    }
  }
}

// The largest finite magnitude of each expert, a part per workgroup.
template <bool F32, bool STRIDED>
__global__ void __launch_bounds__(256) fp4_amax_kernel(QuantArgs a, Rows rows, int64_t items) {
  __shared__ uint32_t wmax[4];
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t e = blockIdx.y; e < a.experts; e += gridDim.y) {
    const uint8_t* const x = (const uint8_t*)a.x + e * a.rows * a.ld * (F32 ? 4 : 2);
    uint32_t m = 0;
    for (int64_t it0 = (int64_t)blockIdx.x * 256 + threadIdx.x; it0 < items; it0 += kU * step) {
      Raw<F32> r[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) r[u] = load_raw<F32, STRIDED>(x, min(it0 + u * step, items - 1), rows);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t all = raw_amax(r[u]);
        if (finite_bits(all)) {
          m = max(m, all);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t b = __float_as_uint(raw_value(r[u], i)) & 0x7FFFFFFFu;
            m = max(m, finite_bits(b) ? b : 0u);
          }
        }
      }
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0)
      a.partial[e * kQuantParts + blockIdx.x] = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
  }
}

template <bool NV, bool F32>
__global__ void __launch_bounds__(256) fp4_dequantize_kernel(DequantArgs a, int64_t items) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t e = blockIdx.y; e < a.experts; e += gridDim.y) {
    const uint32_t* const codes = (const uint32_t*)(a.codes + e * a.rows * (a.K / 2));
    const uint8_t* const scales = a.scales + e * a.rows * (a.K / (NV ? 16 : 32));
    uint4* const out = (uint4*)((uint8_t*)a.out + e * a.rows * a.K * (F32 ? 4 : 2));
    const float g = NV ? a.global[e] : 1.0f;
    for (int64_t it0 = (int64_t)blockIdx.x * 256 + threadIdx.x; it0 < items; it0 += kU * step) {
      uint32_t w[kU], sb[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t it = min(it0 + u * step, items - 1);
        w[u] = codes[it];
        sb[u] = scales[it / (NV ? 2 : 4)];
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t it = it0 + u * step;
        if (it >= items) break;
        // code times block scale is exact in fp32 (2 and 4 significant bits) but for MXFP4's ends; the global
        // rounds it, and bf16 outputs are rounded once more
        const float s = NV ? __builtin_amdgcn_cvt_f32_fp8((int)sb[u], 0) : ue8m0_to_f32(sb[u]);
        f32x2_t f[4];
        fp4x8_to_f32(w[u], f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[i].x = f[i].x * s;
          f[i].y = f[i].y * s;
          if (NV) {
            f[i].x *= g;
            f[i].y *= g;
          }
        }
        if constexpr (F32) {
          out[2 * it] = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                                   __float_as_uint(f[1].y));
          out[2 * it + 1] = make_uint4(__float_as_uint(f[2].x), __float_as_uint(f[2].y), __float_as_uint(f[3].x),
                                       __float_as_uint(f[3].y));
        } else {
          out[it] = make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y), pack_bf16(f[2].x, f[2].y),
                               pack_bf16(f[3].x, f[3].y));
        }
      }
    }
  }
}

// Workgroups for `items` items of each of `experts` experts: enough that a
// thread takes kU, at most kMaxBlocks in all.
dim3 grid_for(int64_t items, int64_t experts, int64_t most) {
  const int64_t y = experts < 65535 ? experts : 65535;
  int64_t x = (items + 256 * kU - 1) / (256 * kU);
  const int64_t lim = most / y > 1 ? most / y : 1;
  x = x < lim ? x : lim;
  return dim3((unsigned)x, (unsigned)y);
}

template <bool NV, bool F32>
hipError_t quantize(QuantArgs a, hipStream_t st) {
  const bool strided = a.ld != a.K;
  if (!NV && !strided) {  // nothing tells the experts apart
    a.rows *= a.experts;
    a.experts = 1;
  }
  const int64_t items = a.rows * (a.K / 8);
  // K / 8 is 2 or more
  const Rows rows{a.K / 8, UINT64_MAX / (uint64_t)(a.K / 8) + 1, a.ld - a.K};
  int parts = 0;
  if (NV && a.partial) {
    dim3 grid = grid_for(items, a.experts, 2048);
    if (grid.x > kQuantParts) grid.x = kQuantParts;
    parts = (int)grid.x;
    if (strided)
      hipLaunchKernelGGL((fp4_amax_kernel<F32, true>), grid, dim3(256), 0, st, a, rows, items);
    else
      hipLaunchKernelGGL((fp4_amax_kernel<F32, false>), grid, dim3(256), 0, st, a, rows, items);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid = grid_for(items, a.experts, kMaxBlocks);
  if (strided)
    hipLaunchKernelGGL((fp4_quantize_kernel<NV, F32, true>), grid, dim3(256), 0, st, a, rows, items, parts);
  else
    hipLaunchKernelGGL((fp4_quantize_kernel<NV, F32, false>), grid, dim3(256), 0, st, a, rows, items, parts);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp4_quantize(const QuantArgs& a, hipStream_t st) {
  if (a.nvfp4) return a.f32 ? quantize<true, true>(a, st) : quantize<true, false>(a, st);
  return a.f32 ? quantize<false, true>(a, st) : quantize<false, false>(a, st);
}

hipError_t launch_fp4_dequantize(const DequantArgs& in, hipStream_t st) {
  DequantArgs a = in;
  if (!a.nvfp4) {
    a.rows *= a.experts;
    a.experts = 1;
  }
  const int64_t items = a.rows * (a.K / 8);
  const dim3 grid = grid_for(items, a.experts, kMaxBlocks);
#define MOE_DEQ(NV, F32) hipLaunchKernelGGL((fp4_dequantize_kernel<NV, F32>), grid, dim3(256), 0, st, a, items)
  if (a.nvfp4) {
    if (a.f32) MOE_DEQ(true, true);
    else MOE_DEQ(true, false);
  } else {
    if (a.f32) MOE_DEQ(false, true);
    else MOE_DEQ(false, false);
  }
#undef MOE_DEQ
  return hipGetLastError();
}

}  // namespace moe
