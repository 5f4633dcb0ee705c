// Norms before and after a block, fused with its gate and residual:
//   b  = y (+ y2)
//   n  = b / sqrt(mean(b^2) + eps) * (post_w + offset)     (b without post_w)
//   h' = residual_scale * h + branch_scale * g * n          g: gate or sigmoid(gate)
//   x  = h' / sqrt(mean(h'^2) + eps) * (pre_w + offset)
// with h' as it is stored (rounded to the residual's type), so that the fused
// call and a call that norms a stored h' agree bit for bit.  Sums in fp32.
//
// Every input is read once and every output written once: a row's values stay
// in registers (WPR waves per row, NV groups of 8 consecutive values per
// lane) between the two row sums.  Bound by memory: M = 4096, H = 4096 with a
// branch, a gate per channel and the next norm takes 25 us (134 MB, 5.3 TB/s),
// M = 16384, H = 7168 with an fp32 residual and two branches 334 us (1.65 GB,
// 4.9 TB/s); a copy of 1 GiB reaches 5.2 TB/s.  M = 1: 3.2 us.
#include <hip/hip_runtime.h>

#include "block.h"
#include "decode.h"

namespace moe {
namespace {

typedef float f32x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x8_t load8_bf16(const uint16_t* p) {
  const uint4 r = *(const uint4*)p;
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  f32x8_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return v;
}

__device__ __forceinline__ f32x8_t load8_f32(const float* p) {
  const float4 a = *(const float4*)p, b = *(const float4*)(p + 4);
  return f32x8_t{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

template <bool F32>
__device__ __forceinline__ f32x8_t load8(const void* p, int64_t i) {
  if constexpr (F32) return load8_f32((const float*)p + i);
  return load8_bf16((const uint16_t*)p + i);
}

__device__ __forceinline__ uint4 pack8(const f32x8_t& v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sum over the WPR waves of a row; `slot` alternates between two LDS areas,
// so one barrier per sum is enough.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* slot) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) v += slot[i];
  }
  return v;
}

// HF32, WF32: the residual's and the weights' type; VGATE: a gate with a
// value per channel (else one per token, or none).  These are compile-time,
// since with the gate's kind and the weights' type as runtime branches hipcc
// (ROCm 7.2) compiled the channel gate's load with an address register that
// was set on the other branch only.
template <int WPR, int NV, bool HF32, bool WF32, bool VGATE>
__global__ void __launch_bounds__(WPR < 4 ? 256 : WPR * 64) block_norm_kernel(NormArgs a) {
  __shared__ float sums[2][WPR > 1 ? WPR : 1];
  constexpr int kRows = WPR < 4 ? 4 / WPR : 1;
  const int64_t row = a.row0 + (int64_t)blockIdx.x * kRows + (kRows > 1 ? threadIdx.x / (64 * WPR) : 0);
  if (kRows > 1 && row >= a.M) return;  // one wave per row: no barrier follows
  const int t = kRows > 1 ? threadIdx.x % (64 * WPR) : threadIdx.x;
  const int H = a.H;
  const int64_t base = row * H;
  const float inv_h = 1.0f / (float)H;
  f32x8_t h[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * WPR * 64 + t) * 8;
    h[i] = c < H ? load8<HF32>(a.h, base + c) : f32x8_t{};
  }
  if (a.y) {
    f32x8_t b[NV];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * WPR * 64 + t) * 8;
      b[i] = c < H ? load8_bf16(a.y + base + c) : f32x8_t{};
      if (a.y2 && c < H) b[i] += load8_bf16(a.y2 + base + c);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += b[i][j] * b[i][j];
    }
    float r = 1.0f;
    if (a.post_w) r = 1.0f / sqrtf(row_sum<WPR>(ss, sums[0]) * inv_h + a.eps);
    float token_gate = 1.0f;
    if (!VGATE && a.gate) {
      if constexpr (WF32)
        token_gate = ((const float*)a.gate)[row];
      else
        token_gate = __uint_as_float((uint32_t)((const uint16_t*)a.gate)[row] << 16);
      if (a.gate_sigmoid) token_gate = 1.0f / (1.0f + __expf(-token_gate));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * WPR * 64 + t) * 8;
      if (c < H) {
        f32x8_t n = b[i];
        if (a.post_w) {
          const f32x8_t w = load8<WF32>(a.post_w, c);
#pragma unroll
          for (int j = 0; j < 8; ++j) n[j] = n[j] * r * (w[j] + a.weight_offset);
        }
        if constexpr (VGATE) {
          f32x8_t g = load8<WF32>(a.gate, row * a.gate_row + c);
          if (a.gate_sigmoid)
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = 1.0f / (1.0f + __expf(-g[j]));
#pragma unroll
          for (int j = 0; j < 8; ++j) n[j] *= g[j];
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) n[j] *= token_gate;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = a.residual_scale * h[i][j] + a.branch_scale * n[j];
        if constexpr (HF32) {
          float* o = (float*)a.h_out + base + c;
          *(float4*)o = make_float4(h[i][0], h[i][1], h[i][2], h[i][3]);
          *(float4*)(o + 4) = make_float4(h[i][4], h[i][5], h[i][6], h[i][7]);
        } else {
          const uint4 p = pack8(h[i]);
          *(uint4*)((uint16_t*)a.h_out + base + c) = p;
          const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            h[i][2 * j] = __uint_as_float(w[j] << 16);
            h[i][2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
          }
        }
      }
    }
  }
  if (a.pre_w) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += h[i][j] * h[i][j];  // values past H are zero
    const float r = 1.0f / sqrtf(row_sum<WPR>(ss, sums[1]) * inv_h + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * WPR * 64 + t) * 8;
      if (c < H) {
        const f32x8_t w = load8<WF32>(a.pre_w, c);
        f32x8_t n;
#pragma unroll
        for (int j = 0; j < 8; ++j) n[j] = h[i][j] * r * (w[j] + a.weight_offset);
        *(uint4*)(a.x_out + base + c) = pack8(n);
      }
    }
  }
}

template <int WPR, int NV>
hipError_t launch_nv(const NormArgs& a, hipStream_t st) {
  constexpr int kRows = WPR < 4 ? 4 / WPR : 1, kThreads = WPR < 4 ? 256 : WPR * 64;
  // A launch has fewer than 2^32 threads (one of more left rows undone, with no
  // error): more rows take several.
  constexpr int64_t kLaunchRows = (1ll << 31) / kThreads * kRows;
  NormArgs part = a;
  for (part.row0 = 0; part.row0 < a.M; part.row0 += kLaunchRows) {
    const int64_t rows = a.M - part.row0 < kLaunchRows ? a.M - part.row0 : kLaunchRows;
    const dim3 grid((unsigned)((rows + kRows - 1) / kRows)), block(kThreads);
#define MOE_NORM(HF, WF, VG) hipLaunchKernelGGL((block_norm_kernel<WPR, NV, HF, WF, VG>), grid, block, 0, st, part)
#define MOE_NORM_G(HF, WF)   \
  if (a.gate_vector)         \
    MOE_NORM(HF, WF, true);  \
  else                       \
    MOE_NORM(HF, WF, false)
    if (a.h_f32 && a.w_f32) {
      MOE_NORM_G(true, true);
    } else if (a.h_f32) {
      MOE_NORM_G(true, false);
    } else if (a.w_f32) {
      MOE_NORM_G(false, true);
    } else {
      MOE_NORM_G(false, false);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
#undef MOE_NORM_G
#undef MOE_NORM
  return hipSuccess;
}

}  // namespace

// One wave per row up to 1024 values, four up to 8192, sixteen up to 32768.
hipError_t launch_block_norm(const NormArgs& a, hipStream_t st) {
  if (a.H <= 512) return launch_nv<1, 1>(a, st);
  if (a.H <= 1024) return launch_nv<1, 2>(a, st);
  if (a.H <= 2048) return launch_nv<4, 1>(a, st);
  if (a.H <= 4096) return launch_nv<4, 2>(a, st);
  if (a.H <= 8192) return launch_nv<4, 4>(a, st);
  if (a.H <= 16384) return launch_nv<16, 2>(a, st);
  return launch_nv<16, 4>(a, st);
}

}  // namespace moe
