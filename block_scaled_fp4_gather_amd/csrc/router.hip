// Router of the expert layer: logits z = x Wr^T, scores, the k experts of
// each token and their weights.
//
// The experts taken, and their order, are those of the scores in exact
// arithmetic (up to 64-bit rounding), whatever the batch: the logits come
// from the matrix cores in fp32 with a bound on their error, and where two
// scores that decide something lie within it, the wave that selects for this
// token recomputes the logits of the experts concerned in 64 bits.  So the
// same token gets the same experts alone and in any batch.
//
// Two launches: route_logits (partial sums over K slices, so that few tokens
// still fill the chip) and route_select (one wave per token).
#include <hip/hip_runtime.h>

#include "block.h"
#include "decode.h"
#include "gemm_util.h"

namespace moe {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

// ---- weight preparation

// bf16 of v, nearest-even, as fp32
__device__ __forceinline__ float as_bf16(float v) { return __uint_as_float((uint32_t)f32_to_bf16_rne(v) << 16); }

template <bool F32>
__global__ void __launch_bounds__(256)
    router_prepare_kernel(RouterShape s, const void* __restrict__ weight, uint8_t* __restrict__ prepared) {
  const int kb = s.kblocks();
  const int64_t chunks = (int64_t)s.subtiles() * kb * 64;
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t it = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; it < chunks; it += stride) {
    const int lane = (int)(it & 63);
    const int64_t sb = it >> 6;
    const int e = (int)(sb / kb) * 16 + (lane & 15);
    const int h0 = (int)(sb % kb) * 32 + (lane >> 4) * 8;
    const bool in = e < s.E && h0 < s.H;  // H % 8 == 0
    uint16_t p[3][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (F32) {
        // three bf16 terms: each remainder is exact, and 3 x 8 bits hold all
        // 24 (rounding to nearest leaves a remainder of at most half a step,
        // so a term never needs more bits than are left)
        const float v = in ? ((const float*)weight)[(int64_t)e * s.H + h0 + j] : 0.0f;
        const float a = as_bf16(v);
        const float b = as_bf16(v - a);
        p[0][j] = (uint16_t)(__float_as_uint(a) >> 16);
        p[1][j] = (uint16_t)(__float_as_uint(b) >> 16);
        p[2][j] = f32_to_bf16_rne((v - a) - b);
      } else {
        p[0][j] = in ? ((const uint16_t*)weight)[(int64_t)e * s.H + h0 + j] : (uint16_t)0;
      }
    }
#pragma unroll
    for (int q = 0; q < (F32 ? 3 : 1); ++q) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = (uint32_t)p[q][2 * j] | ((uint32_t)p[q][2 * j + 1] << 16);
      *(uint4*)(prepared + q * s.plane_bytes() + it * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Norms, rounded up: the fp32 sum is off by less than 2^-13 of itself for
// H <= 65536 (256 lanes, trees).
template <bool F32>
__global__ void __launch_bounds__(256)
    router_norms_kernel(RouterShape s, const void* __restrict__ weight, float* __restrict__ norms) {
  __shared__ float sums[4];
  const int e = blockIdx.x;
  float ss = 0.0f;
  for (int h = threadIdx.x; h < s.H; h += 256) {
    const float v = F32 ? ((const float*)weight)[(int64_t)e * s.H + h]
                        : __uint_as_float((uint32_t)((const uint16_t*)weight)[(int64_t)e * s.H + h] << 16);
    ss += v * v;
  }
  for (int d = 32; d >= 1; d >>= 1) ss += __shfl_xor(ss, d);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = ss;
  __syncthreads();
  if (threadIdx.x == 0) norms[e] = sqrtf(sums[0] + sums[1] + sums[2] + sums[3]) * 1.001f + 1e-30f;
}

// ---- logits

// How a call of M tokens is cut: 16 tt tokens and 128 experts per workgroup,
// H in `splits` slices of `per` K blocks.
struct LogitPlan {
  int tt, splits, per;
};

LogitPlan logit_plan(const RouterShape& s, int64_t M) {
  LogitPlan p;
  p.tt = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  const int64_t groups = ((M + 16 * p.tt - 1) / (16 * p.tt)) * ((s.E + 127) / 128);
  int64_t splits = 512 / groups;
  splits = splits < 1 ? 1 : splits > 16 ? 16 : splits;
  const int kb = s.kblocks();
  if (splits > kb) splits = kb;
  p.per = (int)((kb + splits - 1) / splits);
  p.splits = (kb + p.per - 1) / p.per;
  return p;
}

// Partial logits f32 [split][M][16 subtiles] and partial sums of x^2
// f32 [split][M].
int64_t partial_floats(const RouterShape& s, int64_t M) {
  const LogitPlan p = logit_plan(s, M);
  return p.splits * M * (16 * (int64_t)s.subtiles() + 1);
}

// Wave w of a workgroup takes expert subtiles 2 w and 2 w + 1 of its 128
// experts, the 16 TT tokens and the K blocks of its slice.
template <int TT, int NP>
__global__ void __launch_bounds__(256)
    route_logits_kernel(RouterShape s, const uint8_t* __restrict__ prepared, const uint16_t* __restrict__ x, int M,
                        int per, float* __restrict__ part, float* __restrict__ xx) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int kb = s.kblocks(), ns = s.subtiles(), Ep = 16 * ns;
  const int64_t tok0 = (int64_t)blockIdx.x * (16 * TT);
  const int sub0 = blockIdx.y * 8 + 2 * wave;
  const int b0 = blockIdx.z * per, b1 = min(kb, b0 + per);
  if (sub0 >= ns) return;
  const bool two = sub0 + 1 < ns;
  const int64_t plane = s.plane_bytes();
  const bool norms = blockIdx.y == 0 && wave == 0;
  f32x4_t acc[2][TT];
  float sq[TT];
  const uint16_t* xr[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    acc[0][t] = acc[1][t] = f32x4_t{};
    sq[t] = 0.0f;
    xr[t] = x + min(tok0 + 16 * t + r, (int64_t)M - 1) * s.H + g * 8;
  }
  for (int b = b0; b < b1; ++b) {
    bf16x8_t bop[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (b * 32 + g * 8 < s.H) v = *(const uint4*)(xr[t] + b * 32);
      bop[t] = __builtin_bit_cast(bf16x8_t, v);
      if (norms)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v = (float)bop[t][j] * 0x1p32f;  // squares of 2^-95 .. 2^31 neither vanish nor overflow
          sq[t] = fmaf(v, v, sq[t]);
        }
    }
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int64_t at = ((int64_t)(f && two ? sub0 + 1 : sub0) * kb + b) * 1024 + lane * 16;
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        const bf16x8_t a = __builtin_bit_cast(bf16x8_t, *(const uint4*)(prepared + q * plane + at));
#pragma unroll
        for (int t = 0; t < TT; ++t)
          acc[f][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, bop[t], acc[f][t], 0, 0, 0);
      }
    }
  }
  const int64_t split = blockIdx.z;
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int64_t m = tok0 + 16 * t + r;
    if (m < M) {
      float* o = part + (split * M + m) * Ep + sub0 * 16 + 4 * g;
      *(f32x4_t*)o = acc[0][t];
      if (two) *(f32x4_t*)(o + 16) = acc[1][t];
    }
    if (norms) {
      float v = sq[t];
      v += __shfl_xor(v, 16);
      v += __shfl_xor(v, 32);
      if (m < M && g == 0) xx[split * M + m] = v;
    }
  }
}

// ---- selection: one wave per token, lane l holds experts l + 64 i

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = fmax(v, __shfl_xor(v, d));
  return v;
}

// Largest value over the wave, in lane order moves (row shifts, then the
// two row broadcasts; lane 63 ends with the result): an eighth of the
// latency of six exchanges through LDS.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#define MOE_STEP(CTRL) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false))
  MOE_STEP(0x111);  // row_shr:1
  MOE_STEP(0x112);
  MOE_STEP(0x114);
  MOE_STEP(0x118);
  MOE_STEP(0x142);  // row_bcast:15
  MOE_STEP(0x143);  // row_bcast:31
#undef MOE_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// fp32 as an unsigned integer of the same order, above 0 for every number;
// 0 stands for "not to be taken".
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}

// Largest key of the wave (each lane's NI) and its lowest expert.
template <int NI>
__device__ __forceinline__ uint32_t wave_best_key(const uint32_t (&key)[NI], int lane, int& e) {
  uint32_t v = key[0];
  int at = 0;
#pragma unroll
  for (int i = 1; i < NI; ++i)
    if (key[i] > v) {
      v = key[i];
      at = i;
    }
  const uint32_t best = wave_max_u32(v);
  const uint64_t owners = __ballot(v == best);
  if (__popcll(owners) == 1) {
    const int l = __ffsll((unsigned long long)owners) - 1;
    e = __builtin_amdgcn_readlane(at, l) * 64 + l;
  } else {
    e = 0x7FFF - (int)wave_max_u32(v == best ? (uint32_t)(0x7FFF - (at * 64 + lane)) : 0u);
  }
  return best;
}

// Largest value and its expert, ties to the lowest index.
__device__ __forceinline__ void wave_best(double& v, int& e) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const double ov = __shfl_xor(v, d);
    const int oe = __shfl_xor(e, d);
    if (ov > v || (ov == v && oe < e)) {
      v = ov;
      e = oe;
    }
  }
}

// Orders a wave's LDS accesses for the compiler; the hardware runs them in
// order.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The same value, unknown to the compiler: what it derived from v before (a
// mask register per comparison) is not kept for later uses.
__device__ __forceinline__ int renew(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Logit of expert e in 64 bits: products of bf16 values are exact.
__device__ __forceinline__ double exact_logit(const RouterShape& s, const uint8_t* __restrict__ prepared,
                                              const uint16_t* __restrict__ xr, int e, int lane) {
  const int kb = s.kblocks();
  double sum = 0.0;
  for (int c = lane; c * 8 < s.H; c += 64) {
    const uint4 xv = *(const uint4*)(xr + c * 8);
    const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
    const int64_t at = ((int64_t)(e >> 4) * kb + (c >> 2)) * 1024 + ((c & 3) * 16 + (e & 15)) * 16;
    for (int q = 0; q < s.planes; ++q) {
      const uint4 wv = *(const uint4*)(prepared + q * s.plane_bytes() + at);
      const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum = fma((double)__uint_as_float(xw[j] << 16), (double)__uint_as_float(ww[j] << 16), sum);
        sum = fma((double)__uint_as_float(xw[j] & 0xFFFF0000u), (double)__uint_as_float(ww[j] & 0xFFFF0000u), sum);
      }
    }
  }
  return wave_sum(sum);
}

constexpr double kNone = -__builtin_inf();
constexpr int kNobody = 1 << 30;

// What a wave of the selection keeps in LDS.
template <int NI>
struct SelectLds {
  double z[64 * NI];     // the token's logits, in 64 bits where recomputed
  double t[64 * NI];     // scores in 64 bits of what was recomputed (by expert, then by list place)
  uint16_t e[64 * NI];   // list: experts, best first
  uint16_t run[64 * NI]; // list: first place of the run of unsure neighbours a place belongs to
  int taken[64];
  // where the results go: kept here while the experts are chosen, which needs
  // all the scalar registers
  int* ids;
  float *w, *logits;
};

// Recomputes the logits of the experts in `want` (bit i: this lane's expert
// lane + 64 i).
template <int NI>
__device__ __forceinline__ void refine(const RouterShape& s, SelectLds<NI>& L, const uint8_t* __restrict__ prepared,
                                       const uint16_t* __restrict__ xr, uint32_t want, int lane) {
#pragma unroll 1
  for (int i = 0; i < NI; ++i) {
    uint64_t todo = __ballot(want >> i & 1u);
    while (todo) {
      const int l = __ffsll((unsigned long long)todo) - 1;
      todo &= todo - 1;
      const double v = exact_logit(s, prepared, xr, l + 64 * i, lane);
      if (lane == l) L.z[lane + 64 * i] = v;
    }
  }
  wave_sync();
}

// Which experts a token takes, best first, into L.taken; returns how many.
//
// Scores are first compared in 32 bits with a common bound on their errors.
// Groups: if the border between the groups taken and left is unsure, the
// logits of all that could be among a group's two largest are recomputed and
// the groups compared in 64 bits.  Experts: the list of the largest scores is
// cut into runs of neighbours nearer than twice the bound, as far as the run
// that holds the k-th; the order of runs is certain, and within a run it is
// that of the recomputed scores.
template <int NI, bool GROUPS>
__device__ __forceinline__ int select_experts(const RouterShape& s, SelectLds<NI>& L,
                                              const uint8_t* __restrict__ prepared, const uint16_t* __restrict__ xr,
                                              const float (&z)[NI], float bound, const float* __restrict__ bias,
                                              int lane) {
  const int E = s.E;
  const bool scored = bias != nullptr || GROUPS;
  float t[NI];
  float err = bound, zmax = 0.0f;
  if (scored) {
    if (s.sigmoid) {
#pragma unroll
      for (int i = 0; i < NI; ++i) t[i] = 1.0f / (1.0f + expf(-z[i]));
      err = 0.25f * bound;
    } else {
      uint32_t key = 0;
#pragma unroll
      for (int i = 0; i < NI; ++i) key = max(key, z[i] == z[i] ? order_key(z[i]) : 0u);
      zmax = key_value(wave_max_u32(key));
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        t[i] = expf(z[i] - zmax);
        sum += t[i];
      }
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
#pragma unroll
      for (int i = 0; i < NI; ++i) t[i] /= sum;
      err = 2.0f * bound;
    }
    err += 0x1p-20f;  // scores are at most 1, with a few roundings of 2^-24 each
    if (bias) {
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const float b = lane + 64 * i < E ? bias[lane + 64 * i] : 0.0f;
        t[i] += b;
        if (fabsf(b) < __builtin_inff()) most = fmaxf(most, fabsf(b));
      }
      err += __uint_as_float(wave_max_u32(__float_as_uint(most))) * 0x1p-22f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i) t[i] = z[i];
  }
  lane = renew(lane);
  uint32_t key[NI], open = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const bool in = lane + 64 * i < E;
    key[i] = in && t[i] > -__builtin_inff() ? order_key(t[i]) : 0u;  // not NaN
    if (in) open |= 1u << i;
  }
  // With a bias on a softmax a recomputed score still carries the other
  // logits' errors, through the sum: then all are recomputed.  (Without one
  // the sum is a common factor.)
  const bool whole = bias != nullptr && !s.sigmoid;
  bool all = !(bound < __builtin_inff());
  int n = 0;
  bool runs = false;

#pragma unroll 1
  while (true) {
    lane = renew(lane);
    double total = 1.0;
    if (all) {
      if (bound != 0.0f) refine<NI>(s, L, prepared, xr, open, lane);
      double mx = kNone, sum = 0.0;
#pragma unroll 1
      for (int e = lane; e < E; e += 64) mx = fmax(mx, L.z[e]);
      zmax = (float)wave_max(mx);
      if (whole) {
#pragma unroll 1
        for (int e = lane; e < E; e += 64) sum += exp(L.z[e] - (double)zmax);
        total = wave_sum(sum);
      }
    }
    // score in 64 bits; what may not be taken gets -infinity
    auto exact_score = [&](int e, bool for_groups) {
      double v = L.z[e];
      if (bias || for_groups) {
        v = exp(s.sigmoid ? -v : v - (double)zmax);
        v = s.sigmoid ? 1.0 / (1.0 + v) : v / total;
        if (bias) v += (double)bias[e];
      }
      return v == v ? v : kNone;
    };

    uint64_t in_groups = ~0ull;
    const int size = GROUPS ? E / s.groups : E;
    if constexpr (GROUPS) {
      float score = -__builtin_inff();  // lane q: that of group q
      uint32_t near = 0;                // could be among the two largest of their groups
#pragma unroll 1
      for (int q = 0; q < s.groups; ++q) {
        lane = renew(lane);
        uint32_t in[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) in[i] = (lane + 64 * i) / size == q ? key[i] : 0u;
        int e1, e2;
        const uint32_t k1 = wave_best_key<NI>(in, lane, e1);
        uint32_t rest[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) rest[i] = lane + 64 * i == e1 ? 0u : in[i];
        const uint32_t k2 = wave_best_key<NI>(rest, lane, e2);
        if (lane == q && k2 != 0u) score = key_value(k1) + key_value(k2);
        const float floor = k2 != 0u ? key_value(k2) - 2.0f * err : -__builtin_inff();
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (in[i] != 0u && !(key_value(in[i]) < floor)) near |= 1u << i;
      }
      uint32_t gk[1] = {lane < s.groups ? (score == score ? order_key(score) : 1u) : 0u};
      float last = 0.0f, next = -__builtin_inff();
      in_groups = 0;
#pragma unroll 1
      for (int q = 0; q <= s.top_groups && q < s.groups; ++q) {
        int e;
        const float v = key_value(wave_best_key<1>(gk, lane, e));
        if (q == s.top_groups) {
          next = v;
          break;
        }
        last = v;
        in_groups |= 1ull << e;
        if (lane == e) gk[0] = 0u;
      }
      // two sums of two scores, and the sums' own roundings
      if (all || (s.top_groups < s.groups &&
                  !(last - next > 4.0f * err + 0x1p-22f * (fabsf(last) + fabsf(next))))) {
        if (whole && !all) {
          all = true;
          continue;
        }
        if (all) near = open;
        if (!all && bound != 0.0f) refine<NI>(s, L, prepared, xr, near, lane);
#pragma unroll 1
        for (int i = 0; i < NI; ++i) {
          const int e = lane + 64 * i;
          L.t[e] = near >> i & 1u ? exact_score(e, true) : kNone;
        }
        wave_sync();
        double gs = kNone;
#pragma unroll 1
        for (int q = 0; q < s.groups; ++q) {
          double v1 = kNone, v2 = kNone;
          int e1 = kNobody, e2 = kNobody;
          for (int e = q * size + lane; e < (q + 1) * size; e += 64)
            if (L.t[e] > v1) {
              v1 = L.t[e];
              e1 = e;
            }
          wave_best(v1, e1);
          for (int e = q * size + lane; e < (q + 1) * size; e += 64)
            if (e != e1 && L.t[e] > v2) {
              v2 = L.t[e];
              e2 = e;
            }
          wave_best(v2, e2);
          if (lane == q && e2 != kNobody) gs = v1 + v2;
        }
        in_groups = 0;
#pragma unroll 1
        for (int q = 0; q < s.top_groups; ++q) {
          const bool free = lane < s.groups && !(in_groups >> lane & 1ull);
          double v = free ? gs : kNone;
          int e = free ? lane : kNobody;
          wave_best(v, e);
          in_groups |= 1ull << e;
        }
        wave_sync();
      }
    }

    // the list: key of expert e in the groups taken; within them, without a
    // bias, the order is that of the logits
    lane = renew(lane);
    uint32_t left[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      left[i] = GROUPS && !(in_groups >> ((lane + 64 * i) / size & 63) & 1ull) ? 0u : key[i];
      if (!bias && left[i] != 0u) left[i] = order_key(z[i]);
    }
    n = 0;
    runs = all;
    if (all) {  // one run of all that may be taken, in any order
#pragma unroll 1
      for (int i = 0; i < NI; ++i) {
        const int e = lane + 64 * i;
        const bool in = e < E && (!GROUPS || (in_groups >> (e / size & 63) & 1ull)) &&
                        exact_score(e, false) > kNone;
        const uint64_t who = __ballot(in);
        if (in) {
          const int at = n + __popcll(who & ((1ull << lane) - 1ull));
          L.e[at] = (uint16_t)e;
          L.run[at] = 0;
        }
        n += __popcll(who);
      }
    } else {
      const float apart = 2.0f * (bias ? err : bound);
      float prev = 0.0f;
      int start = 0;
#pragma unroll 1
      while (true) {
        lane = renew(lane);
        int e;
        const uint32_t best = wave_best_key<NI>(left, lane, e);
        if (best == 0u) break;
        const float v = key_value(best);
        const bool unsure = n > 0 && apart > 0.0f && !(prev - v > apart);
        if (n >= s.k && !unsure) break;
        if (!unsure) start = n;
        runs |= unsure;
        if (lane == 0) {
          L.e[n] = (uint16_t)e;
          L.run[n] = (uint16_t)start;
        }
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (lane + 64 * i == e) left[i] = 0u;
        prev = v;
        ++n;
      }
    }
    wave_sync();
    if (runs && whole && !all) {
      all = true;
      continue;
    }

    if (!runs) {
      if (lane < n) L.taken[lane] = L.e[lane];
    } else {
      if (!all && bound != 0.0f) {
        uint32_t want = 0;
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          const int e = L.e[j], r = L.run[j];
          if (e % 64 == lane && (r != j || (j + 1 < n && L.run[j + 1] == r))) want |= 1u << (e / 64);
        }
        refine<NI>(s, L, prepared, xr, want, lane);
      }
#pragma unroll 1
      for (int j = lane; j < n; j += 64) L.t[j] = exact_score(L.e[j], false);
      wave_sync();
#pragma unroll 1
      for (int j = lane; j < n; j += 64) {
        const int r = L.run[j], e = L.e[j];
        const double v = L.t[j];
        int at = r;
        for (int i = r; i < n && L.run[i] == r; ++i) at += L.t[i] > v || (L.t[i] == v && L.e[i] < e);
        if (at < s.k) L.taken[at] = e;
      }
    }
    wave_sync();
    return n < s.k ? n : s.k;
  }
}

template <int NI, bool GROUPS>
__global__ void __launch_bounds__(256)
    route_select_kernel(RouterShape s, const uint8_t* __restrict__ prepared, const uint16_t* __restrict__ x, int M,
                        int splits, float coef, const float* __restrict__ part, const float* __restrict__ xx,
                        const float* __restrict__ bias, int* __restrict__ ids, float* __restrict__ wout,
                        float* __restrict__ logits) {
  __shared__ SelectLds<NI> lds[4];
  int lane = threadIdx.x & 63;
  const int64_t m = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (m >= M) return;  // waves do not wait for each other
  SelectLds<NI>& L = lds[threadIdx.x >> 6];
  const int E = s.E, Ep = 16 * s.subtiles(), k = s.k;
  const float* const norms = (const float*)(prepared + s.norms_offset());

  float z[NI];
  uint32_t wn = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    z[i] = 0.0f;
    if (lane + 64 * i < E) wn = max(wn, __float_as_uint(norms[lane + 64 * i]));  // norms are not negative
  }
  float x2 = 0.0f;
  const float* p0 = part + m * Ep + lane;
#pragma unroll 4
  for (int q = 0; q < splits; ++q) {
    x2 += xx[(int64_t)q * M + m];  // of 2^32 x
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (lane + 64 * i < E) z[i] += p0[(int64_t)q * M * Ep + 64 * i];
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    if (lane + 64 * i >= E) z[i] = -__builtin_inff();
    L.z[lane + 64 * i] = (double)z[i];
  }
  if (lane == 0) {
    L.ids = ids + m * k;
    L.w = wout + m * k;
    L.logits = logits ? logits + m * E : nullptr;
  }
  wave_sync();
  // ||x|| ||w|| times the coefficient of the plan, which counts the roundings
  const float bound = sqrtf(x2) * (1.001f * 0x1p-32f) * __uint_as_float(wave_max_u32(wn)) * coef;
  const int kept = select_experts<NI, GROUPS>(s, L, prepared, x + m * s.H, z, bound, bias, lane);
  lane = renew(lane);

  // weights: the taken experts' probabilities, from their logits
  const bool on = lane < kept;
  const int taken = on ? L.taken[lane] : 0;
  const double zw = L.z[taken];
  const double mx = s.sigmoid || kept == 0 ? 0.0 : wave_max(on ? zw : kNone);  // of those taken
  double p = exp(s.sigmoid ? -zw : zw - mx);
  if (s.sigmoid) {
    p = on ? 1.0 / (1.0 + p) : 0.0;
  } else {
    p = on ? p : 0.0;
    if (!s.renorm) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (lane + 64 * i < E) sum += expf((float)(L.z[lane + 64 * i] - mx));
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
      p /= (double)sum;
    }
  }
  if (s.renorm) {
    const double sum = wave_sum(p);
    p = sum == 0.0 ? 0.0 : p / sum;
  }
  if (lane < k) {
    L.ids[lane] = on ? taken : -1;
    L.w[lane] = on ? (float)(p * (double)s.scale) : 0.0f;
  }
  float* const lo = L.logits;
  if (lo)
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = lane + 64 * i;
      if (e < E) lo[e] = (float)L.z[e];
    }
}

}  // namespace

int64_t router_workspace(const RouterShape& s, int64_t max_tokens) {
  // The slices change only from one number of token tiles to the next, and
  // partial_floats() grows with M in between: its largest value is at a full
  // last tile (up to where one slice is left) or at the last M.
  const int64_t last = max_tokens < 1 ? 1 : max_tokens;
  int64_t most = partial_floats(s, last);
  for (int64_t M = 16; M < last && M <= 64 * 512; M = M < 64 ? 2 * M : M + 64) {
    const int64_t n = partial_floats(s, M);
    if (n > most) most = n;
  }
  return align256(4 * most);
}

hipError_t launch_router_prepare(const RouterShape& s, const void* weight, uint8_t* prepared, hipStream_t st) {
  const int64_t blocks = ((int64_t)s.subtiles() * s.kblocks() * 64 + 255) / 256;
  const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192));
  float* const norms = (float*)(prepared + s.norms_offset());
  if (s.planes == 3) {
    hipLaunchKernelGGL(router_prepare_kernel<true>, grid, dim3(256), 0, st, s, weight, prepared);
    hipLaunchKernelGGL(router_norms_kernel<true>, dim3(s.E), dim3(256), 0, st, s, weight, norms);
  } else {
    hipLaunchKernelGGL(router_prepare_kernel<false>, grid, dim3(256), 0, st, s, weight, prepared);
    hipLaunchKernelGGL(router_norms_kernel<false>, dim3(s.E), dim3(256), 0, st, s, weight, norms);
  }
  return hipGetLastError();
}

hipError_t launch_route(const RouterShape& s, const uint8_t* prepared, const uint16_t* x, int M, const float* bias,
                        int32_t* ids, float* w, float* logits, uint8_t* ws, hipStream_t st) {
  const LogitPlan p = logit_plan(s, M);
  float* const part = (float*)ws;
  float* const xx = part + (int64_t)p.splits * M * 16 * s.subtiles();
  const dim3 grid((unsigned)((M + 16 * p.tt - 1) / (16 * p.tt)), (unsigned)((s.E + 127) / 128), (unsigned)p.splits);
#define MOE_LOGITS(TT, NP) \
  hipLaunchKernelGGL((route_logits_kernel<TT, NP>), grid, dim3(256), 0, st, s, prepared, x, M, p.per, part, xx)
  if (s.planes == 3) {
    if (p.tt == 1) MOE_LOGITS(1, 3);
    else if (p.tt == 2) MOE_LOGITS(2, 3);
    else MOE_LOGITS(4, 3);
  } else {
    if (p.tt == 1) MOE_LOGITS(1, 1);
    else if (p.tt == 2) MOE_LOGITS(2, 1);
    else MOE_LOGITS(4, 1);
  }
#undef MOE_LOGITS
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 sgrid((unsigned)((M + 3) / 4));
  // Error bound of a logit, over ||x|| ||w||.  A matrix instruction adds 32
  // products to its accumulator C with an error of at most 2^-22 (|C| + the
  // sum of their magnitudes); a slice has `per` of them for each plane, C is
  // at most the magnitudes so far, and sum |x w| <= ||x|| ||w||.  The slices
  // are then added in fp32.
  const float coef = (float)((0.5 * p.per * s.planes + 1.0) * 0x1p-22 + p.splits * 0x1p-24);
#define MOE_SELECT_G(NI, G)                                                                                         \
  hipLaunchKernelGGL((route_select_kernel<NI, G>), sgrid, dim3(256), 0, st, s, prepared, x, M, p.splits, coef, part, \
                     xx, bias, ids, w, logits)
#define MOE_SELECT(NI)      \
  if (s.groups > 1)         \
    MOE_SELECT_G(NI, true); \
  else                      \
    MOE_SELECT_G(NI, false)
  if (s.E <= 64) {
    MOE_SELECT(1);
  } else if (s.E <= 128) {
    MOE_SELECT(2);
  } else if (s.E <= 256) {
    MOE_SELECT(4);
  } else {
    MOE_SELECT(8);
  }
#undef MOE_SELECT_G
#undef MOE_SELECT
  return hipGetLastError();
}

}  // namespace moe
