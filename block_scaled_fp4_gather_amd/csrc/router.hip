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
// Two launches: the logits (partial sums over slices of H, so that few tokens
// still fill the chip), route_few or route_gemm, and route_select (one wave per
// token); with a softmax and a bias a third, route_whole.
#include <hip/hip_runtime.h>

#include <type_traits>

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

// Rows as they are, and norms, rounded up.  Squares are summed in 64 bits: in
// 32 those of weights below 2^-63 vanish, and the bound that the norms stand
// in would be too small to see that logits are near each other.
template <bool F32>
__global__ void __launch_bounds__(256)
    router_rows_kernel(RouterShape s, const void* __restrict__ weight, uint8_t* __restrict__ prepared) {
  __shared__ double sums[4];
  const int e = blockIdx.x;
  float* const norms = (float*)(prepared + s.norms_offset());
  constexpr int kSize = F32 ? 4 : 2;
  const uint4* const from = (const uint4*)((const uint8_t*)weight + (int64_t)e * s.H * kSize);  // H % 8 == 0
  uint4* const to = (uint4*)(prepared + s.rows_offset() + (int64_t)e * s.H * kSize);
  for (int i = threadIdx.x; i < s.H * kSize / 16; i += 256) to[i] = from[i];
  double ss = 0.0;
  for (int h = threadIdx.x; h < s.H; h += 256) {
    const double v = F32 ? ((const float*)weight)[(int64_t)e * s.H + h]
                        : __uint_as_float((uint32_t)((const uint16_t*)weight)[(int64_t)e * s.H + h] << 16);
    ss += v * v;
  }
  for (int d = 32; d >= 1; d >>= 1) ss += __shfl_xor(ss, d);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = ss;
  __syncthreads();
  if (threadIdx.x == 0) norms[e] = (float)sqrt(sums[0] + sums[1] + sums[2] + sums[3]) * 1.001f + 0x1p-148f;
}

// ---- logits

// The matrix instruction's accumulator takes this many instructions before it
// is added to a second one and cleared: the roundings of a chain grow with its
// length and so does the bound on the logits' error, on which it hangs how
// many have to be recomputed.
constexpr int kChain = 8;

// How a call of M tokens is cut.
//   few tokens: 16 tt tokens x 16 experts per workgroup, H in `splits` slices
//     of `per` K blocks, a slice dealt to the workgroup's 4 waves;
//   many: BM x BE tiles (route_gemm), H in `splits` slices of `per` K blocks.
// Both with selection: H = 7168, E = 256, M = 160: 21.7 us few, 32.6 many,
// M = 256: 25.2 and 30.9, M = 512: 37.0 and 33.0; H = 4096, E = 128, M = 160:
// 16.6 and 15.0, M = 512: 19.5 and 15.9; H = 2560, fp32 E = 512, M = 512: 29.7
// and 24.8.
struct LogitPlan {
  bool gemm;
  int tt, bm, be, splits, per;
};

// K blocks (of 32) of a step of the tiled kernel
constexpr int gemm_step(int planes) { return planes == 1 ? 2 : 1; }
static_assert(RouterShape::kPadBlocks % kChain == 0, "the tiled kernel takes whole chains");

// Workgroups that one slice of the tiled kernel may leave idle are used by
// further ones, up to kMostSplits.
constexpr int64_t kMostSplits = 8;
int64_t gemm_workgroups(int be) { return be == 256 ? 256 : 512; }
int gemm_experts(const RouterShape& s) { return s.E <= 128 || s.planes == 3 ? 128 : 256; }
int gemm_tokens(const RouterShape& s) { return gemm_experts(s) == 256 || s.planes == 3 ? 128 : 64; }

LogitPlan logit_plan(const RouterShape& s, int64_t M) {
  LogitPlan p{};
  p.gemm = M > 256;
  const int kb = p.gemm ? s.kblocks() : s.blocks();
  int64_t splits;
  if (!p.gemm) {
    p.tt = M <= 16 ? 1 : M <= 32 ? 2 : 4;
    splits = (kb + 31) / 32;
  } else {
    p.be = gemm_experts(s);
    p.bm = gemm_tokens(s);
    const int64_t tiles = ((M + p.bm - 1) / p.bm) * ((s.E + p.be - 1) / p.be);
    splits = gemm_workgroups(p.be) / tiles;
    splits = splits < 1 ? 1 : splits > kMostSplits ? kMostSplits : splits;
  }
  const int unit = p.gemm ? kChain / s.planes : 4;  // whole chains; a block for each wave
  const int64_t units = (kb + unit - 1) / unit;
  if (splits > units) splits = units;
  p.per = (int)((units + splits - 1) / splits) * unit;
  p.splits = (kb + p.per - 1) / p.per;
  return p;
}

// Partial logits f32 [split][M][16 subtiles] and partial sums of x^2 f32
// [split][M].
int64_t partial_floats(const RouterShape& s, int64_t M) {
  const LogitPlan p = logit_plan(s, M);
  return p.splits * M * (16 * (int64_t)s.subtiles() + 1);
}

// x's squared norms come from the matrix cores too: a token tile times itself
// has them on its diagonal, which lane l holds in accumulator l % 4 if l / 16
// is l % 16 / 4.  (On the VALU a tile takes 48 instructions for one.)
__device__ __forceinline__ bool on_diagonal(int lane) { return (lane >> 4) == ((lane & 15) >> 2); }
__device__ __forceinline__ float diagonal(f32x4_t v, int lane) {
  const float a = lane & 1 ? v[1] : v[0], b = lane & 1 ? v[3] : v[2];
  return lane & 2 ? b : a;
}

// Few tokens: the weights are read once (per 64 tokens), straight into
// registers.  Four waves share a slice of H and join their sums in LDS.  M = 1,
// H = 7168, E = 256: 3.4 us, of which a launch that does nothing takes 2.
template <int TT, int NP>
__global__ void __launch_bounds__(256)
    route_few_kernel(RouterShape s, const uint8_t* __restrict__ prepared, const uint16_t* __restrict__ x, int M,
                     int per, float* __restrict__ part, float* __restrict__ xx) {
  __shared__ f32x4_t sums[4][TT][64];
  __shared__ f32x4_t squares[4][TT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int kb = s.blocks(), Ep = 16 * s.subtiles();
  const int sub = blockIdx.x;
  const int64_t split = blockIdx.y, tok0 = (int64_t)blockIdx.z * (16 * TT);
  const int b0 = (int)split * per + wave, b1 = min(kb, (int)(split + 1) * per);
  const bool norms = sub == 0;
  const int64_t plane = s.plane_bytes();
  const uint8_t* const w0 = prepared + (int64_t)sub * s.kblocks() * 1024 + lane * 16;
  f32x4_t acc[TT], chain[TT], sq[TT];
  const uint16_t* xr[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    acc[t] = chain[t] = sq[t] = f32x4_t{};
    xr[t] = x + min(tok0 + 16 * t + r, (int64_t)M - 1) * s.H + g * 8;
  }
  // the slice's blocks of this wave, kAhead at a time: all loads first
  constexpr int kAhead = TT == 4 || NP == 3 ? 2 : 4;
  static_assert(kAhead * NP <= kChain, "chain length");
  int in_chain = 0;
#pragma unroll 1
  for (int b = b0; b < b1; b += 4 * kAhead) {
    uint4 wv[kAhead][NP], xv[kAhead][TT];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int bi = b + 4 * i;
#pragma unroll
      for (int q = 0; q < NP; ++q) wv[i][q] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int t = 0; t < TT; ++t) xv[i][t] = make_uint4(0, 0, 0, 0);
      if (bi < b1) {
#pragma unroll
        for (int q = 0; q < NP; ++q) wv[i][q] = *(const uint4*)(w0 + q * plane + (int64_t)bi * 1024);
        if (bi * 32 + g * 8 < s.H)
#pragma unroll
          for (int t = 0; t < TT; ++t) xv[i][t] = *(const uint4*)(xr[t] + bi * 32);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const bf16x8_t bop = __builtin_bit_cast(bf16x8_t, xv[i][t]);
        if (norms) sq[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bop, bop, sq[t], 0, 0, 0);
#pragma unroll
        for (int q = 0; q < NP; ++q)
          chain[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, wv[i][q]), bop, chain[t], 0,
                                                             0, 0);
      }
    in_chain += kAhead * NP;
    if (in_chain + kAhead * NP > kChain) {
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        acc[t] += chain[t];
        chain[t] = f32x4_t{};
      }
      in_chain = 0;
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    sums[wave][t][lane] = acc[t] + chain[t];
    if (norms) squares[wave][t][lane] = sq[t];
  }
  __syncthreads();
  for (int t = wave; t < TT; t += 4) {
    const int64_t m = tok0 + 16 * t + r;
    if (m < M) {
      const f32x4_t v = (sums[0][t][lane] + sums[1][t][lane]) + (sums[2][t][lane] + sums[3][t][lane]);
      *(f32x4_t*)(part + (split * M + m) * Ep + sub * 16 + 4 * g) = v;
      if (norms && on_diagonal(lane))
        xx[split * M + m] = diagonal(
            (squares[0][t][lane] + squares[1][t][lane]) + (squares[2][t][lane] + squares[3][t][lane]), lane);
    }
  }
}

// Many tokens: BM tokens x BE experts per workgroup, so that x is read once
// for up to BE experts; x and the weights go to LDS by direct copies, two
// steps ahead in a ring of three slots, one barrier per step.  8 waves, each
// 16 FE experts x 16 TT tokens.
//
// M = 16384, H = 7168, E = 256: 71 us, 3.3 TB/s of x and 0.85 PFLOP/s; M = 4096,
// H = 4096, E = 128: 13.8 us.  A step's LDS reads, products and barrier bound it
// more than memory: a version of 85 us still took 70 without its copies.
//
// An x slot holds BM rows of 32 S values; the 16-byte chunk c of row r is at
// position c ^ row_swz(r).
template <int BM, int BE, int FE, int NP>
struct RouteGemm {
  static constexpr int S = gemm_step(NP);           // K blocks of 32 per step
  static constexpr int kWaves = 8;
  static constexpr int WE = BE / 16 / FE, WM = kWaves / WE;  // waves over experts and tokens
  static constexpr int TT = BM / 16 / WM;           // token tiles of a wave
  static constexpr int kRow = 64 * S;               // bytes of an x row in a slot
  static constexpr int kX = BM * kRow, kW = NP * S * (BE / 16) * 1024;
  static constexpr int kSlot = kX + kW;
  static constexpr int kXCopies = kX / 1024 / kWaves, kWCopies = kW / 1024 / kWaves;
  static constexpr int kCopies = kXCopies + kWCopies;
  static constexpr int kLds = 3 * kSlot;
  static_assert(kX % (1024 * kWaves) == 0 && kW % (1024 * kWaves) == 0 && TT >= 1, "whole copies per wave");
  static_assert(WE * FE * 16 == BE && WM * TT * 16 == BM && TT <= WE, "whole tiles; a wave's norms are of one tile");
};

template <int BM, int BE, int FE, int NP>
__global__ void __launch_bounds__(512)
    route_gemm_kernel(RouterShape s, const uint8_t* __restrict__ prepared, const uint16_t* __restrict__ x, int M,
                      int per, float* __restrict__ part, float* __restrict__ xx) {
  using G = RouteGemm<BM, BE, FE, NP>;
  constexpr int S = G::S, TT = G::TT, kChunks = G::kRow / 16;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int we = wave % G::WE, wm = wave / G::WE;
  const int kb = s.kblocks(), ns = s.subtiles(), Ep = 16 * ns;
  const int64_t split = blockIdx.z, tok0 = (int64_t)blockIdx.x * BM;
  const int b0 = (int)split * per, b1 = min(kb, b0 + per);
  const int nsteps = (b1 - b0) / S;  // whole chains
  const int xlast = (s.H - 1) / (32 * S) * S;
  const int sub0 = blockIdx.y * (BE / 16);

  // Copies of this wave, 1 KiB each: rows of x (past the last token it is
  // repeated), then [plane][subtile][block of the step] of the weights.
  const uint8_t* const xb = (const uint8_t*)(x + tok0 * s.H);
  uint32_t xoff[G::kXCopies];
  int xchunk[G::kXCopies];
#pragma unroll
  for (int c = 0; c < G::kXCopies; ++c) {
    const int row = (c * G::kWaves + wave) * (64 / kChunks) + lane / kChunks;
    xchunk[c] = ((lane % kChunks) ^ row_swz<G::kRow>(row)) * 16;
    xoff[c] = (uint32_t)min((int64_t)row, M - 1 - tok0) * (uint32_t)(2 * s.H);
  }
  const uint8_t* wsrc[G::kWCopies];
  int wblock[G::kWCopies];
#pragma unroll
  for (int c = 0; c < G::kWCopies; ++c) {
    const int kib = c * G::kWaves + wave;
    const int sub = kib / S % (BE / 16), q = kib / S / (BE / 16);
    wblock[c] = kib % S;
    wsrc[c] = prepared + q * s.plane_bytes() + (int64_t)min(sub0 + sub, ns - 1) * kb * 1024;
  }
  const uint32_t lds0 = lds_addr(smem) + wave * 1024;
  // Copy c of a step (the same number for every wave).  Past the last step it
  // repeats that and is not used; past the end of x's rows it repeats their
  // last values, for which the weights are zero.  (They count in the norm,
  // which then gives a bound on the high side.)
  auto copy = [&](int step, int ring, int c) {
    const int b = b0 + min(step, nsteps - 1) * S, bx = min(b, xlast);
    const uint32_t to = lds0 + ring * G::kSlot + c * 8192;
    if (c < G::kXCopies)
      dma16_at(xb + (int64_t)bx * 64, xoff[c] + (uint32_t)min(xchunk[c], 2 * (s.H - 8) - bx * 64), to);
    else
      dma16_at(wsrc[c - G::kXCopies] + (int64_t)(b + wblock[c - G::kXCopies]) * 1024, lane * 16, to);
  };

  f32x4_t acc[FE][TT], chain[FE][TT];
#pragma unroll
  for (int f = 0; f < FE; ++f)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[f][t] = chain[f][t] = f32x4_t{};
  f32x4_t sq{};
  // the waves of a row of tiles share its tokens' norms: this one's tile
  const int tn = min(we, TT - 1);
  const bool norms = blockIdx.y == 0 && we < TT;
  int xat[S], nat[S];  // rows 16 apart have the same swizzle
#pragma unroll
  for (int j = 0; j < S; ++j) {
    xat[j] = (wm * TT * 16 + r) * G::kRow + ((4 * j + g) ^ row_swz<G::kRow>(r)) * 16;
    nat[j] = xat[j] + tn * 16 * G::kRow;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int c = 0; c < G::kCopies; ++c) copy(i, i, c);
  constexpr int kFlush = kChain / (S * NP);  // steps of a chain
  static_assert(kFlush >= 1, "chain length");
  int ring = 0;
  auto run = [&](int step, auto starts) {  // starts: the step that begins a chain
    vm_wait<G::kCopies>();  // this wave's copies of the step have landed, those of the next may not have
    __syncthreads();        // everyone's have, and everyone is done with the step before
    const uint8_t* const slot = smem + ring * G::kSlot;
    const uint8_t* const wslot = slot + G::kX + we * FE * S * 1024 + lane * 16;
    const int last = ring == 0 ? 2 : ring - 1;  // slot of the step before
    ring = ring == 2 ? 0 : ring + 1;
    // operands of an instruction group are read a group ahead
    bf16x8_t xv[2][TT], nv[2], wv[2][FE];
    auto read_x = [&](int j) {
#pragma unroll
      for (int t = 0; t < TT; ++t) xv[j & 1][t] = *(const bf16x8_t*)(slot + xat[j] + t * 16 * G::kRow);
      nv[j & 1] = *(const bf16x8_t*)(slot + nat[j]);
    };
    auto read_w = [&](int i) {
      const int j = i / NP, q = i % NP;
#pragma unroll
      for (int f = 0; f < FE; ++f) wv[i & 1][f] = *(const bf16x8_t*)(wslot + ((q * (BE / 16) + f) * S + j) * 1024);
    };
    read_x(0);
    read_w(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < G::kCopies; ++c) copy(step + 2, last, c);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < S * NP; ++i) {
      const int j = i / NP;
      if (i % NP == 0 && j + 1 < S) read_x(j + 1);
      if (i + 1 < S * NP) read_w(i + 1);
      __builtin_amdgcn_sched_barrier(0);
      if (i % NP == 0) sq = __builtin_amdgcn_mfma_f32_16x16x32_bf16(nv[j & 1], nv[j & 1], sq, 0, 0, 0);
#pragma unroll
      for (int f = 0; f < FE; ++f)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          if (decltype(starts)::value && i == 0) {
            acc[f][t] += chain[f][t];
            chain[f][t] = f32x4_t{};
          }
          chain[f][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[i & 1][f], xv[j & 1][t], chain[f][t], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
    }
  };
#pragma unroll 1
  for (int step = 0; step < nsteps; step += kFlush) {
    run(step, std::true_type{});
#pragma unroll
    for (int u = 1; u < kFlush; ++u) run(step + u, std::false_type{});
  }
  vm_wait<0>();  // no copy may land after the workgroup's LDS is released
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int64_t m = tok0 + (wm * TT + t) * 16 + r;
    if (m < M)
#pragma unroll
      for (int f = 0; f < FE; ++f) {
        const int sub = sub0 + we * FE + f;
        if (sub < ns) *(f32x4_t*)(part + (split * M + m) * Ep + sub * 16 + 4 * g) = acc[f][t] + chain[f][t];
      }
  }
  const int64_t m = tok0 + (wm * TT + tn) * 16 + r;
  if (norms && m < M && on_diagonal(lane)) xx[split * M + m] = diagonal(sq, lane);
}

// ---- selection: one wave per token, a workgroup of its own (in workgroups of
// four, tokens with something to recompute keep the places of those without:
// M = 16384, E = 256 in groups took 67 us for 59); lane l holds experts
// NI l .. NI l + NI - 1.  Bound by the chain of dependent steps: M = 1 takes
// 8 us, and 5 waves a SIMD hide it in part for many tokens (4: 75 us for 66).
// About 15 of the 59 us go into recomputed logits.

// What every lane has alike, told to the compiler: branches on it need no
// masks.
__device__ __forceinline__ float uniform(float v) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

template <class T>
__device__ __forceinline__ const T* uniform(const T* p) {
  const uint64_t u = (uint64_t)p;
  return (const T*)((uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(u >> 32)) << 32 |
                    (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)u));
}

// v of the lane that CTRL's move names, 0 bits where there is none
template <int CTRL>
__device__ __forceinline__ double moved(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum over the wave, in lane order moves as below.
__device__ __forceinline__ double wave_sum(double v) {
  v += moved<0x111>(v);
  v += moved<0x112>(v);
  v += moved<0x114>(v);
  v += moved<0x118>(v);
  v += moved<0x142>(v);
  v += moved<0x143>(v);
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
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

// Largest key of the wave (each lane's NI) and its lowest expert: that of the
// lowest lane, which holds the lowest experts.
template <int NI>
__device__ __forceinline__ uint32_t wave_best_key(const uint32_t (&key)[NI], int& e) {
  uint32_t v = key[0];
  int at = 0;
#pragma unroll
  for (int i = 1; i < NI; ++i)
    if (key[i] > v) {
      v = key[i];
      at = i;
    }
  const uint32_t best = wave_max_u32(v);
  const int l = __ffsll((unsigned long long)__ballot(v == best)) - 1;
  e = l * NI + __builtin_amdgcn_readlane(at, l);
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

// exp(v) within (|v| + 2) 2^-23 of itself, 0 where that is below the normal
// numbers: two instructions, where scores only need to be compared.
__device__ __forceinline__ float fast_exp(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504f); }

// The same value, unknown to the compiler: what it derived from v before (a
// mask register per comparison) is not kept for later uses.
__device__ __forceinline__ int renew(int v) {
  asm volatile("" : "+v"(v));
  return v;
}
__device__ __forceinline__ RouterShape renew(RouterShape s) {
  asm volatile("" : "+s"(s.E), "+s"(s.k), "+s"(s.groups), "+s"(s.top_groups));
  int sigmoid = s.sigmoid, renorm = s.renorm;
  asm volatile("" : "+s"(sigmoid), "+s"(renorm));
  s.sigmoid = sigmoid;
  s.renorm = renorm;
  return s;
}

// Logits of experts e[0] and e[1] in 64 bits, in which products of a bf16 and
// an fp32 value are exact, from the weights' rows.  A lane takes every 64th
// chunk of 8 values; the operands of kAhead of them are loaded before they are
// used.  (From the operand layout, where 16 bytes of an expert are followed by
// 240 of others', M = 37 with fp32 weights
// took 21 us for 18.)
template <bool F32, int kAhead>
__device__ __forceinline__ void exact_logits(int H, const uint8_t* __restrict__ rows, const uint16_t* __restrict__ xr,
                                             const int (&e)[2], int lane, double (&sum)[2]) {
  constexpr int kW = F32 ? 2 : 1;  // 16-byte pieces of a chunk of weights
  const int chunks = H / 8;
  const uint4* row[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    row[p] = (const uint4*)rows + (int64_t)e[p] * (chunks * kW);
    sum[p] = 0.0;
  }
#pragma unroll 1
  for (int c0 = lane; c0 < chunks; c0 += 64 * kAhead) {
    uint4 xv[kAhead], wv[kAhead][2][kW];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int c = c0 + 64 * i;
      xv[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int h = 0; h < kW; ++h) wv[i][p][h] = make_uint4(0, 0, 0, 0);
      if (c < chunks) {
        xv[i] = *(const uint4*)(xr + c * 8);
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int h = 0; h < kW; ++h) wv[i][p][h] = row[p][c * kW + h];
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const uint32_t xw[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double xd = (double)__uint_as_float(j % 2 ? xw[j / 2] & 0xFFFF0000u : xw[j / 2] << 16);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint4 v = wv[i][p][F32 ? j / 4 : 0];
          const uint32_t ww[4] = {v.x, v.y, v.z, v.w};
          const uint32_t w = F32 ? ww[j % 4] : j % 2 ? ww[j / 2] & 0xFFFF0000u : ww[j / 2] << 16;
          sum[p] = fma(xd, (double)__uint_as_float(w), sum[p]);
        }
        if (j % 2) __builtin_amdgcn_sched_barrier(0);  // few conversions at a time: registers
      }
    }
  }
  sum[0] = wave_sum(sum[0]);
  sum[1] = wave_sum(sum[1]);
}

constexpr double kNone = -__builtin_inf();
constexpr int kNobody = 1 << 30;
constexpr int kLater = -2;  // in place of a token's first expert: left to route_whole_kernel

// What a wave of the selection keeps in LDS.
template <int NI>
struct SelectLds {
  double z[64 * NI];     // the token's logits, in 64 bits where recomputed
  double t[64 * NI];     // scores in 64 bits of what was recomputed (by expert, then by list place)
  uint16_t e[64 * NI];   // list: experts, best first
  uint16_t run[64 * NI]; // list: first place of the run of unsure neighbours a place belongs to
  int taken[64];
  // where the token's row and the results are: kept here while the experts are
  // chosen, which needs all the scalar registers
  const uint16_t* x;
  const uint8_t* rows;  // of the weights
  const float* bias;
  int H, size;
  float scale;
  int* ids;
  float *w, *logits;
};

// Recomputes the logits of experts first, first + 1, first + step, ..
template <int NI, bool F32>
__device__ __forceinline__ void all_logits(SelectLds<NI>& L, int E, int first, int step, int lane) {
  const int H = __builtin_amdgcn_readfirstlane(L.H);
#pragma unroll 1
  for (int e0 = first; e0 < E; e0 += step) {
    lane = renew(lane);
    const int e[2] = {e0, min(e0 + 1, E - 1)};
    double v[2];
    exact_logits<F32, F32 ? 1 : 2>(H, uniform(L.rows), uniform(L.x), e, lane, v);
    if (lane < 2) L.z[lane == 0 ? e[0] : e[1]] = lane == 0 ? v[0] : v[1];
  }
}

// Recomputes logits, two at a time: those of the first n places of the list
// that are in runs of more than one, or with n = 0 those of the experts in
// `want` (bit i: this lane's i-th).
template <int NI, bool F32>
__device__ __forceinline__ void refine(SelectLds<NI>& L, uint32_t want, int n, int lane) {
  const int H = __builtin_amdgcn_readfirstlane(L.H);
#pragma unroll 1
  for (int i = 0; i < (n != 0 ? (n + 63) / 64 : NI); ++i) {
    int expert = lane * NI + i;
    bool in = want >> (i & 31) & 1u;
    if (n != 0) {
      const int j = i * 64 + lane;
      in = false;
      if (j < n) {
        const int r = L.run[j];
        expert = L.e[j];
        in = r != j || (j + 1 < n && L.run[j + 1] == r);
      }
    }
    uint64_t todo = __ballot(in);
#pragma unroll 1
    while (todo) {
      int e[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if (p == 1 && todo == 0) {
          e[1] = e[0];
        } else {
          e[p] = __builtin_amdgcn_readlane(expert, __ffsll((unsigned long long)todo) - 1);
          todo &= todo - 1;
        }
      }
      double v[2];
      exact_logits<F32, F32 ? 1 : 2>(H, uniform(L.rows), uniform(L.x), e, lane, v);
      if (lane < 2) L.z[lane == 0 ? e[0] : e[1]] = lane == 0 ? v[0] : v[1];
    }
  }
  wave_sync();
}

// Sum of the two largest of L.t in group q, and the second of them; -inf
// where fewer than two may be taken.
template <int NI>
__device__ __forceinline__ double group_top2(const SelectLds<NI>& L, int q, int size, double& second) {
  double v1 = kNone, v2 = kNone;
#pragma unroll 1
  for (int c = 0; c < size; ++c) {
    const double v = L.t[q * size + c];
    v2 = fmax(v2, fmin(v1, v));
    v1 = fmax(v1, v);
  }
  second = v2;
  return v2 > kNone ? v1 + v2 : kNone;
}

// Largest bound on the logits for which scores of a softmax are bounded by it
// (as below); past it all logits of the token are recomputed.  Hidden states
// and weights of ordinary size stay below 0.01.
constexpr float kScoreBound = 0.25f;

// Which experts a token takes, best first, into L.taken; returns how many, or
// -1 where all logits have to be recomputed for a softmax with a bias.
//
// Scores are first compared in 32 bits with a common bound on their errors.
// Groups: if the border between the groups taken and left is unsure, the
// logits of all that could be among a group's two largest are recomputed and
// the groups compared in 64 bits.  Experts: the list of the largest scores is
// cut into runs of neighbours nearer than twice the bound, as far as the run
// that holds the k-th; the order of runs is certain, and within a run it is
// that of the recomputed scores.
template <int NI, bool GROUPS, bool F32>
__device__ __forceinline__ int select_experts(const RouterShape& s, SelectLds<NI>& L, const float (&z)[NI],
                                              float bound, const float* __restrict__ bias,
                                              const float (&biases)[NI], int size, int per_group, int lane) {
  const int E = s.E;
  const bool scored = bias != nullptr || GROUPS;
  bound = uniform(bound);
  float t[NI];
  float err = bound, zmax = 0.0f;
  if (scored) {
    if (s.sigmoid) {
#pragma unroll
      for (int i = 0; i < NI; ++i) t[i] = __builtin_amdgcn_rcpf(1.0f + fast_exp(-z[i]));
      // a score p <= 1 is within |z| 2^-23 (1 - p) p, at most 2^-25, and a few roundings of 2^-24 of itself
      err = 0.25f * bound + 0x1p-20f;
    } else {
      uint32_t key = 0;
#pragma unroll
      for (int i = 0; i < NI; ++i) key = max(key, z[i] == z[i] ? order_key(z[i]) : 0u);
      zmax = key_value(wave_max_u32(key));
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        t[i] = fast_exp(z[i] - zmax);
        sum += t[i];
      }
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
      const float top = uniform(1.0f / sum);  // the largest score
#pragma unroll
      for (int i = 0; i < NI; ++i) t[i] *= top;
      // exp(z - zmax) / sum, each part within a factor of e^bound: off by at most
      // e^(2 bound) - 1 <= 2 bound (1 + 1.2 bound) of itself for bounds up to
      // kScoreBound.  The terms e of the sum are off by 3 |log e| 2^-24, by
      // log E on the mean, and the sum by at most 14 roundings.
      err = (2.0f * bound * (1.0f + 1.2f * bound) + 0x1p-18f) * top;
    }
    if (bias) {
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const float b = biases[i];
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
  uint32_t key[NI], zk[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const bool in = lane * NI + i < E;
    key[i] = in && t[i] > -__builtin_inff() ? order_key(t[i]) : 0u;  // not NaN
    zk[i] = order_key(z[i]);
  }
  // With a bias on a softmax a recomputed score still carries the other
  // logits' errors, through the sum, which is off by up to `bound` of itself:
  // scores p + b whose difference is within that of the difference of their p
  // need all logits recomputed.  (Without a bias the sum is a common factor.
  // With all recomputed wherever two scores are unsure, M = 13712 tokens,
  // H = 416, E = 444 took 928 us for 149.)
  const bool whole = bias != nullptr && !s.sigmoid;
  // Passes: each recomputes what the one before found missing (the groups'
  // largest; the unsure runs') and decides anew.
  uint32_t want = 0u;
  bool have_groups = false, have_runs = false;
  const int lanes_per_group = GROUPS && size % NI == 0 && ((size / NI) & (size / NI - 1)) == 0 ? size / NI : 0;
  int group[NI];  // n / size = n * (2^20 / size, rounded up) / 2^20 for n < 512: n (size - 1) < 2^20
#pragma unroll
  for (int i = 0; i < NI; ++i) group[i] = GROUPS ? renew(__umul24(lane * NI + i, per_group) >> 20 & 63) : 0;
  int n = 0;
  bool listed = false, runs = false;  // the list stands; it has unsure neighbours

#pragma unroll 1
  while (true) {
    lane = renew(lane);
#pragma unroll
    for (int i = 0; i < NI; ++i) {  // nothing derived from these is worth a register from pass to pass
      key[i] = (uint32_t)renew((int)key[i]);
      group[i] = renew(group[i]);
      zk[i] = (uint32_t)renew((int)zk[i]);
    }
    if (bound != 0.0f) refine<NI, F32>(L, want, listed ? n : 0, lane);  // logits of a zero row are exact
    want = 0u;
    double total = 1.0;
    if (whole && listed) {
      double sum = 0.0;
#pragma unroll 1
      for (int e = lane; e < E; e += 64) sum += exp(L.z[e] - (double)zmax);
      total = wave_sum(sum);
    }
    // score in 64 bits; what may not be taken gets -infinity
    auto exact_score = [&](int e, bool for_groups) {
      double v = L.z[e];
      if (bias || for_groups) {
        v = exp(s.sigmoid ? -v : v - (double)zmax);
        v = s.sigmoid ? 1.0 / (1.0 + v) : v / total;
        if (bias) v += (double)L.bias[e];
      }
      return v == v ? v : kNone;
    };

    uint64_t in_groups = ~0ull;
    if (GROUPS && !listed) {
      float score = -__builtin_inff();  // lane q: that of group q
      uint32_t near = 0;                // could be among the two largest of their groups
      if (lanes_per_group > 0) {        // groups of whole lanes, a power of two of them: all groups at once
        uint32_t k1 = 0u, k2 = 0u;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          k2 = max(k2, min(k1, key[i]));
          k1 = max(k1, key[i]);
        }
#pragma unroll 1
        for (int d = 1; d < lanes_per_group; d <<= 1) {
          const uint32_t o1 = (uint32_t)__shfl_xor((int)k1, d), o2 = (uint32_t)__shfl_xor((int)k2, d);
          k2 = max(max(k2, o2), min(k1, o1));
          k1 = max(k1, o1);
        }
        const float own = k2 != 0u ? key_value(k1) + key_value(k2) : -__builtin_inff();
        score = __shfl(own, lane * lanes_per_group & 63);
        const float floor = k2 != 0u ? key_value(k2) - 2.0f * err : -__builtin_inff();
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (key[i] != 0u && !(key_value(key[i]) < floor)) near |= 1u << i;
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) L.t[lane * NI + i] = key[i] != 0u ? (double)key_value(key[i]) : kNone;
        wave_sync();
        double second;
        const double both = group_top2<NI>(L, lane < s.groups ? lane : 0, size, second);
        if (lane < s.groups) score = (float)both;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const float floor = (float)__shfl(second, group[i]) - 2.0f * err;
          if (key[i] != 0u && !(key_value(key[i]) < floor)) near |= 1u << i;
        }
        wave_sync();
      }
      uint32_t gk[1] = {lane < s.groups ? (score == score ? order_key(score) : 1u) : 0u};
      float last = 0.0f, next = -__builtin_inff();
      in_groups = 0;
#pragma unroll 1
      for (int q = 0; q <= s.top_groups && q < s.groups; ++q) {
        int e;
        const float v = key_value(wave_best_key<1>(gk, e));
        if (q == s.top_groups) {
          next = v;
          break;
        }
        last = v;
        in_groups |= 1ull << e;
        if (lane == e) gk[0] = 0u;
      }
      // two sums of two scores, and the sums' own roundings
      const float apart = 4.0f * err + 0x1p-22f * (fabsf(last) + fabsf(next));
      if (s.top_groups < s.groups && !(last - next > apart)) {
        // groups that are surely taken or surely left need no exact score
        const bool in = score - next > apart, out = last - score > apart;
        const uint64_t clear = __ballot(in || out);
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (clear >> group[i] & 1ull) near &= ~(1u << i);
        if (!have_groups) {
          if (whole) return -1;
          have_groups = true;
          want = near;
          continue;
        }
#pragma unroll 1
        for (int i = 0; i < NI; ++i)
          L.t[lane * NI + i] = near >> i & 1u ? exact_score(lane * NI + i, true) : kNone;
        wave_sync();
        double gs = in ? -kNone : kNone;
        double second;
        if (lane < s.groups && !in && !out) gs = group_top2<NI>(L, lane, size, second);
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
    if (!listed) {
      uint32_t left[NI], may = 0;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (!GROUPS || (in_groups >> group[i] & 1ull)) may |= 1u << i;
        left[i] = may >> i & 1u ? key[i] : 0u;
        if (!bias && left[i] != 0u) left[i] = zk[i];
      }
      n = 0;
      runs = false;
      const float apart = 2.0f * (bias ? err : bound);
      float prev = 0.0f;
      int start = 0;
#pragma unroll 1
      while (true) {
        lane = renew(lane);
        int e;
        const uint32_t best = wave_best_key<NI>(left, e);
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
          if (lane * NI + i == e) left[i] = 0u;
        prev = v;
        ++n;
      }
      wave_sync();
    }

    if (!runs) {
      if (lane < n) L.taken[lane] = L.e[lane];
    } else {
      if (!have_runs) {
        have_runs = true;
        listed = true;
        continue;
      }
#pragma unroll 1
      for (int j = lane; j < n; j += 64) L.t[j] = exact_score(L.e[j], false);
      wave_sync();
      // e^bound - 1 at most, for bounds up to 0.01 and up to kScoreBound
      const double off = whole ? (bound < 0.01f ? 1.01 * bound : 1.0) : 0.0;
      bool unsure = false;
#pragma unroll 1
      for (int j = lane; j < n; j += 64) {
        const int r = L.run[j], e = L.e[j];
        const double v = L.t[j];
        int at = r;
        for (int i = r; i < n && L.run[i] == r; ++i) {
          at += L.t[i] > v || (L.t[i] == v && L.e[i] < e);
          if (off != 0.0 && i != j && fabs(v) < -kNone) {
            const double d = L.t[i] - v, dp = d - ((double)L.bias[L.e[i]] - (double)L.bias[e]);
            unsure |= dp != 0.0 && !(fabs(d) > off * fabs(dp));
          }
        }
        if (at < s.k) L.taken[at] = e;
      }
      if (__ballot(unsure) != 0ull) return -1;
    }
    wave_sync();
    return n < s.k ? n : s.k;
  }
}

// The same from logits that are all exact, scores in 64 bits throughout; always
// returns how many.
template <int NI>
__device__ __forceinline__ int select_all(const RouterShape& shape, SelectLds<NI>& L, const float* __restrict__ bias,
                                          int size, int lane) {
  const RouterShape s = renew(shape);
  const int E = s.E;
  double zmax = 0.0, total = 1.0;
  if (!s.sigmoid) {
    double mx = kNone, sum = 0.0;
#pragma unroll 1
    for (int e = lane; e < E; e += 64) mx = fmax(mx, L.z[e]);
    zmax = wave_max(mx);
#pragma unroll 1
    for (int e = lane; e < E; e += 64) sum += exp(L.z[e] - zmax);
    total = wave_sum(sum);
    if (total != total) return 0;  // a NaN or +infinity among the logits: no probabilities
  }
  auto scores = [&](bool logits) {  // -infinity for what may not be taken
#pragma unroll 1
    for (int e = lane; e < E; e += 64) {
      double v = L.z[e];
      if (!logits) {
        v = exp(s.sigmoid ? -v : v - zmax);
        v = s.sigmoid ? 1.0 / (1.0 + v) : v / total;
        if (bias) v += (double)bias[e];
      }
      L.t[e] = v == v ? v : kNone;
    }
    wave_sync();
  };
  uint64_t in_groups = ~0ull;
  if (s.groups > 1) {
    scores(false);
    lane = renew(lane);
    double second;
    const double gs = group_top2<NI>(L, lane < s.groups ? lane : 0, size, second);
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
  if (s.groups == 1 || !bias) scores(!bias);  // without a bias the order is that of the logits
  int n = 0;
#pragma unroll 1
  for (; n < s.k; ++n) {
    lane = renew(lane);
    double v = kNone;
    int best = kNobody;
#pragma unroll 1
    for (int e = lane; e < E; e += 64) {
      const double c = L.t[e];
      if (c > v && (s.groups == 1 || (in_groups >> (e / size) & 1ull))) {
        v = c;
        best = e;
      }
    }
    wave_best(v, best);
    if (!(v > kNone)) break;
    if (lane == 0) {
      L.taken[n] = best;
      L.t[best] = kNone;
    }
    wave_sync();
  }
  return n;
}

// The taken experts' probabilities, from their logits, and the outputs.
template <int NI>
__device__ __forceinline__ void finish(const RouterShape& shape, SelectLds<NI>& L, int kept, int lane) {
  const RouterShape s = renew(shape);
  const int E = s.E, k = s.k;
  const bool on = lane < kept;
  const int taken = on ? L.taken[lane] : 0;
  const double zw = L.z[taken];
  // the largest logit of those taken, from a finite one on: weights of -infinity
  // leave logits of -infinity, which a bias may have taken, with p = 0
  const double mx = s.sigmoid || kept == 0 ? 0.0 : fmax(wave_max(on ? zw : kNone), -0x1p1000);
  double p = exp(s.sigmoid ? -zw : zw - mx);
  if (s.sigmoid) {
    p = on ? 1.0 / (1.0 + p) : 0.0;
  } else {
    p = on ? p : 0.0;
    if (!s.renorm) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (lane * NI + i < E) sum += expf((float)(L.z[lane * NI + i] - mx));
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
    L.w[lane] = on ? (float)(p * (double)L.scale) : 0.0f;
  }
  float* const lo = L.logits;
  if (lo)
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = lane * NI + i;
      if (e < E) lo[e] = (float)L.z[e];
    }
}

template <int NI, bool GROUPS, bool F32>
__global__ void __launch_bounds__(64, NI <= 4 ? 5 : 4)
    route_select_kernel(RouterShape s, const uint8_t* __restrict__ prepared, const uint16_t* __restrict__ x, int M,
                        int splits, float coef, float root, int size, int per_group, const float* __restrict__ part,
                        const float* __restrict__ xx, const float* __restrict__ bias, int* __restrict__ ids,
                        float* __restrict__ wout, float* __restrict__ logits) {
  __shared__ SelectLds<NI> L;
  int lane = threadIdx.x;
  const int64_t m = blockIdx.x;
  const int E = s.E, Ep = 16 * s.subtiles(), k = s.k;
  const float* const norms = (const float*)(prepared + s.norms_offset());

  // all that is needed from memory, in flight together
  typedef float vec_t __attribute__((ext_vector_type(NI)));
  float wnorm[NI], biases[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    wnorm[i] = norms[min(lane * NI + i, E - 1)];
    biases[i] = 0.0f;
  }
  if (bias)
#pragma unroll
    for (int i = 0; i < NI; ++i) biases[i] = bias[min(lane * NI + i, E - 1)];
  float x2 = 0.0f;
  vec_t zv = {};
  // a lane's experts are all below Ep, a multiple of 16, or none is
  const float* p0 = part + m * Ep + min(lane * NI, Ep - NI);
#pragma unroll 8
  for (int q = 0; q < splits; ++q) {
    x2 += xx[(int64_t)q * M + m];
    zv += *(const vec_t*)(p0 + (int64_t)q * M * Ep);
  }
  uint32_t wn = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) wn = max(wn, __float_as_uint(wnorm[i]));  // norms are not negative
  float z[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    z[i] = lane * NI + i < E ? zv[i] : -__builtin_inff();
    L.z[lane * NI + i] = (double)z[i];
  }
  if (lane == 0) {
    L.x = x + m * s.H;
    L.rows = prepared + s.rows_offset();
    L.bias = bias;
    L.H = s.H;
    L.size = size;
    L.scale = s.scale;
    L.ids = ids + m * k;
    L.w = wout + m * k;
    L.logits = logits ? logits + m * E : nullptr;
  }
  wave_sync();
  // ||x|| ||w|| times the coefficient of the plan, which counts the roundings
  float xnorm = sqrtf(x2);
  if (x2 < 0x1p-60f) {  // squares may have vanished: sqrt(H) times the largest value instead, and 0 for a row of zeros
    uint32_t most = 0;
    for (int c = lane * 2; c < s.H; c += 128) {
      const uint32_t v = *(const uint32_t*)(x + m * s.H + c);
      most = max(most, max(v << 16 & 0x7FFFFFFFu, v & 0x7FFF0000u));
    }
    xnorm = __uint_as_float(wave_max_u32(most)) * root;
  }
  const float most = __uint_as_float(wave_max_u32(wn));
  float bound = xnorm * 1.001f * most * coef;
  // What numbers below the normal ones lose, at most 2^-126 each: three
  // products of a value of x and the terms of a weight, a value of x, the terms
  // of a weight; root = sqrt(H), and a row's magnitudes add up to root ||.||.
  if (xnorm != 0.0f) bound += 0x1p-124f * root * (root + xnorm + most);
  if (x2 != x2) bound = 0.0f;  // a NaN in x makes every logit NaN: nothing to recompute
  int kept = -1;
  const bool shares = !s.sigmoid && (GROUPS || bias != nullptr);  // scores of a softmax are compared
  if (bound < (shares ? kScoreBound : __builtin_inff())) {
    kept = select_experts<NI, GROUPS, F32>(s, L, z, bound, bias, biases, size, per_group, lane);
  } else if (bias == nullptr || s.sigmoid) {  // no bound that serves: all logits
    all_logits<NI, F32>(L, E, 0, 2, renew(lane));
    wave_sync();
    kept = select_all<NI>(s, L, uniform(L.bias), __builtin_amdgcn_readfirstlane(L.size), renew(lane));
  }
  lane = renew(lane);
  if (kept < 0) {
    if (lane == 0) L.ids[0] = kLater;
    return;
  }
  finish<NI>(s, L, kept, lane);
}

// Tokens of a softmax with a bias left by the selection: all logits in 64
// bits, a workgroup to a token and pairs of experts dealt to its 8 waves.
// (By the one wave of the selection they held up a call of M = 13712 tokens,
// H = 416, E = 444 for 773 us; now it takes 149.)
template <bool F32>
__global__ void __launch_bounds__(512)
    route_whole_kernel(RouterShape s, const uint8_t* __restrict__ prepared, const uint16_t* __restrict__ x, int M,
                       int size, const float* __restrict__ bias, int* ids, float* __restrict__ wout,
                       float* __restrict__ logits) {
  constexpr int NI = kRouterMaxExperts / 64;
  __shared__ SelectLds<NI> L;
  int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll 1
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    lane = renew(lane);
    if (ids[m * s.k] != kLater) continue;  // the same for all: it is written behind the barrier
    if (threadIdx.x == 0) {
      L.x = x + m * s.H;
      L.rows = prepared + s.rows_offset();
      L.H = s.H;
    }
    __syncthreads();
    all_logits<NI, F32>(L, s.E, 2 * wave, 16, lane);
    __syncthreads();
    if (wave == 0) {
      if (lane == 0) {
        L.scale = s.scale;
        L.ids = ids + m * s.k;
        L.w = wout + m * s.k;
        L.logits = logits ? logits + m * s.E : nullptr;
      }
      wave_sync();
      const int kept = select_all<NI>(s, L, bias, size, renew(lane));
      finish<NI>(s, L, kept, renew(lane));
    }
    __syncthreads();
  }
}

}  // namespace

int64_t router_workspace(const RouterShape& s, int64_t max_tokens) {
  // partial_floats() grows with M while the slices stay as many, so its
  // largest value is at the largest M of some number of slices: that of the
  // few tokens' kernel, or of the token tiles that leave room for n slices, or
  // the last M.  (Called for each call: not in a loop over M.)
  const int64_t last = max_tokens < 1 ? 1 : max_tokens;
  int64_t most = partial_floats(s, last);
  auto take = [&](int64_t M) {
    const int64_t n = M < last ? partial_floats(s, M) : 0;
    if (n > most) most = n;
  };
  take(256);
  const int be = gemm_experts(s);
  const int64_t tiles = gemm_workgroups(be) / ((s.E + be - 1) / be);
  for (int n = 1; n <= kMostSplits; ++n) take(tiles / n * gemm_tokens(s));
  return align256(4 * most);
}

hipError_t launch_router_prepare(const RouterShape& s, const void* weight, uint8_t* prepared, hipStream_t st) {
  const int64_t blocks = ((int64_t)s.subtiles() * s.kblocks() * 64 + 255) / 256;
  const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192));
  if (s.planes == 3) {
    hipLaunchKernelGGL(router_prepare_kernel<true>, grid, dim3(256), 0, st, s, weight, prepared);
    hipLaunchKernelGGL(router_rows_kernel<true>, dim3(s.E), dim3(256), 0, st, s, weight, prepared);
  } else {
    hipLaunchKernelGGL(router_prepare_kernel<false>, grid, dim3(256), 0, st, s, weight, prepared);
    hipLaunchKernelGGL(router_rows_kernel<false>, dim3(s.E), dim3(256), 0, st, s, weight, prepared);
  }
  return hipGetLastError();
}

hipError_t launch_route(const RouterShape& s, const uint8_t* prepared, const uint16_t* x, int M, const float* bias,
                        int32_t* ids, float* w, float* logits, uint8_t* ws, hipStream_t st) {
  const LogitPlan p = logit_plan(s, M);
  float* const part = (float*)ws;
  float* const xx = part + (int64_t)p.splits * M * 16 * s.subtiles();
  if (p.gemm) {
    const dim3 grid((unsigned)((M + p.bm - 1) / p.bm), (unsigned)((s.E + p.be - 1) / p.be), (unsigned)p.splits);
    if (s.planes == 3)
      hipLaunchKernelGGL((route_gemm_kernel<128, 128, 4, 3>), grid, dim3(512), (RouteGemm<128, 128, 4, 3>::kLds), st, s,
                         prepared, x, M, p.per, part, xx);
    else if (p.be == 256)
      hipLaunchKernelGGL((route_gemm_kernel<128, 256, 4, 1>), grid, dim3(512), (RouteGemm<128, 256, 4, 1>::kLds), st, s,
                         prepared, x, M, p.per, part, xx);
    else
      hipLaunchKernelGGL((route_gemm_kernel<64, 128, 2, 1>), grid, dim3(512), (RouteGemm<64, 128, 2, 1>::kLds), st, s,
                         prepared, x, M, p.per, part, xx);
  } else {
    const dim3 grid((unsigned)s.subtiles(), (unsigned)p.splits, (unsigned)((M + 16 * p.tt - 1) / (16 * p.tt)));
#define MOE_LOGITS(TT, NP) \
  hipLaunchKernelGGL((route_few_kernel<TT, NP>), grid, dim3(256), 0, st, s, prepared, x, M, p.per, part, xx)
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
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 sgrid((unsigned)M);
  // Error bound of a logit, over ||x|| ||w||, which is at least the sum A of
  // the magnitudes |x w|.  v_mfma_f32_16x16x32_bf16 adds its 32 products in
  // four groups of 8 (measured): within a group they are cut to multiples of
  // 2^-24 of the largest's power of two (at most 7 * 2^-24 of the group's
  // magnitudes), and each group's sum is added to the accumulator C, at most
  // the magnitudes of its chain of kChain instructions, with one rounding.
  // The chains, the waves' sums and the slices are added in fp32.
  const float coef = (float)((4.0 * kChain + 8.0 + (p.per * s.planes / (kChain / 2) + 4.0) + p.splits) * 0x1p-24);
  const float root = sqrtf((float)s.H);
  const int size = s.E / s.groups, per_group = ((1 << 20) + size - 1) / size;
#define MOE_SELECT_G(NI, G, F32)                                                                                  \
  hipLaunchKernelGGL((route_select_kernel<NI, G, F32>), sgrid, dim3(64), 0, st, s, prepared, x, M, p.splits, coef, \
                     root, size, per_group, part, xx, bias, ids, w, logits)
#define MOE_SELECT(NI)                                                 \
  if (s.groups > 1 && s.planes == 3) MOE_SELECT_G(NI, true, true);     \
  else if (s.groups > 1) MOE_SELECT_G(NI, true, false);                \
  else if (s.planes == 3) MOE_SELECT_G(NI, false, true);               \
  else MOE_SELECT_G(NI, false, false)
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
  if (bias == nullptr || s.sigmoid) return hipGetLastError();
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 wgrid((unsigned)(M < 2048 ? M : 2048));
  if (s.planes == 3)
    hipLaunchKernelGGL(route_whole_kernel<true>, wgrid, dim3(512), 0, st, s, prepared, x, M, size, bias, ids, w,
                       logits);
  else
    hipLaunchKernelGGL(route_whole_kernel<false>, wgrid, dim3(512), 0, st, s, prepared, x, M, size, bias, ids, w,
                       logits);
  return hipGetLastError();
}

}  // namespace moe
