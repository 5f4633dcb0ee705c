// Linear map with MXFP4 weights and MXFP4 activations:
//   y[m][n] = sum over blocks b of 32:  sw[n][b] sx[m][b] sum_{k in b} c[n][k] q[m][k]
// with E2M1 codes c and q and UE8M0 scales, on v_mfma_scale_f32_*_f8f6f4, which
// takes codes and scales as they are stored: both operands E2M1, at twice the
// rate of its FP8 forms.  Few tokens take its 16x16x128 form, which wastes least
// of them, tiles the 32x32x64 one (tile_loop.h).  Sums are fp32; a product of two
// codes has at most 4 significant bits.  An activation of the framework follows
// where asked for, and one rounding to bf16.
//
// Tokens are quantised as fp4_quant.hip does, and kept in the operand order of
// the prepared weights (Fp4Shape), so that a wave's load or copy is 1 KiB in a
// row.  Operands: A = weights, B = tokens: four of a lane's accumulators are
// consecutive outputs of one token.
//
// Measured (M tokens, K, N; without the tokens' own quantisation): 8192 7168
// 2 x 2048 118 us, 4.1 PFLOP/s.  By K, 3584 7168 14336, it takes 66 116 216 (and 67
// 116 215 without the activation, N 4096): 17 us beside the steps, and the steps at
// 4.9 PFLOP/s, where the instruction alone reaches 6.6 on such data.  The matrix
// cores are busy 55% of the waves' cycles, and 18% are waits; what the rest is has
// not been found (LDS moves 192 KB a step, 1536 of 2048 cycles).  37 320 2560 3.8 us
// and 512 4096 4096 15 us, latency of few steps; 1 7168 2 x 2048 5.2 us with it,
// 3.0 TB/s of weights.
#include <hip/hip_runtime.h>

#include "act.h"
#include "experts.h"
#include "fp4_codes.h"
#include "tile_loop.h"

namespace moe {
namespace {

// ---- operand order of rows that have codes and scales

// Rows of a matrix [rows][K] as subtiles of 16; `gated` pairs row blocks of
// two halves of N rows.
struct RowMap {
  int64_t N;
  bool gated;
  __device__ int64_t row(int64_t sub, int r) const {  // < 0: none
    const int64_t n = (gated ? sub >> 1 : sub) * 16 + r;
    return n >= N ? -1 : gated && (sub & 1) ? N + n : n;
  }
};

__global__ void __launch_bounds__(256)
    fp4_pack_kernel(RowMap map, int K, int64_t subs, int ksteps, int64_t pairs, const uint8_t* __restrict__ codes,
                    const uint8_t* __restrict__ scales, uint8_t* __restrict__ packed, uint32_t* __restrict__ pscales) {
  const int units = K / 32, kb = 2 * ksteps;
  const int64_t step = (int64_t)gridDim.x * blockDim.x, me = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (int64_t it = me; it < subs * kb * 64; it += step) {
    const int lane = (int)(it & 63);
    const int64_t sb = it >> 6, sub = sb / kb;
    const int u = (int)(sb - sub * kb) * 4 + (lane >> 4);
    const int64_t row = map.row(sub, lane & 15);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row >= 0 && u < units) v = *(const uint4*)(codes + (row * units + u) * 16);
    ((uint4*)packed)[it] = v;
  }
  for (int64_t it = me; it < ksteps * pairs * 64; it += step) {
    const int lane = (int)(it & 63);
    const int64_t sp = it >> 6, s = sp / pairs, pair = sp - s * pairs;
    const int64_t row = map.row(2 * pair + ((lane >> 4) & 1), lane & 15);
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = (int)(8 * s) + 2 * i + (lane >> 5);
      if (row >= 0 && u < units) v |= (uint32_t)scales[row * units + u] << (8 * i);
    }
    pscales[it] = v;
  }
}

// ---- tokens

// A workgroup per 16 tokens and 512 values: each wave takes 4 tokens, and the
// codes are put in operand order in LDS.
__global__ void __launch_bounds__(256)
    fp4_tokens_kernel(const uint16_t* __restrict__ x, int M, int K, int ksteps, int64_t pairs,
                      uint8_t* __restrict__ packed, uint8_t* __restrict__ pscales) {
  __shared__ uint4 turned[256];
  __shared__ uint8_t bytes[16][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t group = blockIdx.x;
  const int q = blockIdx.y;
  const int c = q * 512 + lane * 8;
  uint4 raw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = group * 16 + wave * 4 + i;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (c < K && row < M) raw[i] = *(const uint4*)(x + row * K + c);
  }
  // this lane's unit of 32 values: K block unit / 4, lane group unit % 4
  const int unit = lane / 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = wave * 4 + i;
    uint32_t m = amax8(raw[i]);
    m = max(m, (uint32_t)__shfl_xor((int)m, 1));
    m = max(m, (uint32_t)__shfl_xor((int)m, 2));
    const uint32_t byte = mxfp4_scale_byte(m);
    ((uint32_t*)turned)[((unit / 4) * 64 + unit % 4 * 16 + r) * 4 + lane % 4] = mxfp4_codes8(raw[i], byte);
    if (lane % 4 == 0) bytes[r][unit] = (uint8_t)byte;
  }
  __syncthreads();
  const int t = threadIdx.x, kb = 2 * ksteps;
  if (q * 4 + t / 64 < kb) ((uint4*)(packed + (group * kb + q * 4) * 1024))[t] = turned[t];
  // dwords of 16 rows x 2 halves of a step's quarters
  const int s = q * 2 + t / 32;
  if (t < 64 && s < ksteps) {
    const int r = t & 15, h = (t >> 4) & 1, u = (t / 32) * 8 + h;
    *(uint32_t*)(pscales + ((s * pairs + group / 2) * 64 + 32 * h + 16 * (group & 1) + r) * 4) =
        bytes[r][u] | bytes[r][u + 2] << 8 | bytes[r][u + 4] << 16 | (uint32_t)bytes[r][u + 6] << 24;
  }
}

__device__ __forceinline__ i32x8_t wide(const i32x4_t& v) { return i32x8_t{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// The gated activations of act.h with the hardware's reciprocal (off by a unit
// in the last place; few tokens get the exact one) for their quotients: a tile of 256 x 256 has 128 of them a
// lane, and nothing beside them.
template <int KIND>
__device__ __forceinline__ float quick_act(const ActParams& p, float g, float u) {
  if constexpr (KIND == kActGeluTanh) {
    const float z = 0.7978845608028654f * (g + 0.044715f * g * g * g);
    return g * __builtin_amdgcn_rcpf(1.0f + __expf(-2.0f * z)) * u;
  } else if constexpr (KIND == kActSwigluOai) {
    const float gc = g > p.limit ? p.limit : g;
    const float uc = u > p.limit ? p.limit : (u < -p.limit ? -p.limit : u);
    return gc * __builtin_amdgcn_rcpf(1.0f + __expf(-p.alpha * gc)) * (uc + p.beta);
  } else if constexpr (KIND == kActRelu2) {
    return relu2(g);
  } else {
    return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
  }
}

// ---- few tokens: FS subtiles x 16 TT tokens per workgroup, whose NW waves
// share K in runs of consecutive steps of 256 and join their sums in LDS in
// wave order.  U steps of a wave are in flight.
//
// FUSED: x is quantised by each workgroup itself into LDS, while the first
// weights are on their way.
// HALVES (a gated map): instead of a pair of subtiles a workgroup takes 8 gate
// rows and the 8 up rows of the same outputs as one operand of 16 rows, so that
// twice as many workgroups share the weights.

template <int NW>
constexpr int kFusedUnits = 4 * NW * 16;  // blocks of 32 that 4 passes of the workgroup quantise

template <int FS, int TT, int NW, int U, bool GATED, bool HALVES, bool FUSED>
__global__ void __launch_bounds__(NW * 64)
    fp4_few_kernel(Fp4Shape s, const uint8_t* __restrict__ prepared, const uint8_t* __restrict__ packed,
                   const uint8_t* __restrict__ pscales, const uint16_t* __restrict__ x, int M,
                   uint16_t* __restrict__ out) {
  static_assert(!GATED || (HALVES ? FS == 1 : FS % 2 == 0), "whole gate and up pairs");
  static_assert(!FUSED || TT == 1, "few tokens");
  __shared__ f32x4_t part[NW][FS * TT][64];
  __shared__ uint4 qcodes[FUSED ? kFusedUnits<NW> : 1];
  __shared__ uint8_t qscale[FUSED ? kFusedUnits<NW> : 4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ks = s.ksteps(), kb = s.kblocks(), ns = s.subtiles(), units = 4 * kb;
  const int sub0 = blockIdx.x * FS;
  const int64_t groups = (M + 15) / 16, tok0 = (int64_t)blockIdx.y * (16 * TT);
  const int r = lane & 15, g = lane >> 4;
  // HALVES: the half blockIdx.x % 2 of both subtiles of pair blockIdx.x / 2
  const int hsub = (blockIdx.x & ~1u) + (r >> 3);
  const int hlane = 16 * g + (blockIdx.x & 1) * 8 + (r & 7);
  const int64_t wpairs = Fp4Shape::pair_cols(ns), xpairs = Fp4Shape::pair_cols(groups);
  const uint32_t* const ws = (const uint32_t*)(prepared + s.codes_bytes(ns));
  const int per = (ks + NW - 1) / NW, s0 = wave * per, s1 = min(ks, s0 + per);

  struct Operands {
    i32x4_t a[U][FS][2], b[U][TT][2];
    uint32_t sa[U][FS], sb[U][TT];  // scales of the two K blocks in bytes 0 and 2
  };
  auto load = [&](int at, Operands& o) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // steps past the run are loaded again, and not multiplied
      const int su = min(at + u, ks - 1);
#pragma unroll
      for (int f = 0; f < FS; ++f) {
        const int64_t sub = HALVES ? hsub : min(sub0 + f, ns - 1);
        const int l = HALVES ? hlane : lane;
        const uint8_t* const p = prepared + (sub * kb + 2 * su) * 1024 + l * 16;
        o.a[u][f][0] = *(const i32x4_t*)p;
        o.a[u][f][1] = *(const i32x4_t*)(p + 1024);
        o.sa[u][f] = ws[(su * wpairs + (sub >> 1)) * 64 + 32 * (g & 1) + 16 * (int)(sub & 1) + (l & 15)] >> (8 * (g >> 1));
      }
      if constexpr (!FUSED)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const int64_t group = min(tok0 / 16 + t, groups - 1);
          const uint8_t* const p = packed + (group * kb + 2 * su) * 1024 + lane * 16;
          o.b[u][t][0] = *(const i32x4_t*)p;
          o.b[u][t][1] = *(const i32x4_t*)(p + 1024);
          o.sb[u][t] = ((const uint32_t*)pscales)[(su * xpairs + (group >> 1)) * 64 + 32 * (g & 1) + 16 * (int)(group & 1) + r] >>
                       (8 * (g >> 1));
        }
    }
  };
  f32x4_t acc[FS][TT];
#pragma unroll
  for (int f = 0; f < FS; ++f)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[f][t] = f32x4_t{};
  auto multiply = [&](int at, Operands& o) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (at + u >= s1) break;  // uniform
      if constexpr (FUSED) {
        const int unit = min(r, M - 1) * units + min(at + u, ks - 1) * 8 + g;
        o.b[u][0][0] = *(const i32x4_t*)(qcodes + unit);
        o.b[u][0][1] = *(const i32x4_t*)(qcodes + unit + 4);
        o.sb[u][0] = qscale[unit] | (uint32_t)qscale[unit + 4] << 16;
      }
#pragma unroll
      for (int f = 0; f < FS; ++f)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          acc[f][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(o.a[u][f][0]), wide(o.b[u][t][0]), acc[f][t],
                                                                       4, 4, 0, (int)o.sa[u][f], 0, (int)o.sb[u][t]);
          acc[f][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(o.a[u][f][1]), wide(o.b[u][t][1]), acc[f][t],
                                                                       4, 4, 2, (int)o.sa[u][f], 2, (int)o.sb[u][t]);
        }
    }
  };

  Operands o;
  if constexpr (FUSED) {
    // 4 lanes per block of 32; block `unit` of all tokens is K block unit % units
    // of token unit / units
    const int all = M * units;
    uint4 raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int unit = (i * NW * 64 + (int)threadIdx.x) / 4, row = unit / units;
      const int c = (unit - row * units) * 32 + (lane & 3) * 8;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (unit < all && c < s.K) raw[i] = *(const uint4*)(x + (int64_t)row * s.K + c);
    }
    __builtin_amdgcn_sched_barrier(0);  // x first: it is needed first
    load(s0, o);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int unit = (i * NW * 64 + (int)threadIdx.x) / 4;
      uint32_t m = amax8(raw[i]);
      m = max(m, (uint32_t)__shfl_xor((int)m, 1));
      m = max(m, (uint32_t)__shfl_xor((int)m, 2));
      const uint32_t byte = mxfp4_scale_byte(m), code = mxfp4_codes8(raw[i], byte);
      if (unit < all) {
        ((uint32_t*)qcodes)[unit * 4 + (lane & 3)] = code;
        if ((lane & 3) == 0) qscale[unit] = (uint8_t)byte;
      }
    }
    __syncthreads();
  } else {
    load(s0, o);
    __builtin_amdgcn_sched_barrier(0);
  }
  multiply(s0, o);
#pragma unroll 1
  for (int b = s0 + U; b < s1; b += U) {
    load(b, o);
    __builtin_amdgcn_sched_barrier(0);
    multiply(b, o);
  }
#pragma unroll
  for (int f = 0; f < FS; ++f)
#pragma unroll
    for (int t = 0; t < TT; ++t) part[wave][f * TT + t][lane] = acc[f][t];
  __syncthreads();
  // output tiles of 16 features x 16 tokens, dealt to the waves
  constexpr int kTiles = (GATED && !HALVES ? FS / 2 : FS) * TT;
  for (int i = wave; i < kTiles; i += NW) {
    const int f = i / TT, t = i % TT;
    f32x4_t v{}, w{};
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      v += part[j][(GATED && !HALVES ? 2 * f : f) * TT + t][lane];
      if (HALVES) w += part[j][t][lane ^ 32];
      if (GATED && !HALVES) w += part[j][(2 * f + 1) * TT + t][lane];
    }
    const int n = HALVES ? blockIdx.x * 8 + 4 * g : (GATED ? sub0 / 2 + f : sub0 + f) * 16 + 4 * g;
    const int64_t m = tok0 + 16 * t + r;
    if ((HALVES && g >= 2) || n >= s.N || m >= M) continue;  // N % 8 == 0: the lane's four outputs are all in or all out
    if (s.has_act)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = gated_act(s.act, v[e], w[e]);
    *(uint2*)(out + m * s.N + n) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  }
}

// ---- many tokens

// Rows in operand order: a slot holds ROWS / 16 subtiles x 2 halves x 1 KiB.
// Subtiles past the last are zero.  A wave's fragments are STRIDE fragments
// apart.
template <int ROWS, int STRIDE>
struct PackSource {
  static constexpr int kCopies = ROWS / 32;
  i32x4_t buffer, now;  // kept, and for the next copies
  uint32_t stride;     // bytes of two subtiles
  uint32_t off, soff, gap;  // this lane's bytes of a copy; of the next copy; from one to the next
  uint32_t at;
  int wave;
  __device__ void lanes(int first, int w, int lane) {
    wave = w;
    off = lane * 16;
    at = (uint32_t)first * 4096 + ((lane >> 4) & 1) * 2048 + (lane >> 5) * 256 + (lane & 15) * 16;
  }
  __device__ void set(const uint8_t* p, int kb, int64_t sub0, int64_t subs) {
    // a wave copies one half of every other subtile
    const int64_t mine = (int64_t)(wave / 2) * kb * 1024 + (wave & 1) * 1024;
    const int64_t all = min((int64_t)(ROWS / 16), subs - sub0) * kb * 1024 - mine;
    buffer = buffer_of(uniform(p + sub0 * kb * 1024 + mine), all > 0 ? (uint32_t)all : 0u);
    stride = __builtin_amdgcn_readfirstlane(2 * kb * 1024);
  }
  __device__ __forceinline__ void start(int step) {
    now = scalar(buffer);
    soff = (uint32_t)__builtin_amdgcn_readfirstlane(step * 2048);
    gap = (uint32_t)__builtin_amdgcn_readfirstlane((int)stride);
  }
  __device__ __forceinline__ void copy(int c, uint32_t lds) {
    copy16(now, off, soff, lds + c * 4096);
    soff += gap;
  }
  // 64 values of 32 rows: two of a K block's four lane groups, of two subtiles
  __device__ __forceinline__ i32x4_t read(const uint8_t* area, int quarter, int f) const {
    return *(const i32x4_t*)(area + at + quarter * 512 + f * (STRIDE * 4096));
  }
};

// The scaled instruction and its scales, which come with each step: a dword per
// lane and fragment, the tokens' BM / 32 and then the weights' BN / 32.
template <class T>
struct Fp4Op {
  static constexpr int kPairs = (T::BM + T::BN) / 32;
  static constexpr bool kWide = T::BM == 256 && T::BN == 256;  // 4 pairs, 1 KiB, a wave: one copy
  static constexpr int kCopies = kWide ? 1 : kPairs / 4;
  static constexpr int kRing = kPairs * 256;
  static_assert(kPairs % 4 == 0, "whole copies");
  const uint8_t* src[kCopies];
  uint32_t stride[kCopies];
  const uint8_t* from[kCopies];  // of the next step
  uint32_t lds, lane_off, to;
  const uint8_t* mine;  // this lane's dword of the wave's first token fragment
  int weights;          // from there to its first weight fragment, bytes
  struct Scales {
    uint32_t m[T::FM], n[T::FN];
  };
  __device__ void lanes(uint8_t* ring, int wm, int wn, int wave, int lane) {
    lane_off = lane * (kWide ? 16 : 4);
    lds = lds_addr(ring) + wave * kCopies * (kWide ? 1024 : 256);
    mine = ring + wm * 256 + lane * 4;
    weights = (T::BM / 32 + wn * T::FN - wm) * 256;
  }
  __device__ void set(const uint8_t* xs, int64_t xpairs, int64_t xpair0, const uint8_t* ws, int64_t wpairs,
                      int64_t wpair0, int wave) {
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const int pair = kWide ? wave * 4 : wave * kCopies + c;
      const bool tokens = pair < T::BM / 32;
      stride[c] = (uint32_t)((tokens ? xpairs : wpairs) * 256);
      src[c] = uniform(tokens ? xs + (xpair0 + pair) * 256 : ws + (wpair0 + pair - T::BM / 32) * 256);
    }
  }
  __device__ __forceinline__ void start(int step, int ring) {
    to = lds + ring * kRing;
#pragma unroll
    for (int c = 0; c < kCopies; ++c) from[c] = src[c] + (uint64_t)step * stride[c];
  }
  __device__ __forceinline__ void copy(int c) const {
    if (kWide)
      dma16_at(from[c], lane_off, to);
    else
      dma4_at(from[c], lane_off, to + c * 256);
  }
  __device__ __forceinline__ void read(int ring, Scales& s) const {
    const uint8_t* const p = mine + ring * kRing;
#pragma unroll
    for (int i = 0; i < T::FM; ++i) s.m[i] = *(const uint32_t*)(p + i * T::WM * 256);
#pragma unroll
    for (int i = 0; i < T::FN; ++i) s.n[i] = *(const uint32_t*)(p + weights + i * 256);
  }
  template <int QUARTER, int F, int M>
  __device__ __forceinline__ f32x16_t mul(const i32x4_t& a, const i32x4_t& b, const f32x16_t& c, const Scales& s) const {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(a), wide(b), c, 4, 4, QUARTER, (int)s.n[F], QUARTER,
                                                           (int)s.m[M]);
  }
};

template <class T>
constexpr int kFp4Lds = T::kRing + 2 * Fp4Op<T>::kRing;

// Outputs of a token, at most, of which a fragment's 32 rows are one buffer (TileOut).
constexpr int kTileMaxN = kOutside / (32 * 2);

struct TileArgs {
  Fp4Shape s;
  const uint8_t* prepared;
  const uint8_t* packed;
  const uint8_t* pscales;
  int M, tiles_m, tiles_n;
  uint16_t* out;
};

template <class T, bool GATED>
struct LinearWork {
  PackSource<T::BM, T::WM> p;
  PackSource<T::BN, 1> q;
  Fp4Op<T> op;

  Places places;
  int lane, wave, wm, wn;
  Parked row0, col0;  // of the tile that is computed

  enum { kM, kN, kSteps };

  __device__ LinearWork(uint8_t* ring, int w)
      : lane(threadIdx.x & 63), wave(w), wm(w % T::WM), wn(w / T::WM) {
    p.lanes(wm, wave, lane);
    q.lanes(wn * T::FN, wave, lane);
    op.lanes(ring, wm, wn, wave, lane);
  }
  // Workgroups are dealt to the 8 XCDs in turn: each XCD has a contiguous range
  // of tiles, in bands of 4 token tiles, so that what runs together on it shares
  // token and weight tiles in its L2.
  __device__ bool locate(int i, int& m, int& n) const {
    const auto& a = kernel_args<TileArgs>();
    const int total = a.tiles_m * a.tiles_n, share = (total + 7) / 8;
    const int64_t slot = blockIdx.x / 8 + (int64_t)i * (gridDim.x / 8);
    const int64_t at = (blockIdx.x % 8) * (int64_t)share + slot;
    if (slot >= share || at >= total) return false;
    const int band = (int)at / (4 * a.tiles_n), in_band = (int)at - band * 4 * a.tiles_n;
    const int bm = min(4, a.tiles_m - 4 * band);
    n = in_band / bm;
    m = 4 * band + in_band % bm;
    return true;
  }
  __device__ static Fp4Shape shape() {
    const auto& a = kernel_args<TileArgs>();
    Fp4Shape s;
    s.K = a.s.K;
    s.N = a.s.N;
    s.gated = GATED;
    return s;
  }
  __device__ int steps(int i) const { return places.get(i, kSteps); }
  __device__ int find(int i) {
    int m, n;
    if (!locate(i, m, n)) {
      places.clear(i);
      return 0;
    }
    places.put(i, kM, m);
    places.put(i, kN, n);
    places.put(i, kSteps, shape().ksteps());
    return shape().ksteps();
  }
  __device__ void set_p(int i) {
    const auto& a = kernel_args<TileArgs>();
    p.set(a.packed, shape().kblocks(), (int64_t)places.get(i, kM) * (T::BM / 16), ((int64_t)a.M + 15) / 16);
  }
  __device__ void set_q(int i) {
    const auto& a = kernel_args<TileArgs>();
    const Fp4Shape s = shape();
    const int ns = s.subtiles(), m = places.get(i, kM), n = places.get(i, kN);
    q.set(a.prepared, s.kblocks(), (int64_t)n * (T::BN / 16), ns);
    op.set(a.pscales, Fp4Shape::pair_cols(((int64_t)a.M + 15) / 16), (int64_t)m * (T::BM / 32),
           a.prepared + s.codes_bytes(ns), Fp4Shape::pair_cols(ns), (int64_t)n * (T::BN / 32), wave);
  }
  __device__ int begin(int i) {
    row0 = places.get(i, kM) * T::BM;
    col0 = places.get(i, kN) * T::BN;
    return min(T::FM, (kernel_args<TileArgs>().M - row0 + 32 * T::WM - 1) / (32 * T::WM));
  }
  static constexpr int kStores = (GATED ? 1 : 2) * T::FN;
  template <int A>
  __device__ __forceinline__ void store(f32x16_t (&acc)[T::FN][A]) {
    const auto& a = kernel_args<TileArgs>();
    const ActParams act = {a.s.act.kind, a.s.act.alpha, a.s.act.beta, a.s.act.limit};
    constexpr int kCols = GATED ? 16 : 32;  // outputs of a fragment
    const int m0 = row0, N = a.s.N, n1 = (int)col0 / (GATED ? 2 : 1) + wn * T::FN * kCols;
    // a buffer for each fragment: a whole tile's rows of a wide map pass 32 bits
    // (8192 7168 2 x 2048: 148.3 us a call both ways)
    const uint32_t ld = 2u * (uint32_t)N, row = (threadIdx.x & 31) * ld;
    const uint8_t* const first = uniform(a.out + (int64_t)(m0 + wm * 32) * N + n1);
    const uint64_t gap = 32ull * T::WM * ld;
    const int left = __builtin_amdgcn_readfirstlane(a.M - m0 - wm * 32);
    auto put = [&](auto kind) __attribute__((always_inline)) {
      constexpr int kKind = decltype(kind)::value;
#pragma unroll
      for (int t = 0; t < A; ++t) {
        hold<T>(acc, t);
        const TileOut o(first + t * gap, ld, max(min(32, left - t * 32 * T::WM), 0));
#pragma unroll
        for (int f = 0; f < T::FN; ++f) {
          store_fragment(o, row + 2 * kCols * f, N - n1 - kCols * f, kCols / 8, [&](int i) __attribute__((always_inline)) {
            if constexpr (kKind < 0)
              return acc[f][t][i];
            else
              return quick_act<kKind>(act, acc[f][t][i], GATED ? acc[f][t][i + 8] : 0.0f);  // rows 16 on: up
          });
        }
      }
    };
    if constexpr (GATED) {
      if (act.kind == kActGeluTanh) put(std::integral_constant<int, kActGeluTanh>{});
      else if (act.kind == kActSwigluOai) put(std::integral_constant<int, kActSwigluOai>{});
      else put(std::integral_constant<int, kActSilu>{});
    } else {
      if (a.s.has_act) put(std::integral_constant<int, kActRelu2>{});
      else put(std::integral_constant<int, -1>{});
    }
  }
};

template <class T, bool GATED>
__global__ void __launch_bounds__(256, T::kPerCu) fp4_tile_kernel(TileArgs) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  LinearWork<T, GATED> work(smem + T::kRing, wave);
  tile_loop<T>(work, smem, wave);
}

// ---- launches

struct Tokens {
  const uint8_t* packed;
  const uint8_t* scales;
  const uint16_t* x;
};

template <class T>
hipError_t launch_tile(const Fp4Shape& s, const uint8_t* prepared, const Tokens& x, int M, uint16_t* out,
                       hipStream_t st) {
  const int tm = (M + T::BM - 1) / T::BM, tn = (s.subtiles() + T::BN / 16 - 1) / (T::BN / 16);
  const int64_t n = (int64_t)tm * tn;
  const dim3 grid(n < T::kGrid ? grid8(n) : (unsigned)T::kGrid);
  const TileArgs a{s, prepared, x.packed, x.scales, M, tm, tn, out};
  if (s.gated)
    hipLaunchKernelGGL((fp4_tile_kernel<T, true>), grid, dim3(256), kFp4Lds<T>, st, a);
  else
    hipLaunchKernelGGL((fp4_tile_kernel<T, false>), grid, dim3(256), kFp4Lds<T>, st, a);
  return hipGetLastError();
}

template <int FS, int TT, int NW, int U, bool FUSED>
hipError_t launch_few(const Fp4Shape& s, const uint8_t* prepared, const Tokens& x, int M, uint16_t* out,
                      hipStream_t st) {
  constexpr bool kHalves = FS == 1;
  const dim3 grid((unsigned)((s.subtiles() + FS - 1) / FS), (unsigned)((M + 16 * TT - 1) / (16 * TT)));
  if (s.gated)
    hipLaunchKernelGGL((fp4_few_kernel<FS, TT, NW, U, true, kHalves, FUSED>), grid, dim3(NW * 64), 0, st, s, prepared,
                       x.packed, x.scales, x.x, M, out);
  else
    hipLaunchKernelGGL((fp4_few_kernel<FS, TT, NW, U, false, false, FUSED>), grid, dim3(NW * 64), 0, st, s, prepared,
                       x.packed, x.scales, x.x, M, out);
  return hipGetLastError();
}

}  // namespace

int64_t fp4_workspace(const Fp4Shape& s, int64_t max_tokens) {
  const int64_t groups = max_tokens < 1 ? 1 : (max_tokens + 15) / 16;
  return align256(s.codes_bytes(groups) + s.scales_bytes(groups));
}

hipError_t launch_fp4_prepare(const Fp4Shape& s, const uint8_t* codes, const uint8_t* scales, uint8_t* prepared,
                              hipStream_t st) {
  const int64_t ns = s.subtiles(), subs = Fp4Shape::padded(ns);
  const int64_t blocks = (subs * s.kblocks() * 64 + 255) / 256;
  hipLaunchKernelGGL(fp4_pack_kernel, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st,
                     RowMap{s.N, s.gated}, s.K, subs, s.ksteps(), Fp4Shape::pair_cols(ns), codes, scales, prepared,
                     (uint32_t*)(prepared + s.codes_bytes(ns)));
  return hipGetLastError();
}

hipError_t launch_fp4_linear(const Fp4Shape& s, const uint8_t* prepared, const uint16_t* x, const uint8_t* xcodes,
                             const uint8_t* xscales, int M, uint16_t* out, uint8_t* ws, hipStream_t st) {
  const int64_t groups = (M + 15) / 16, pairs = Fp4Shape::pair_cols(groups);
  uint8_t* const packed = ws;
  uint8_t* const pscales = ws + s.codes_bytes(groups);
  const Tokens t{packed, pscales, x};
  const int ks = s.ksteps();
#define MOE_FEW(...) launch_few<__VA_ARGS__>(s, prepared, t, M, out, st)
  // Up to 4 tokens in one launch, as far as their blocks fit (us, one / two; M K N:
  // 1 7168 2 x 2048 5.2 / 7.7, 4 4096 4096 5.0 / 6.5, 4 320 2560 4.2 / 5.5), and a
  // launch has fewer than 2^32 threads along x.  8 waves where they hold the
  // blocks (8 / 16: 1 7168 2 x 2048 5.2 / 6.2, 1 2048 7168 5.0 / 6.9), with four
  // steps of each in flight where it has more than one (4 / 1: 1 7168 2 x 2048 5.2
  // / 5.5, 1 4096 4096 4.5 / 4.6; where it has one 1 2048 7168 5.3 / 5.0).
  if (x && M <= 4 && M * ks * 8 <= kFusedUnits<16> && s.subtiles() < 1 << 23) {
    if (M * ks * 8 <= kFusedUnits<8>) return ks > 8 ? MOE_FEW(1, 1, 8, 4, true) : MOE_FEW(1, 1, 8, 1, true);
    return MOE_FEW(1, 1, 16, 2, true);
  }
  if (x) {
    hipLaunchKernelGGL(fp4_tokens_kernel, dim3((unsigned)groups, (unsigned)((s.K + 511) / 512)), dim3(256), 0, st, x, M, s.K,
                       ks, pairs, packed, pscales);
  } else {
    const int64_t blocks = (groups * s.kblocks() * 64 + 255) / 256;
    hipLaunchKernelGGL(fp4_pack_kernel, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st,
                       RowMap{M, false}, s.K, groups, ks, pairs, xcodes, xscales, packed, (uint32_t*)pscales);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // Up to 16 tokens: 16 waves where there are steps for them (us, 16 / 4; M K N: 16
  // 4096 4096 6.6 / 7.0, 16 7168 2 x 2048 7.9 / 8.3, 16 2048 7168 6.7 / 6.3, 16 320
  // 2560 5.8 / 5.5), 16 x 16 outputs (the form for 32: 7.4, 8.6, 6.5, 5.8).  Up to
  // 32: 32 x 32 outputs (as up to 16, and as from 33 on: 32 7168 2 x 2048 8.9 / 10.8
  // / 10.0, 32 2048 7168 6.7 / 7.0 / 7.1, but 32 320 2560 6.3 / 5.7 / 6.3).
  // More tokens: the waves of a workgroup share K, and workgroups of more outputs
  // read the tokens less often (us with the tokens' quantisation, 32 x 64 / 64 x
  // 64 outputs / tiles; M K N: 64 4096 4096 8.9 / 10.0 / 16.5, 192 4096 4096 11.9 /
  // 10.8 / 18.6, 512 4096 4096 19.8 / 18.4 / 19.8, 512 7168 2 x 2048 25 / 23 / 30,
  // 768 4096 4096 27 / 25 / 21.7, 384 2048 7168 16 / 17 / 14.3).  More features than
  // a tile can store go the same way, with 64-bit addresses, whatever it takes (256
  // 64 2^25: 31.8 ms / 10.5 in tiles).
  if (M <= 16) return ks > 8 ? MOE_FEW(1, 1, 16, 1, false) : MOE_FEW(1, 1, 4, 1, false);
  if (M <= 32) return MOE_FEW(2, 2, 8, 1, false);
  const int64_t wide = (M + 63) / 64;
  if (wide * ((s.subtiles() + 1) / 2) <= 256) return MOE_FEW(2, 4, 8, 1, false);
  if (wide * ((s.subtiles() + 3) / 4) <= 512 || s.N > kTileMaxN) return MOE_FEW(4, 4, 8, 1, false);
#undef MOE_FEW
  // 256 x 256 tiles move half the bytes into LDS, 128 x 128 ones fill the chip
  // sooner, two a CU (us, 128 / 256; M K N: 2048 4096 4096, 512 tiles of 128, 33 /
  // 40; 1536 2048 7168, 672, 27 / 29; 2048 2048 7168, 896, 33 / 31; 4096 4096 4096,
  // 1024, 55 / 49; 8192 7168 2 x 2048, 2048, 174 / 141).  The rule does not see K:
  // with few steps the small ones stay ahead (8192 320 2560, 1280, 23.7 / 28.3).
  if ((M + 127) / 128 * (int64_t)((s.subtiles() + 7) / 8) <= 3 * 256)
    return launch_tile<Tile<128, 128, 2, 2, 2>>(s, prepared, t, M, out, st);
  return launch_tile<Tile<256, 256, 2, 2, 2>>(s, prepared, t, M, out, st);
}

}  // namespace moe
