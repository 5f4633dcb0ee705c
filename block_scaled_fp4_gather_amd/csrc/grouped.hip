// Products grouped by expert over ragged rows, bf16 with fp32 sums.  Rows
// offsets[e] .. offsets[e + 1] - 1 belong to expert e:
//   forward            y[t]  = W[e] x[t]            W [E][N][K]
//   gradient of x      dx[t] = W[e]^T dy[t]         the forward with W [E][K][N]
//   gradient of W      dW[e] = sum_t dy[t] x[t]^T
// Rows of no expert get zeros, and so does the dW of an expert without rows.
// The offsets are read on the GPU; the host knows the number of rows and
// experts, which bounds the tiles.
//
// Many rows go through the tiles of tile_loop.h, few through a kernel that reads
// the weights straight into registers.  Measured (experts, rows, K, N; forward,
// gradient of x, gradient of W): 128 32768 1536 4096 560 to 590, 560 to 610 and 710
// to 820 us, 0.70, 0.70 and 0.55 PFLOP/s by the medians.  The matrix cores are busy
// 47, 51 and 36% of the cycles, an eighth of that for rows that fill up an expert's
// last 64; the weights or their gradient are 1.6 GB, 316 us at the rate of a copy.
// 32 2060 2560 640: 39, 37 and 35 us, 3.0 to 3.4 TB/s, few steps a tile.  256
// experts, 8 rows, K 7168, N 512: 17 us, 3.4 TB/s.
#include <hip/hip_runtime.h>

#include "experts.h"
#include "tile_loop.h"

namespace moe {
namespace {

static_assert(256ll * 4 * kMaxCols <= kOutside, "a tile's rows, of operands and of fp32 outputs, are one buffer");
static_assert((kGroupMaxRoutes / 128 + kGroupMaxExperts) * (kMaxCols / 128) <= 0x7FFFFFFF, "tiles are counted in 32 bits");

// Rows of expert e, whatever the offsets hold: within [0, rows] and not
// negative in number.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e, int64_t rows, int& a, int& b) {
  a = min(max(constant(offsets + e), 0), (int)rows);
  b = max(a, min(constant(offsets + e + 1), (int)rows));
}

// A workgroup's tile i among `total`: each XCD (workgroups are dealt to the 8 in
// turn) has a contiguous range of them, which its workgroups take in turn, so
// that what runs together on it shares rows and weights in its L2.  < 0: none.
__device__ __forceinline__ int64_t tile_of(int64_t total, int i) {
  const int64_t share = (total + 7) / 8, slot = blockIdx.x / 8 + (int64_t)i * (gridDim.x / 8);
  const int64_t t = (blockIdx.x % 8) * share + slot;
  return slot < share && t < total ? t : -1;
}

struct ForwardArgs {
  GroupedArgs g;
  int tiles_n;
};

// y: row tiles of an expert innermost, then its column tiles.
template <class T, bool KN>
struct ForwardWork {
  RowSource<T::BM, T::WM> p;
  std::conditional_t<KN, ColSource<T::BN, 1>, RowSource<T::BN, 1>> q;
  Bf16Op op;

  Places places;
  int total;      // tiles
  int e, before;  // the expert of the tile that was found last, and the tiles before its
  int lane, wave, wm, wn;
  Parked row0, rows, n0;  // of the tile that is computed
  enum { kRow, kRows, kCol, kExpert };

  __device__ explicit ForwardWork(int w) : lane(threadIdx.x & 63), wave(w), wm(w % T::WM), wn(w / T::WM) {
    p.lanes(wm, wave, lane);
    q.lanes(wn * T::FN, wave, lane);
    // The row tiles of all experts, 64 experts at a time, and the expert where
    // this XCD's share of the tiles starts.
    const auto& args = kernel_args<ForwardArgs>();
    const auto& a = args.g;
    const int32_t* const offsets = a.offsets;
    const int E = a.E, R = (int)a.rows, tiles_n = args.tiles_n;
    int64_t all = 0;
    for (int e0 = 0; e0 < E; e0 += 64) all += __builtin_amdgcn_readlane(tiles_upto(offsets, E, R, e0), 63);
    all *= tiles_n;
    total = all <= 0x7FFFFFFF ? (int)all : 0;  // more only where offsets decrease: no tiles then
    const int start = (int)(blockIdx.x % 8) * ((total + 7) / 8);
    e = before = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int upto = tiles_upto(offsets, E, R, e0), here = before + __builtin_amdgcn_readlane(upto, 63) * tiles_n;
      if (here > start || e0 + 64 >= E) {  // the last expert that starts at or before it, of these 64
        const uint64_t past = __ballot(before + upto * tiles_n <= start);
        const int n = __popcll(past) < 63 ? __popcll(past) : 63;
        e = min(e0 + n, E - 1);
        before += n ? __builtin_amdgcn_readlane(upto, n - 1) * tiles_n : 0;
        break;
      }
      before = here;
    }
  }
  // Inclusive sum over the lanes of the row tiles of expert e0 + lane.
  __device__ static int tiles_upto(const int32_t* offsets, int E, int R, int e0) {
    const int lane = threadIdx.x & 63, x = e0 + lane;
    int n = 0;
    if (x < E) {
      const int a = min(max(offsets[x], 0), R), b = max(a, min(offsets[x + 1], R));
      n = (b - a + T::BM - 1) / T::BM;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(n, d);
      if (lane >= d) n += up;
    }
    return n;
  }
  __device__ int steps(int i) const { return places.get(i, kRows) > 0 ? (kernel_args<ForwardArgs>().g.K + 63) / 64 : 0; }
  __device__ int find(int i) {
    const auto& args = kernel_args<ForwardArgs>();
    const auto& a = args.g;
    const int tiles_n = args.tiles_n;
    const int at = (int)tile_of(total, i);
    if (at < 0) {
      places.clear(i);
      return 0;
    }
    // tiles are found in order: from the last one's expert on
    int r0, r1, nt;
    for (;; ++e) {
      expert_rows(a.offsets, e, a.rows, r0, r1);
      nt = (r1 - r0 + T::BM - 1) / T::BM;
      if (e + 1 >= a.E || before + nt * tiles_n > at) break;
      before += nt * tiles_n;
    }
    const int tn = (at - before) / max(nt, 1), tm = (at - before) - tn * nt;
    const int row = r0 + tm * T::BM;
    places.put(i, kRow, row);
    places.put(i, kRows, max(min(T::BM, r1 - row), 0));
    places.put(i, kCol, tn * T::BN);
    places.put(i, kExpert, e);
    return steps(i);
  }
  __device__ void set_p(int i) {
    const auto& a = kernel_args<ForwardArgs>().g;
    p.set(a.x + (int64_t)places.get(i, kRow) * a.K, places.get(i, kRows), a.K);
  }
  __device__ void set_q(int i) {
    const auto& a = kernel_args<ForwardArgs>().g;
    const int col = places.get(i, kCol);
    const uint16_t* const w = a.w + (int64_t)places.get(i, kExpert) * a.N * a.K;
    if constexpr (KN)
      q.set(w + col, 2 * a.N, a.K, a.N - col, lane);
    else
      q.set(w + (int64_t)col * a.K, a.N - col, a.K);
  }
  __device__ int begin(int i) {
    row0 = places.get(i, kRow);
    rows = places.get(i, kRows);
    n0 = places.get(i, kCol);
    return (rows + 32 * T::WM - 1) / (32 * T::WM);
  }
  static constexpr int kStores = 2 * T::FN;
  template <int A>
  __device__ __forceinline__ void store(f32x16_t (&acc)[T::FN][A]) {
    const auto& a = kernel_args<ForwardArgs>().g;
    const int col = n0 + wn * T::FN * 32;
    const TileOut out(a.y + (int64_t)(int)row0 * a.N + col, 2ll * a.N, rows);
#pragma unroll
    for (int t = 0; t < A; ++t) {
      hold<T>(acc, t);
      const uint32_t row = ((t * T::WM + wm) * 32 + (threadIdx.x & 31)) * out.ld;
#pragma unroll
      for (int f = 0; f < T::FN; ++f)
        store_fragment(out, row + 64 * f, a.N - col - 32 * f, 4, [&](int i) { return acc[f][t][i]; });
    }
  }
};

template <class T, bool KN>
__global__ void __launch_bounds__(256, T::kPerCu) grouped_tile_kernel(ForwardArgs) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  ForwardWork<T, KN> work(wave);
  tile_loop<T>(work, smem, wave);
  const auto& a = kernel_args<ForwardArgs>().g;
  // rows of no expert: before the first expert's and after the last one's
  const int d0 = min(max(a.offsets[0], 0), (int)a.rows), d1 = max(d0, min(a.offsets[a.E], (int)a.rows));
  const int64_t dead = d0 + (a.rows - d1), c8 = a.N / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < dead * c8; i += (int64_t)gridDim.x * 256) {
    const int64_t d = i / c8, row = d < d0 ? d : d1 + (d - d0);
    ((uint4*)(a.y + row * a.N))[i - d * c8] = make_uint4(0, 0, 0, 0);
  }
}

// ---- few rows per expert: what bounds it is the weights, read once

// Row tile `at` of BM rows: its expert, first row and rows (0: there is none).
// Each wave looks by itself: lane l sums the tiles of `per` consecutive experts.
struct RowTile {
  int e, row0, rows;
};
__device__ __forceinline__ RowTile row_tile(const int32_t* __restrict__ offsets, int E, int R, int bm, int at) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) / 64, e0 = min(E, lane * per), e1 = min(E, e0 + per);
  int n = 0;
  for (int e = e0; e < e1; ++e) {
    const int a = min(max(offsets[e], 0), R), b = max(a, min(offsets[e + 1], R));
    n += (b - a + bm - 1) / bm;
  }
  int in = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(in, d);
    if (lane >= d) in += up;
  }
  const uint64_t past = __ballot(in > at);
  if (past == 0) return RowTile{0, 0, 0};
  RowTile t{0, 0, 0};
  int before = in - n;
  for (int e = e0; e < e1; ++e) {
    const int a = min(max(offsets[e], 0), R), b = max(a, min(offsets[e + 1], R));
    const int nt = (b - a + bm - 1) / bm;
    if (before <= at && at < before + nt) {
      t.e = e;
      t.row0 = a + (at - before) * bm;
      t.rows = min(bm, b - t.row0);
    }
    before += nt;
  }
  const int owner = __builtin_ctzll(past);
  return RowTile{__builtin_amdgcn_readlane(t.e, owner), __builtin_amdgcn_readlane(t.row0, owner),
                 __builtin_amdgcn_readlane(t.rows, owner)};
}

// 16 rows x 16 features per S waves, NW / S such features' groups a workgroup.
// The S waves share K in runs of blocks of 64 and join their sums in LDS in wave
// order; a wave has 2 U blocks in flight.  Weights are read as they lie: a lane
// takes chunk g and then chunk 4 + g of its row's 128 bytes of a block, so that
// two loads take whole lines, and the rows of x the same, which is all that the
// instruction asks for: their contraction in the same order.  The workgroups of
// the last row tile clear the rows of no expert.
template <int S, int NW, int U>
__global__ void __launch_bounds__(NW * 64) grouped_few_kernel(GroupedArgs a) {
  __shared__ f32x4_t part[S > 1 ? NW : 1][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4, R = (int)a.rows, n0 = (blockIdx.x * (NW / S) + wave / S) * 16;
  const RowTile t = row_tile(a.offsets, a.E, R, 16, blockIdx.y);
  if (blockIdx.y + 1 == gridDim.y) {
    constexpr int kChunks = NW / S * 2;  // of 8 outputs, of a workgroup
    const int d0 = min(max(a.offsets[0], 0), R), d1 = max(d0, min(a.offsets[a.E], R));
    for (int i = threadIdx.x; i < (d0 + R - d1) * kChunks; i += NW * 64) {
      const int d = i / kChunks, row = d < d0 ? d : d1 + (d - d0), n = (blockIdx.x * kChunks + i % kChunks) * 8;
      if (n < a.N) *(uint4*)(a.y + (int64_t)row * a.N + n) = make_uint4(0, 0, 0, 0);
    }
  }
  if (t.rows <= 0) return;
  const int blocks = (a.K + 63) / 64, per = (blocks + S - 1) / S, b0 = wave % S * per, b1 = min(blocks, b0 + per);
  const uint16_t* const w = a.w + ((int64_t)t.e * a.N + min(n0 + r, a.N - 1)) * a.K;
  const uint16_t* const x = a.x + (int64_t)(t.row0 + min(r, t.rows - 1)) * a.K;
  struct Operands {
    i32x4_t w[U][2], x[U][2];
  };
  auto load = [&](int b, Operands& o) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // blocks past the run and chunks past K are read in their place, and not multiplied or zero
        const int k = min(min(b + u, blocks - 1) * 64 + 32 * h + 8 * g, a.K - 8);
        o.w[u][h] = __builtin_nontemporal_load((const i32x4_t*)(w + k));
        o.x[u][h] = *(const i32x4_t*)(x + k);
      }
  };
  f32x4_t acc{};
  auto multiply = [&](int b, Operands& o) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u >= b1) break;  // uniform
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if ((b + u) * 64 + 32 * h + 32 > a.K) {  // uniform: the last chunks
          const bool in = (b + u) * 64 + 32 * h + 8 * g < a.K;
          o.w[u][h] = in ? o.w[u][h] : i32x4_t{};
          o.x[u][h] = in ? o.x[u][h] : i32x4_t{};
        }
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, o.w[u][h]),
                                                      __builtin_bit_cast(bf16x8_t, o.x[u][h]), acc, 0, 0, 0);
      }
    }
  };
  // Two sets of U blocks take turns; the last of a run loads no more.
  Operands o[2];
  auto turn = [&](int b, Operands& now, Operands& next) __attribute__((always_inline)) {
    if (b + U >= b1) {
      multiply(b, now);
      return false;
    }
    load(b + U, next);
    __builtin_amdgcn_sched_barrier(0);
    multiply(b, now);
    __builtin_amdgcn_sched_barrier(0);
    return true;
  };
  if (b0 < b1) {
    load(b0, o[0]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll 1
    for (int b = b0; turn(b, o[0], o[1]) && turn(b + U, o[1], o[0]); b += 2 * U) {}
  }
  if constexpr (S > 1) {
    part[wave][lane] = acc;
    __syncthreads();
    if (wave % S) return;
#pragma unroll
    for (int q = 1; q < S; ++q) acc += part[wave + q][lane];
  }
  const int n = n0 + 4 * g;
  if (n < a.N && r < t.rows)  // N % 8 == 0: the lane's four outputs are all in or all out
    *(uint2*)(a.y + (int64_t)(t.row0 + r) * a.N + n) = make_uint2(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]));
}

// Row tiles that a launch has at most: one partial tile per expert beyond the whole ones.
int64_t row_tiles(const GroupedArgs& a, int bm) { return a.rows / bm + (a.E < a.rows ? a.E : a.rows); }

template <int S, int NW>
hipError_t few(const GroupedArgs& a, hipStream_t st) {
  constexpr int kFeatures = NW / S * 16;
  hipLaunchKernelGGL((grouped_few_kernel<S, NW, 4>), dim3((unsigned)((a.N + kFeatures - 1) / kFeatures), (unsigned)row_tiles(a, 16)),
                     dim3(NW * 64), 0, st, a);
  return hipGetLastError();
}

struct GradArgs {
  GroupedGradArgs g;
  int tiles_n, tiles_k;
};

// dW: BM rows of N x BN columns of K, over the expert's rows (none: one step of
// zeros).  An expert's tiles in bands of 4 row tiles.
template <class T, bool F32>
struct GradWork {
  ColSource<T::BM, T::WM> p;
  ColSource<T::BN, 1> q;
  Bf16Op op;
  static constexpr int kRow = 64 * T::FN, kTurn = 32 * kRow;  // bytes that a wave turns at a time
  uint8_t* turn;

  Places places;
  int lane, wave, wm, wn;
  Parked e, n0, k0;  // of the tile that is computed
  enum { kExpert, kN, kK, kSteps, kFirst, kRows };

  __device__ GradWork(uint8_t* smem, int w) : turn(smem + T::kRing + w * kTurn), lane(threadIdx.x & 63), wave(w), wm(w % T::WM), wn(w / T::WM) {
    p.lanes(wm, wave, lane);
    q.lanes(wn * T::FN, wave, lane);
  }
  __device__ int steps(int i) const { return places.get(i, kSteps); }
  __device__ int find(int i) {
    const auto& args = kernel_args<GradArgs>();
    const auto& a = args.g;
    const int tiles_n = args.tiles_n, tiles_k = args.tiles_k;
    const int64_t each = (int64_t)tiles_n * tiles_k, at = tile_of(each * a.E, i);
    if (at < 0) {
      places.clear(i);
      return 0;
    }
    const int expert = (int)(at / each);
    const int local = (int)(at - expert * each);
    const int band = local / (4 * tiles_k), in_band = local - band * 4 * tiles_k;
    const int bm = min(4, tiles_n - 4 * band);
    int r0, r1;
    expert_rows(a.offsets, expert, a.rows, r0, r1);
    places.put(i, kExpert, expert);
    places.put(i, kN, (4 * band + in_band % bm) * T::BM);
    places.put(i, kK, in_band / bm * T::BN);
    places.put(i, kSteps, r1 > r0 ? (r1 - r0 + 63) / 64 : 1);
    places.put(i, kFirst, r0);
    places.put(i, kRows, r1 - r0);
    return steps(i);
  }
  __device__ void set_p(int i) {
    const auto& a = kernel_args<GradArgs>().g;
    const int n = places.get(i, kN);
    p.set(a.dy + (int64_t)places.get(i, kFirst) * a.N + n, 2 * a.N, places.get(i, kRows), a.N - n, lane);
  }
  __device__ void set_q(int i) {
    const auto& a = kernel_args<GradArgs>().g;
    const int k = places.get(i, kK);
    q.set(a.x + (int64_t)places.get(i, kFirst) * a.K + k, 2 * a.K, places.get(i, kRows), a.K - k, lane);
  }
  __device__ int begin(int i) {
    e = places.get(i, kExpert);
    n0 = places.get(i, kN);
    k0 = places.get(i, kK);
    return min(T::FM, (kernel_args<GradArgs>().g.N - n0 + 32 * T::WM - 1) / (32 * T::WM));
  }
  static constexpr int kStores = (F32 ? 4 : 2) * T::FN;
  template <int A>
  __device__ __forceinline__ void store(f32x16_t (&acc)[T::FN][A]) {
    const auto& a = kernel_args<GradArgs>().g;
    constexpr int kSize = F32 ? 4 : 2;
    [[maybe_unused]] const int h = (threadIdx.x >> 5) & 1;
    const int n = n0, col = k0 + wn * T::FN * 32;
    const int64_t first = ((int64_t)(int)e * a.N + n) * a.K + col;
    const TileOut out((const uint8_t*)a.dw + first * kSize, (int64_t)kSize * a.K, min(T::BM, a.N - n));
#pragma unroll
    for (int t = 0; t < A; ++t) {
      hold<T>(acc, t);
      const int row = (t * T::WM + wm) * 32;
      if constexpr (F32) {
#pragma unroll
        for (int f0 = 0; f0 < T::FN; f0 += T::FN / 2) {
#pragma unroll
          for (int f = f0; f < f0 + T::FN / 2; ++f)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f32x4_t v = {acc[f][t][4 * q], acc[f][t][4 * q + 1], acc[f][t][4 * q + 2], acc[f][t][4 * q + 3]};
              Turn<kRow>{turn}.put(__builtin_bit_cast(u32x4, v), 8 * (f - f0) + 2 * q + h);
            }
          Turn<kRow>{turn}.store(out, row, 128 * f0, 4 * (a.K - col) - 128 * f0);
        }
      } else {
#pragma unroll
        for (int f = 0; f < T::FN; ++f)
          row_chunks(4, [&](int i) { return acc[f][t][i]; },
                     [&](const u32x4& v, int c) { Turn<kRow>{turn}.put(v, 4 * f + c); });
        Turn<kRow>{turn}.store(out, row, 0, 2 * (a.K - col));
      }
    }
  }
};

template <class T, bool F32>
__global__ void __launch_bounds__(256, T::kPerCu) grouped_grad_kernel(GradArgs) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  GradWork<T, F32> work(smem, wave);
  tile_loop<T>(work, smem, wave);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <class T>
unsigned grid_of(int64_t tiles) {
  return tiles < T::kGrid ? grid8(tiles) : (unsigned)T::kGrid;
}

template <class T>
hipError_t tiles(const GroupedArgs& a, hipStream_t st) {
  const int tn = (int)ceil_div(a.N, T::BN);
  // one workgroup more for the rows of no expert
  const dim3 grid(grid_of<T>(row_tiles(a, T::BM) * tn + 1));
  if (a.w_kn)
    hipLaunchKernelGGL((grouped_tile_kernel<T, true>), grid, dim3(256), T::kRing, st, ForwardArgs{a, tn});
  else
    hipLaunchKernelGGL((grouped_tile_kernel<T, false>), grid, dim3(256), T::kRing, st, ForwardArgs{a, tn});
  return hipGetLastError();
}

template <class T>
hipError_t grads(const GroupedGradArgs& a, hipStream_t st) {
  const int tn = (int)ceil_div(a.N, T::BM), tk = (int)ceil_div(a.K, T::BN);
  const dim3 grid(grid_of<T>((int64_t)a.E * tn * tk));
  constexpr int lds = T::kRing + 4 * GradWork<T, false>::kTurn;
  if (a.f32)
    hipLaunchKernelGGL((grouped_grad_kernel<T, true>), grid, dim3(256), lds, st, GradArgs{a, tn, tk});
  else
    hipLaunchKernelGGL((grouped_grad_kernel<T, false>), grid, dim3(256), lds, st, GradArgs{a, tn, tk});
  return hipGetLastError();
}

// Slots of the second operand, and with Deep of both.  The outputs of the gradient
// take the LDS of one more.
template <int QS>
using Large = Tile<256, 256, 2, 2, QS>;
template <int QS>
using Small = Tile<128, 128, 2, 2, QS>;
template <int S>
using Deep = Tile<128, 128, 2, 2, S, S>;

}  // namespace

// The kernel of few rows where 128 x 128 tiles of the most 16-row tiles would not
// give each CU one: a tile's workgroup has its weights' latency to itself then
// (us, few rows / 128 x 128; E rows K N: 256 8 7168 512 17 / 60, 256 32 7168 512
// 57 / 71, 8 1 4096 4096 9 / 34, 32 64 512 512 6.2 / 8.9; above the bound 256 64
// 7168 512 107 / 99, 128 8 1536 4096 29 / 22, 8 16 4096 4096 63 / 39).  K is
// shared by 4 waves where units of 16 x 16 outputs are few (17 us of the first;
// by one wave 42, by 8 21) and long enough for two sets of loads each.
// 256 x 256 tiles where there is one per CU (128 4096 1536 4096: 316, 128 x 128
// 323; 64 4096 1024 2048: 55, 58), the small ones below that (32 2060 2560 640:
// 29, 47; 16 300 2048 1024: 21, 28).  Small ones that have a CU to themselves take
// all of its LDS (five slots / 3 and 2 and two a CU: 256 64 7168 512 86 / 97, 8 64
// 4096 4096 44 / 48, 8 2000 512 264 9.9 / 9.4; where there are more, 4 8000 1024
// 1024 39 / 31).
// The rules count tiles, however full they are: large ones that are half empty
// lose (256 x 256 / the small ones: 256 32768 1024 128 47 / 30, 256 4096 1024 128 23
// / 19.5; gradient of x of 32 2060 2560 640 32 / 27; of W, below, of the first two
// 35 / 30 and 23 / 19.5).
hipError_t launch_grouped(const GroupedArgs& a, hipStream_t st) {
  const int64_t tiny = row_tiles(a, 16);
  if (!a.w_kn && tiny * ceil_div(a.N, 128) < 256) {
    const int64_t waves = tiny * ceil_div(a.N, 16);
    return waves >= 1024 || a.K < 512 ? few<1, 4>(a, st) : waves >= 512 || a.K < 1024 ? few<2, 4>(a, st) : few<4, 4>(a, st);
  }
  if (row_tiles(a, 256) * ceil_div(a.N, 256) >= 256) return tiles<Large<3>>(a, st);
  return row_tiles(a, 128) * ceil_div(a.N, 128) <= 256 ? tiles<Deep<5>>(a, st) : tiles<Small<3>>(a, st);
}

// The same bound as above (us, 256 x 256 / 128 x 128; E rows K N: 128 32768 1536
// 4096 731 / 959, 128 4096 1536 4096 335 / 458, 16 300 2048 1024 19.7 / 19.9;
// below it 8 200 512 264 9.4 / 5.2); the small ones with four slots or two as there
// (3 20000 1000 72: 71 / 86; 8 2000 512 264: 8.4 / 7.9).
hipError_t launch_grouped_weight_grad(const GroupedGradArgs& a, hipStream_t st) {
  if (a.E * ceil_div(a.N, 256) * ceil_div(a.K, 256) >= 256) return grads<Large<2>>(a, st);
  return a.E * ceil_div(a.N, 128) * ceil_div(a.K, 128) <= 256 ? grads<Deep<4>>(a, st) : grads<Small<2>>(a, st);
}

}  // namespace moe
