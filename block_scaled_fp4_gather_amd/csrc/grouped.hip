// Products grouped by expert over ragged rows, bf16 with fp32 sums.  Rows
// offsets[e] .. offsets[e + 1] - 1 belong to expert e:
//   forward            y[t]  = W[e] x[t]            W [E][N][K]
//   gradient of x      dx[t] = W[e]^T dy[t]         the forward with W [E][K][N]
//   gradient of W      dW[e] = sum_t dy[t] x[t]^T
// Rows of no expert get zeros, and so does the dW of an expert without rows.
// The offsets are read on the GPU; the host knows the number of rows and
// experts, which bounds the tiles.
#include <hip/hip_runtime.h>

#include "experts.h"
#include "tile_loop.h"

namespace moe {
namespace {

// Rows of expert e, whatever the offsets hold: within [0, rows] and not
// negative in number.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e, int64_t rows, int& a, int& b) {
  a = min(max(offsets[e], 0), (int)rows);
  b = max(a, min(offsets[e + 1], (int)rows));
}

// Workgroup -> (expert, row tile, column tile).  An expert's tiles follow each
// other, row tiles innermost, so that what runs together on an XCD shares
// weights and rows in its L2: each XCD (workgroups are dealt to the 8 in turn)
// has a contiguous range of the tiles that there are, which every wave finds
// from the offsets by itself: lane l sums the tiles of `per` consecutive
// experts.
struct GroupedTile {
  int e, row0, rows, tm, tn;
  int spare;  // >= 0: no tile, but this number among the workgroups that have none
  int spares;
  int dead0, dead1;  // rows of no expert: below dead0, from dead1 on
};
__device__ __forceinline__ GroupedTile grouped_tile(const int32_t* __restrict__ offsets, int E, int64_t rows, int bm,
                                                    int tiles_n) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) / 64;
  int n = 0;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e >= E) break;
    int a, b;
    expert_rows(offsets, e, rows, a, b);
    n += (b - a + bm - 1) / bm;
  }
  int in = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(in, d);
    if (lane >= d) in += up;
  }
  const int total = __builtin_amdgcn_readlane(in, 63) * tiles_n;
  const int share = (total + 7) / 8;
  GroupedTile t{};
  const int slot = (int)(blockIdx.x / 8), logical = (int)(blockIdx.x % 8) * share + slot;
  t.spare = -1;
  if (slot >= share || logical >= total) {
    t.spare = slot >= share ? (int)blockIdx.x - 8 * share : 0x7FFFFFFF;
    t.spares = (int)gridDim.x - 8 * share;
    t.dead0 = min(max(offsets[0], 0), (int)rows);
    t.dead1 = max(t.dead0, min(offsets[E], (int)rows));
    return t;
  }
  const int at = logical / tiles_n;  // its place among the row tiles
  const int owner = __builtin_ctzll(__ballot(in > at));
  int first = __builtin_amdgcn_readlane(in - n, owner);
  int e = owner * per, a = 0, b = 0, nt = 0;
  for (;; ++e) {
    expert_rows(offsets, e, rows, a, b);
    nt = (b - a + bm - 1) / bm;
    if (first + nt > at) break;
    first += nt;
  }
  const int local = logical - first * tiles_n;
  t.e = e;
  t.tn = local / nt;
  t.tm = local - t.tn * nt;
  t.row0 = a + t.tm * bm;
  t.rows = min(bm, b - t.row0);
  return t;
}

// Rows of no expert, cleared by the workgroups without a tile.
__device__ __forceinline__ void clear_dead(const GroupedTile& t, int64_t rows, int N, uint16_t* __restrict__ y) {
  if (t.spare >= t.spares) return;
  const int64_t dead = t.dead0 + (rows - t.dead1), c8 = N / 8;
  for (int64_t i = (int64_t)t.spare * blockDim.x + threadIdx.x; i < dead * c8; i += (int64_t)t.spares * blockDim.x) {
    const int64_t d = i / c8, row = d < t.dead0 ? d : t.dead1 + (d - t.dead0);
    ((uint4*)(y + row * N))[i - d * c8] = make_uint4(0, 0, 0, 0);
  }
}

template <class T, bool KN>
__global__ void __launch_bounds__(256, 1) grouped_tile_kernel(GroupedArgs a, int tiles_n) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const GroupedTile t = grouped_tile(a.offsets, a.E, a.rows, T::BM, tiles_n);
  if (t.spare >= 0) {
    clear_dead(t, a.rows, a.N, a.y);
    return;
  }
  const int wm = wave % T::WM, wn = wave / T::WM;
  const int n0 = t.tn * T::BN;
  RowSource<T::BM> p;
  p.init(a.x + (int64_t)t.row0 * a.K, 2ll * a.K, t.rows, a.K, wm * T::FM * 32, wave, lane);
  const uint16_t* const w = a.w + (int64_t)t.e * a.N * a.K;
  f32x16_t acc[T::FN][T::FM];
#pragma unroll
  for (int f = 0; f < T::FN; ++f)
#pragma unroll
    for (int m = 0; m < T::FM; ++m) acc[f][m] = f32x16_t{};
  if constexpr (KN) {
    ColSource<T::BN> q;
    q.init(w + n0, 2ll * a.N, a.K, a.N - n0, wn * T::FN * 32, wave, lane);
    tile_loop<T>(p.steps(), p.ragged(), p, q, Bf16Op{}, smem, wave, acc);
  } else {
    RowSource<T::BN> q;
    q.init(w + (int64_t)n0 * a.K, 2ll * a.K, min(T::BN, a.N - n0), a.K, wn * T::FN * 32, wave, lane);
    tile_loop<T>(p.steps(), p.ragged(), p, q, Bf16Op{}, smem, wave, acc);
  }
  __syncthreads();
  const int m1 = wm * T::FM * 32, n1 = n0 + wn * T::FN * 32;
  store_rows<T, false>(smem, wave, lane, a.y + (int64_t)(t.row0 + m1) * a.N + n1, a.N, t.rows - m1, a.N - n1,
                       [&](int f, int m, int i) { return acc[f][m][i]; });
}

// dW[e]: BM rows of N x BN columns of K, over the expert's rows.
template <class T, bool F32>
__global__ void __launch_bounds__(256, 1) grouped_grad_kernel(GroupedGradArgs a, int tiles_n, int tiles_k) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t per = (int64_t)gridDim.x / 8;
  const int64_t logical = (blockIdx.x % 8) * per + blockIdx.x / 8;
  const int64_t each = (int64_t)tiles_n * tiles_k;
  if (logical >= each * a.E) return;
  const int e = (int)(logical / each), local = (int)(logical - e * each);
  // bands of 4 row tiles: what runs together shares dy and x
  const int band = local / (4 * tiles_k), in_band = local - band * 4 * tiles_k;
  const int bm = min(4, tiles_n - 4 * band);
  const int tk = in_band / bm, tn = 4 * band + in_band % bm;
  int r0, r1;
  expert_rows(a.offsets, e, a.rows, r0, r1);
  const int n0 = tn * T::BM, k0 = tk * T::BN;
  const int wm = wave % T::WM, wn = wave / T::WM;
  f32x16_t acc[T::FN][T::FM];
#pragma unroll
  for (int f = 0; f < T::FN; ++f)
#pragma unroll
    for (int m = 0; m < T::FM; ++m) acc[f][m] = f32x16_t{};
  if (r1 > r0) {
    ColSource<T::BM> p;
    ColSource<T::BN> q;
    p.init(a.dy + (int64_t)r0 * a.N + n0, 2ll * a.N, r1 - r0, a.N - n0, wm * T::FM * 32, wave, lane);
    q.init(a.x + (int64_t)r0 * a.K + k0, 2ll * a.K, r1 - r0, a.K - k0, wn * T::FN * 32, wave, lane);
    tile_loop<T>(p.steps(), p.ragged(), p, q, Bf16Op{}, smem, wave, acc);
    __syncthreads();
  }
  const int n1 = n0 + wm * T::FM * 32, k1 = k0 + wn * T::FN * 32;
  const int64_t at = ((int64_t)e * a.N + n1) * a.K + k1;
  if constexpr (F32) {
    const int r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int m = 0; m < T::FM; ++m)
#pragma unroll
      for (int f = 0; f < T::FN; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4_t v = {acc[f][m][4 * q], acc[f][m][4 * q + 1], acc[f][m][4 * q + 2], acc[f][m][4 * q + 3]};
          const int n = 32 * m + r, k = 32 * f + 8 * q + 4 * h;
          if (n1 + n < a.N && k1 + k < a.K) *(f32x4_t*)((float*)a.dw + at + (int64_t)n * a.K + k) = v;
        }
  } else {
    store_rows<T, false>(smem, wave, lane, (uint16_t*)a.dw + at, a.K, a.N - n1, a.K - k1,
                         [&](int f, int m, int i) { return acc[f][m][i]; });
  }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Workgroups: at most one partial row tile per expert beyond the whole ones,
// and some without a tile, for the rows of no expert.
template <class T>
int64_t tile_blocks(const GroupedArgs& a) {
  return (a.rows / T::BM + (a.E < a.rows ? a.E : a.rows)) * ceil_div(a.N, T::BN) + 7 + 64;
}
template <class T>
int64_t grad_blocks(const GroupedGradArgs& a) {
  return a.E * ceil_div(a.N, T::BM) * ceil_div(a.K, T::BN) + 7;
}

template <class T>
hipError_t tiles(const GroupedArgs& a, hipStream_t st) {
  const int tn = (int)ceil_div(a.N, T::BN);
  const dim3 grid((unsigned)(tile_blocks<T>(a) / 8 * 8));
  if (a.w_kn)
    hipLaunchKernelGGL((grouped_tile_kernel<T, true>), grid, dim3(256), 2 * T::kSlot, st, a, tn);
  else
    hipLaunchKernelGGL((grouped_tile_kernel<T, false>), grid, dim3(256), 2 * T::kSlot, st, a, tn);
  return hipGetLastError();
}

template <class T>
hipError_t grads(const GroupedGradArgs& a, hipStream_t st) {
  const int tn = (int)ceil_div(a.N, T::BM), tk = (int)ceil_div(a.K, T::BN);
  const dim3 grid((unsigned)(grad_blocks<T>(a) / 8 * 8));
  if (a.f32)
    hipLaunchKernelGGL((grouped_grad_kernel<T, true>), grid, dim3(256), 2 * T::kSlot, st, a, tn, tk);
  else
    hipLaunchKernelGGL((grouped_grad_kernel<T, false>), grid, dim3(256), 2 * T::kSlot, st, a, tn, tk);
  return hipGetLastError();
}

using Large = Tile<256, 256, 2, 2>;
using Small = Tile<128, 128, 2, 2>;

bool large(const GroupedArgs& a) { return a.rows >= 128ll * a.E; }
bool large(const GroupedGradArgs& a) { return a.N > 128 && a.K > 128; }

constexpr int64_t kMaxGrid = ((int64_t)1 << 24) - 8;

}  // namespace

bool grouped_fits(const GroupedArgs& a) {
  return (large(a) ? tile_blocks<Large>(a) : tile_blocks<Small>(a)) <= kMaxGrid;
}
bool grouped_fits(const GroupedGradArgs& a) {
  return (large(a) ? grad_blocks<Large>(a) : grad_blocks<Small>(a)) <= kMaxGrid;
}

hipError_t launch_grouped(const GroupedArgs& a, hipStream_t st) {
  return large(a) ? tiles<Large>(a, st) : tiles<Small>(a, st);
}

hipError_t launch_grouped_weight_grad(const GroupedGradArgs& a, hipStream_t st) {
  return large(a) ? grads<Large>(a, st) : grads<Small>(a, st);
}

}  // namespace moe
