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

// In LDS, by the 4 waves: row tiles before expert e in start[e], e up to E, and
// its first row and rows.
struct Experts {
  int* start;
  int2* rows;
};
__device__ __forceinline__ void tile_starts(const int32_t* __restrict__ offsets, int E, int64_t rows, int bm,
                                            const Experts& x) {
  __shared__ int sums[4];
  int* const start = x.start;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = (E + 255) / 256, e0 = min(E, (int)threadIdx.x * per), e1 = min(E, e0 + per);
  int n = 0;
  for (int e = e0; e < e1; ++e) {
    int a, b;
    expert_rows(offsets, e, rows, a, b);
    start[e] = n;
    x.rows[e] = make_int2(a, b - a);
    n += (b - a + bm - 1) / bm;
  }
  int in = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(in, d);
    if (lane >= d) in += up;
  }
  if (lane == 63) sums[wave] = in;
  __syncthreads();
  int before = in - n;
  for (int w = 0; w < wave; ++w) before += sums[w];
  for (int e = e0; e < e1; ++e) start[e] += before;
  if (threadIdx.x == 255) start[E] = before + n;
  __syncthreads();
}

// The expert whose row tiles hold tile `at`: the last one that starts at or
// before it.  Every wave looks by itself, 64 experts at a time.
__device__ __forceinline__ int tile_expert(const int* start, int E, int at) {
  const int lane = threadIdx.x & 63, per = (E + 63) / 64;
  const int seg = __popcll(__ballot(lane * per < E && start[min(lane * per, E)] <= at)) - 1;
  const int e = seg * per + lane;
  return seg * per + __popcll(__ballot(lane < per && e < E && start[min(e, E)] <= at)) - 1;
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
  int active;

  Experts x;
  Places places;
  int lane, wave, wm, wn;
  Parked row0, rows, n0;  // of the tile that is computed

  __device__ ForwardWork(const Experts& experts, const Places& ring, int w)
      : x(experts), places(ring), lane(threadIdx.x & 63), wave(w), wm(w % T::WM), wn(w / T::WM) {
    p.lanes(wm, wave, lane);
    q.lanes(wn * T::FN, wave, lane);
  }
  __device__ int fetch(int i) {
    const auto& args = kernel_args<ForwardArgs>();
    const auto& a = args.g;
    const int tiles_n = args.tiles_n;
    const int at = (int)tile_of((int64_t)__builtin_amdgcn_readfirstlane(x.start[a.E]) * tiles_n, i);
    if (at < 0) {
      places.put(i, make_int4(0, 0, 0, 0));
      return 0;
    }
    const int e = tile_expert(x.start, a.E, at / tiles_n);
    const int first = __builtin_amdgcn_readfirstlane(x.start[e]) * tiles_n;
    const int r0 = __builtin_amdgcn_readfirstlane(x.rows[e].x), n = __builtin_amdgcn_readfirstlane(x.rows[e].y);
    const int nt = (n + T::BM - 1) / T::BM;
    const int tn = (at - first) / nt, tm = (at - first) - tn * nt;
    const int row = r0 + tm * T::BM, count = min(T::BM, n - tm * T::BM), col = tn * T::BN;
    places.put(i, make_int4(row, count, col, 0));
    p.set(a.x + (int64_t)row * a.K, count, a.K);
    const uint16_t* const w = a.w + (int64_t)e * a.N * a.K;
    if constexpr (KN)
      q.set(w + col, 2 * a.N, a.K, a.N - col, lane);
    else
      q.set(w + (int64_t)col * a.K, a.N - col, a.K);
    return p.steps();
  }
  __device__ int begin(int i) {
    const int4 t = places.get(i);
    row0 = t.x;
    rows = t.y;
    n0 = t.z;
    active = (t.y + 32 * T::WM - 1) / (32 * T::WM);
    return t.y > 0 ? p.steps() : 0;  // the same for every tile
  }
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
__global__ void __launch_bounds__(256, T::kPerCu) grouped_tile_kernel(ForwardArgs args) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int4 ring[4][4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Experts x{(int*)(smem + 2 * T::kSlot) + 2 * args.g.E, (int2*)(smem + 2 * T::kSlot)};
  tile_starts(args.g.offsets, args.g.E, args.g.rows, T::BM, x);
  ForwardWork<T, KN> work(x, Places{ring[wave]}, wave);
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
  int active;

  Places places;
  int lane, wave, wm, wn;
  Parked e, n0, k0;  // of the tile that is computed

  __device__ GradWork(const Places& ring, int w)
      : places(ring), lane(threadIdx.x & 63), wave(w), wm(w % T::WM), wn(w / T::WM) {
    p.lanes(wm, wave, lane);
    q.lanes(wn * T::FN, wave, lane);
  }
  __device__ int fetch(int i) {
    const auto& args = kernel_args<GradArgs>();
    const auto& a = args.g;
    const int tiles_n = args.tiles_n, tiles_k = args.tiles_k;
    const int64_t each = (int64_t)tiles_n * tiles_k, at = tile_of(each * a.E, i);
    if (at < 0) {
      places.put(i, make_int4(0, 0, 0, 0));
      return 0;
    }
    const int expert = (int)(at / each);
    const int local = (int)(at - expert * each);
    const int band = local / (4 * tiles_k), in_band = local - band * 4 * tiles_k;
    const int bm = min(4, tiles_n - 4 * band);
    const int n = (4 * band + in_band % bm) * T::BM, k = in_band / bm * T::BN;
    int r0, r1;
    expert_rows(a.offsets, expert, a.rows, r0, r1);
    const int steps = r1 > r0 ? (r1 - r0 + 63) / 64 : 1;
    places.put(i, make_int4(expert, n, k, steps));
    p.set(a.dy + (int64_t)r0 * a.N + n, 2 * a.N, r1 - r0, a.N - n, lane);
    q.set(a.x + (int64_t)r0 * a.K + k, 2 * a.K, r1 - r0, a.K - k, lane);
    return steps;
  }
  __device__ int begin(int i) {
    const int4 t = places.get(i);
    e = t.x;
    n0 = t.y;
    k0 = t.z;
    active = min(T::FM, (kernel_args<GradArgs>().g.N - t.y + 32 * T::WM - 1) / (32 * T::WM));
    return t.w;
  }
  template <int A>
  __device__ __forceinline__ void store(f32x16_t (&acc)[T::FN][A]) {
    const auto& a = kernel_args<GradArgs>().g;
    constexpr int kSize = F32 ? 4 : 2;
    const int h = (threadIdx.x >> 5) & 1, n = n0, col = k0 + wn * T::FN * 32;
    const int64_t first = ((int64_t)(int)e * a.N + n) * a.K + col;
    const TileOut out((const uint8_t*)a.dw + first * kSize, (int64_t)kSize * a.K, min(T::BM, a.N - n));
#pragma unroll
    for (int t = 0; t < A; ++t) {
      hold<T>(acc, t);
      const uint32_t row = ((t * T::WM + wm) * 32 + (threadIdx.x & 31)) * out.ld;
#pragma unroll
      for (int f = 0; f < T::FN; ++f) {
        if constexpr (F32) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4_t v = {acc[f][t][4 * q], acc[f][t][4 * q + 1], acc[f][t][4 * q + 2], acc[f][t][4 * q + 3]};
            const int c = 32 * f + 8 * q + 4 * h;
            out.put(__builtin_bit_cast(u32x4, v), c < a.K - col ? row + 4 * c : kOutside);
          }
        } else {
          store_fragment(out, row + 64 * f, a.K - col - 32 * f, 4, [&](int i) { return acc[f][t][i]; });
        }
      }
    }
  }
};

template <class T, bool F32>
__global__ void __launch_bounds__(256, T::kPerCu) grouped_grad_kernel(GradArgs) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  __shared__ int4 ring[4][4];
  GradWork<T, F32> work(Places{ring[wave]}, wave);
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
  // at most one partial row tile per expert beyond the whole ones; one workgroup for the rows of no expert
  const dim3 grid(grid_of<T>((a.rows / T::BM + (a.E < a.rows ? a.E : a.rows)) * tn + 1));
  const unsigned lds = 2 * T::kSlot + 12 * a.E + 4;
  if (a.w_kn)
    hipLaunchKernelGGL((grouped_tile_kernel<T, true>), grid, dim3(256), lds, st, ForwardArgs{a, tn});
  else
    hipLaunchKernelGGL((grouped_tile_kernel<T, false>), grid, dim3(256), lds, st, ForwardArgs{a, tn});
  return hipGetLastError();
}

template <class T>
hipError_t grads(const GroupedGradArgs& a, hipStream_t st) {
  const int tn = (int)ceil_div(a.N, T::BM), tk = (int)ceil_div(a.K, T::BN);
  const dim3 grid(grid_of<T>((int64_t)a.E * tn * tk));
  if (a.f32)
    hipLaunchKernelGGL((grouped_grad_kernel<T, true>), grid, dim3(256), 2 * T::kSlot, st, GradArgs{a, tn, tk});
  else
    hipLaunchKernelGGL((grouped_grad_kernel<T, false>), grid, dim3(256), 2 * T::kSlot, st, GradArgs{a, tn, tk});
  return hipGetLastError();
}

using Large = Tile<256, 256, 2, 2>;
using Small = Tile<128, 128, 2, 2>;

}  // namespace

hipError_t launch_grouped(const GroupedArgs& a, hipStream_t st) {
  return a.rows >= 64ll * a.E ? tiles<Large>(a, st) : tiles<Small>(a, st);
}

hipError_t launch_grouped_weight_grad(const GroupedGradArgs& a, hipStream_t st) {
  return a.N > 128 && a.K > 128 ? grads<Large>(a, st) : grads<Small>(a, st);
}

}  // namespace moe
