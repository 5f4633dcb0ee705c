// The routes of tokens grouped by expert, for the products of grouped.hip.
//
// group: a stable counting sort.  A route r = token * k + slot of a valid
// expert gets the grouped row place[r]; an expert's rows are offsets[e] ..
// offsets[e + 1] - 1, in the order of their routes; order[] is the inverse of
// place[].  Stable, so that sums over an expert's rows (weight gradients) have
// one order and the same bits from run to run.  Every wave takes a contiguous
// run of routes, 64 at a time; the lanes of a slice that have the same expert
// find each other by a ballot per bit of the expert's number, and each wave
// counts in a histogram of its own, so no atomic is needed.  One workgroup and
// launch up to 4096 routes (1024 of more than 1024 experts); beyond, a launch that
// counts and one that places, with the counts of all blocks in the workspace and a
// launch between that sums them.  Latency bounds it: 5.3 us for 8 routes of 256
// experts, 19 us for 32768 of 128.
//
// gather, combine and its gradient move whole rows and are bound by memory: a
// lane takes 8 values (16 bytes) at a time.  combine adds a token's rows in
// the order of its slots, in fp32, and rounds once.  Of 4096 tokens x 8 routes x
// 4096 values: 73 us (4.1 TB/s), 67 to 84 (3.6 to 4.5), 100 (5.7).
#include <hip/hip_runtime.h>

#include "decode.h"
#include "experts.h"

namespace moe {
namespace {

constexpr int kPerLane = 4;  // slices of 64 routes per wave

// Waves of a workgroup: their histograms (16 bits a counter) share the LDS.
template <int NW>
constexpr int kHistExperts = NW == 16 ? 1024 : kGroupMaxExperts;
template <int NW>
constexpr int kBlockRoutes = NW * 64 * kPerLane;

int waves_for(int E) { return E <= kHistExperts<16> ? 16 : 4; }

template <typename IdT>
__device__ __forceinline__ int route_expert(const IdT* ids, int64_t r, int64_t R, int E) {
  if (r >= R) return -1;
  const int64_t v = (int64_t)ids[r];
  return v >= 0 && v < E ? (int)v : -1;
}

// Counts the wave's routes of expert e[i] (slice i) in hist (cleared) and
// gives each its rank among the wave's routes of the same expert.
template <int PER>
__device__ __forceinline__ void wave_ranks(const int (&e)[PER], int bits, uint16_t* hist, int (&rank)[PER]) {
  const int lane = threadIdx.x & 63;
  const uint64_t below = lane ? ~0ull >> (64 - lane) : 0ull;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    uint64_t same = __ballot(e[i] >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((e[i] >> b) & 1);
      same &= (e[i] >> b) & 1 ? set : ~set;
    }
    rank[i] = 0;
    if (e[i] >= 0) {
      rank[i] = hist[e[i]] + __popcll(same & below);
    }
    __builtin_amdgcn_wave_barrier();
    if (e[i] >= 0 && (same >> lane) == 1ull) hist[e[i]] = (uint16_t)(rank[i] + 1);  // the last of them
    __builtin_amdgcn_wave_barrier();
  }
}

// Exclusive prefix over a value per thread of a workgroup, and the total.
template <int NW>
__device__ __forceinline__ int block_prefix(int v, int* total) {
  __shared__ int sums[NW];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int in = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(in, d);
    if (lane >= d) in += up;
  }
  __syncthreads();
  if (lane == 63) sums[wave] = in;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < wave) before += sums[w];
    all += sums[w];
  }
  *total = all;
  return before + in - v;
}

// COUNT: counts[block][e] of the workgroup's routes.  Otherwise the places;
// with several blocks, `counts` holds every block's routes of an expert in the
// blocks before it and `totals` the sums over all.
template <typename IdT, int NW, bool COUNT>
__global__ void __launch_bounds__(NW * 64)
    group_routes_kernel(const IdT* __restrict__ ids, int64_t R, int E, int bits, int* __restrict__ counts,
                        const int* __restrict__ totals, int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                        int32_t* __restrict__ place) {
  extern __shared__ __align__(16) uint16_t hist[];  // [NW][E] counters, then int [E]: an expert's first row
  int* const first = (int*)(hist + (int64_t)NW * ((E + 1) / 2 * 2));
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, es = (E + 1) / 2 * 2;
  uint16_t* const mine = hist + wave * es;
  const int64_t r0 = (int64_t)blockIdx.x * kBlockRoutes<NW> + wave * 64 * kPerLane + lane;
  int e[kPerLane], rank[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) e[i] = route_expert(ids, r0 + 64 * i, R, E);
  for (int q = threadIdx.x; q < NW * es / 2; q += NW * 64) ((uint32_t*)hist)[q] = 0;
  __syncthreads();
  wave_ranks(e, bits, mine, rank);
  __syncthreads();
  // per expert: the waves' counts become what the waves before them have, and
  // the total the expert's first row
  const int per = (E + NW * 64 - 1) / (NW * 64);
  const int q0 = min(E, (int)threadIdx.x * per), q1 = min(E, q0 + per);
  const bool one = gridDim.x == 1;
  int run = 0;
  for (int q = q0; q < q1; ++q) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int c = hist[w * es + q];
      hist[w * es + q] = (uint16_t)n;
      n += c;
    }
    if (COUNT) counts[(int64_t)blockIdx.x * E + q] = n;
    if (!COUNT) {
      first[q] = run;
      run += one ? n : totals[q];
    }
  }
  if (COUNT) return;
  int valid;
  const int start = block_prefix<NW>(run, &valid);
  for (int q = q0; q < q1; ++q) {
    const int at = start + first[q];
    if (blockIdx.x == 0) offsets[q] = at;
    first[q] = at + (one ? 0 : counts[(int64_t)blockIdx.x * E + q]);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) offsets[E] = valid;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int64_t r = r0 + 64 * i;
    if (r >= R) break;
    int p = -1;
    if (e[i] >= 0) {
      p = first[e[i]] + mine[e[i]] + rank[i];
      order[p] = (int32_t)r;
    }
    place[r] = p;
    if (r >= valid) order[r] = -1;  // rows of no route
  }
}

// counts[block][e] becomes the sum over the blocks before it, totals[e] that
// over all: 16 experts x 16 runs of blocks per workgroup.
__global__ void __launch_bounds__(256) group_prefix_kernel(int blocks, int E, int* __restrict__ counts,
                                                           int* __restrict__ totals) {
  __shared__ int sums[16][17];
  const int i = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int e = blockIdx.x * 16 + i;
  const int per = (blocks + 15) / 16, b0 = min(blocks, part * per), b1 = min(blocks, b0 + per);
  int n = 0;
  if (e < E)
    for (int b = b0; b < b1; ++b) n += counts[(int64_t)b * E + e];
  sums[part][i] = n;
  __syncthreads();
  int run = 0, all = 0;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    if (q < part) run += sums[q][i];
    all += sums[q][i];
  }
  if (e >= E) return;
  if (part == 0) totals[e] = all;
  for (int b = b0; b < b1; ++b) {
    int* const at = counts + (int64_t)b * E + e;
    const int c = *at;
    *at = run;
    run += c;
  }
}

// ---- rows

// 2048 columns of a row per wave: its lanes' 4 loads are in flight together.
constexpr int kRowLoads = 4, kWaveCols = 64 * 8 * kRowLoads;

// A workgroup takes 4 rows, a wave each, of the column chunk blockIdx.y: a
// launch's x has 64 threads a row, however long that is.
__device__ __forceinline__ int64_t wave_row() {
  return (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

__global__ void __launch_bounds__(256)
    gather_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ order, int64_t rows, int k, int H,
                  uint16_t* __restrict__ out) {
  const int64_t row = wave_row();
  const int col = blockIdx.y * kWaveCols + (threadIdx.x & 63) * 8;
  if (row >= rows) return;
  const int r = order[row];
  const uint16_t* const src = x + (int64_t)(r < 0 ? 0 : r / k) * H;
  uint4 v[kRowLoads];
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i) {
    const int c = col + 512 * i;
    v[i] = make_uint4(0, 0, 0, 0);
    if (r >= 0 && c < H) v[i] = *(const uint4*)(src + c);
  }
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i)
    if (col + 512 * i < H) *(uint4*)(out + row * H + col + 512 * i) = v[i];
}

__device__ __forceinline__ void widen(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// out[t] = sum over t's placed slots j of w[t][j] (1 without w) y[place[t][j]].
// 512 columns per wave; 4 rows in flight.
__global__ void __launch_bounds__(256)
    combine_kernel(const uint16_t* __restrict__ y, const int32_t* __restrict__ place, const float* __restrict__ w,
                   int64_t tokens, int k, int H, uint16_t* __restrict__ out) {
  const int64_t t = wave_row();
  const int c = blockIdx.y * 512 + (threadIdx.x & 63) * 8;
  if (t >= tokens || c >= H) return;
  const int32_t* const at = place + t * k;
  float acc[8] = {};
  for (int j0 = 0; j0 < k; j0 += 4) {
    uint4 v[4];
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int p = j0 + j < k ? at[j0 + j] : -1;
      v[j] = make_uint4(0, 0, 0, 0);
      f[j] = 0.0f;
      if (p >= 0) {
        v[j] = *(const uint4*)(y + (int64_t)p * H + c);
        f[j] = w ? w[t * k + j0 + j] : 1.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a[8];
      widen(v[j], a);
      // an absent slot adds +0 to a sum that is never -0: the same as leaving it out
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(f[j], a[i], acc[i]);
    }
  }
  *(uint4*)(out + t * H + c) = narrow(acc);
}

// Gradient of combine: dy[place[r]] = w[r] dout[r / k], dw[r] = <dout[r / k],
// y[place[r]]>; routes of no expert have dw 0, rows of no route dy 0.  NW
// waves per route r, which also clear row r where that has no route.
template <int NW>
__global__ void __launch_bounds__(256)
    combine_grad_kernel(const uint16_t* __restrict__ dout, const uint16_t* __restrict__ y,
                        const int32_t* __restrict__ place, const int32_t* __restrict__ order,
                        const float* __restrict__ w, int64_t routes, int k, int H, uint16_t* __restrict__ dy,
                        float* __restrict__ dw) {
  __shared__ float part[4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t r = (int64_t)blockIdx.x * (4 / NW) + wave / NW;
  const bool in = r < routes;
  const int p = in ? place[r] : -1;
  const bool lone = in && order[r] < 0;  // grouped row r has no route
  const float f = p >= 0 ? w[r] : 0.0f;
  const uint16_t* const g = dout + (in ? r / k : 0) * H;
  const int64_t py = (int64_t)(p < 0 ? 0 : p) * H;
  float dot = 0.0f;
  constexpr int kIn = 4;
  for (int c0 = (wave % NW) * 512 + lane * 8; c0 < H; c0 += kIn * NW * 512) {
    uint4 a[kIn], b[kIn];
#pragma unroll
    for (int u = 0; u < kIn; ++u) {
      const int c = c0 + u * NW * 512;
      a[u] = b[u] = make_uint4(0, 0, 0, 0);
      if (p >= 0 && c < H) {
        a[u] = *(const uint4*)(g + c);
        b[u] = *(const uint4*)(y + py + c);
      }
    }
#pragma unroll
    for (int u = 0; u < kIn; ++u) {
      const int c = c0 + u * NW * 512;
      if (c >= H) continue;
      float ga[8], ya[8];
      widen(a[u], ga);
      widen(b[u], ya);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dot = fmaf(ga[i], ya[i], dot);
        ga[i] *= f;
      }
      if (p >= 0) *(uint4*)(dy + py + c) = narrow(ga);
      if (lone) *(uint4*)(dy + r * H + c) = make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d);
  if (NW > 1) {
    if (lane == 0) part[wave] = dot;
    __syncthreads();
    dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i) dot += part[i];
  }
  if (in && lane == 0 && wave % NW == 0) dw[r] = p >= 0 ? dot : 0.0f;
}

template <typename IdT, int NW>
hipError_t group(const IdT* ids, int64_t R, int E, int32_t* offsets, int32_t* order, int32_t* place, uint8_t* ws,
                 hipStream_t st) {
  const int64_t blocks = (R + kBlockRoutes<NW> - 1) / kBlockRoutes<NW>;
  const unsigned grid = (unsigned)(blocks < 1 ? 1 : blocks);
  const unsigned lds = (unsigned)((int64_t)NW * ((E + 1) / 2 * 2) * 2 + 4 * E);
  int bits = 1;
  while (bits < 31 && (1 << bits) < E) ++bits;
  int* const totals = (int*)ws;
  int* const counts = totals + (E + 63) / 64 * 64;
  if (grid > 1) {
    hipLaunchKernelGGL((group_routes_kernel<IdT, NW, true>), dim3(grid), dim3(NW * 64), lds, st, ids, R, E, bits, counts,
                       (const int*)nullptr, offsets, order, place);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(group_prefix_kernel, dim3((E + 15) / 16), dim3(256), 0, st, (int)grid, E, counts, totals);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((group_routes_kernel<IdT, NW, false>), dim3(grid), dim3(NW * 64), lds, st, ids, R, E, bits, counts,
                     (const int*)totals, offsets, order, place);
  return hipGetLastError();
}

template <typename IdT>
hipError_t group_any(const IdT* ids, int64_t R, int E, int32_t* offsets, int32_t* order, int32_t* place, uint8_t* ws,
                     hipStream_t st) {
  return waves_for(E) == 16 ? group<IdT, 16>(ids, R, E, offsets, order, place, ws, st)
                            : group<IdT, 4>(ids, R, E, offsets, order, place, ws, st);
}

}  // namespace

int64_t group_routes_workspace(int64_t routes, int E) {
  const int64_t per = waves_for(E) == 16 ? kBlockRoutes<16> : kBlockRoutes<4>;
  const int64_t blocks = (routes + per - 1) / per;
  return blocks <= 1 ? 256 : align256(4 * ((E + 63) / 64 * 64 + blocks * E));
}

hipError_t launch_group_routes(const void* ids, bool i64, int64_t routes, int E, int32_t* offsets, int32_t* order,
                               int32_t* place, uint8_t* ws, hipStream_t st) {
  return i64 ? group_any((const int64_t*)ids, routes, E, offsets, order, place, ws, st)
             : group_any((const int32_t*)ids, routes, E, offsets, order, place, ws, st);
}

hipError_t launch_gather_routes(const uint16_t* x, const int32_t* order, int64_t routes, int k, int H, uint16_t* out,
                                hipStream_t st) {
  hipLaunchKernelGGL(gather_kernel, dim3((unsigned)((routes + 3) / 4), (H + kWaveCols - 1) / kWaveCols), dim3(256), 0, st,
                     x, order, routes, k, H, out);
  return hipGetLastError();
}

hipError_t launch_combine_routes(const uint16_t* y, const int32_t* place, const float* w, int64_t tokens, int k, int H,
                                 uint16_t* out, hipStream_t st) {
  hipLaunchKernelGGL(combine_kernel, dim3((unsigned)((tokens + 3) / 4), (H + 511) / 512), dim3(256), 0, st, y, place, w,
                     tokens, k, H, out);
  return hipGetLastError();
}

hipError_t launch_combine_routes_grad(const uint16_t* dout, const uint16_t* y, const int32_t* place,
                                      const int32_t* order, const float* w, int64_t tokens, int k, int H, uint16_t* dy,
                                      float* dw, hipStream_t st) {
  const int64_t routes = tokens * k;
  // few routes: a workgroup each, so that a row's loads are in flight together (us,
  // four waves a route / one; H 7168: 8 routes 3.4 / 5.4, 512 4.7 / 6.4, 1024 7.9 /
  // 8.0, 2048 16.5 / 13.0; H 1024: 1024 3.6 / 3.3, 2048 5.3 / 3.7)
  if (routes <= 1024)
    hipLaunchKernelGGL((combine_grad_kernel<4>), dim3((unsigned)routes), dim3(256), 0, st, dout, y, place, order, w, routes,
                       k, H, dy, dw);
  else
    hipLaunchKernelGGL((combine_grad_kernel<1>), dim3((unsigned)((routes + 3) / 4)), dim3(256), 0, st, dout, y, place,
                       order, w, routes, k, H, dy, dw);
  return hipGetLastError();
}

}  // namespace moe
