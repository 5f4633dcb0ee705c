// Main loop of the products of many rows (grouped.hip, fp4_linear.hip): a
// workgroup of 4 waves computes BM x BN outputs, each wave BM / WM x BN / WN of
// them from 32 x 32 matrix instructions whose operands are 32 bytes of a row:
// 16 bf16 or 64 E2M1 values, 16 bytes a lane.  A step is 128 bytes of the
// contraction, two halves of two such quarters.
//
// Both operands come to LDS by direct copies, in a ring of two slots, and from
// there to registers half a step before they are multiplied:
//   half 0 of step s   multiply half 0; read half 1
//   barrier            slot s is read, and the copies for step s + 1 are there
//   half 1             multiply half 1; copy step s + 2 over slot s; read half
//                      0 of step s + 1
// so that a copy has a whole step (2048 cycles of the matrix cores at 256 x
// 256) and an LDS read half of one to arrive, with one barrier a step.  One
// wave per SIMD then keeps its matrix core busy by itself; a wave's 128 x 128
// outputs, which halve the LDS reads of 128 x 64, need 256 accumulators.
// One wave issues a 16 x 16 instruction every 30 cycles or so, though bf16 and
// E2M1 ones take 16 (measured: 1.4 and 5.0 PFLOP/s of zeros; 2.1 and 6.5 with
// two waves); of the 32 x 32 ones, which take 32, it loses little (2.2, 8.5).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "decode.h"
#include "gemm_util.h"

namespace moe {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

// What copies read in the place of values past the end of a contraction.
static __device__ const uint4 zero_chunk = {0, 0, 0, 0};

// f(integral_constant<int, 0>) .. f(integral_constant<int, N - 1>).  (The loop
// over a half's products is past what the compiler unrolls by itself, and an
// accumulator with an index of run time would be memory.)
template <class F, int... I>
__device__ __forceinline__ void static_for(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for(std::make_integer_sequence<int, N>{}, f);
}

template <int BM_, int BN_, int WM_, int WN_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int FM = BM / 32 / WM, FN = BN / 32 / WN;  // a wave's fragments of 32 rows
  static constexpr int kM = BM * 128, kSlot = (BM + BN) * 128;
  static_assert(WM * WN == 4 && BM % 32 == 0 && BN % 32 == 0 && FM > 0 && FN > 0, "4 waves, whole copies");
};

// A value that is not computed ahead of its place: what the cut step alone
// needs stays out of the registers of the whole loop.
__device__ __forceinline__ uint32_t here(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Rows whose contraction is contiguous (bf16): a slot holds ROWS x 128 bytes,
// 16-byte chunk c of row r at position c ^ row_swz(r).  Rows past the last are
// the last again; contraction past its end is zero.
template <int ROWS>
struct RowSource {
  static constexpr int kCopies = ROWS / 32;
  const uint8_t* base;
  uint32_t off[kCopies];  // of this lane's chunk of each copy (8 rows a wave, 32 a workgroup)
  uint32_t chunk;
  uint32_t bytes;  // of the contraction
  uint32_t at;     // of this lane's chunk of quarter 0 in fragment 0

  __device__ void init(const void* p, int64_t ld_bytes, int rows, int64_t k, int first, int wave, int lane) {
    base = (const uint8_t*)p;
    bytes = (uint32_t)(2 * k);
    const int row = wave * 8 + lane / 8;
    chunk = ((lane & 7) ^ row_swz<128>(row)) * 16;
#pragma unroll
    for (int c = 0; c < kCopies; ++c) off[c] = (uint32_t)min(c * 32 + row, rows - 1) * (uint32_t)ld_bytes + chunk;
    const int r = lane & 31, h = lane >> 5;
    at = (uint32_t)(first + r) * 128 + (h ^ row_swz<128>(r)) * 16;
  }
  __device__ int steps() const { return (int)((bytes + 127) / 128); }
  __device__ bool ragged() const { return bytes % 128 != 0; }
  template <bool TAIL>
  __device__ __forceinline__ void copy(int step, int c, uint32_t lds) const {
    const uint8_t* const from = base + (int64_t)step * 128;
    if (TAIL) {
      const bool in = (uint32_t)step * 128 + chunk < bytes;
      dma16(in ? (const void*)(from + here(off[c])) : (const void*)&zero_chunk, lds + c * 4096);
    } else {
      dma16_at(from, off[c], lds + c * 4096);
    }
  }
  __device__ __forceinline__ i32x4_t read(const uint8_t* area, int quarter, int f) const {
    return *(const i32x4_t*)(area + (at ^ (quarter * 32)) + f * 4096);
  }
};

// Operands whose contraction is the memory's row (bf16): a slot holds 64 rows
// of COLS values, and the transposing LDS read gives a lane 4 consecutive
// contraction values of one column.  It takes 4 rows x 32 bytes per 16 lanes;
// 32-byte chunk c of row k is at c ^ (2 (k % 4) + 8 (k / 8 % 2)), so that the 4
// rows and the 2 chunks next to each other of 32 lanes lie in different banks.
// Columns past the last chunk are that chunk again; rows past the last are zero.
template <int COLS>
struct ColSource {
  static constexpr int kCopies = COLS / 32;
  static constexpr int kRow = COLS * 2, kLanes = kRow / 16, kRows = 64 / kLanes;  // a copy's lanes per row, and rows
  static constexpr int kMask = kRow / 32 - 1;
  const uint8_t* base;
  uint32_t off[kCopies];
  int64_t ld;
  int row, rows;           // this lane's row of copy 0; rows of the contraction
  uint32_t at;             // this lane's row and place in a 32-byte chunk
  uint32_t swz, first;     // of its row; its chunk in fragment 0

  __device__ static int swizzle(int k) { return ((k & 3) << 1 | (k & 8)) & kMask; }
  __device__ void init(const void* p, int64_t ld_bytes, int64_t n, int64_t cols, int first_col, int wave, int lane) {
    base = (const uint8_t*)p;
    ld = ld_bytes;
    rows = (int)n;
    row = wave * kRows + lane / kLanes;
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const int k = c * 4 * kRows + row;
      const int chunk = (lane % kLanes) ^ (swizzle(k) << 1);
      off[c] = (uint32_t)k * (uint32_t)ld_bytes + (uint32_t)min((int64_t)chunk, cols / 8 - 1) * 16;
    }
    const int i = lane & 15, q = lane >> 4;
    const int k = 8 * (q >> 1) + (i >> 2);
    at = (uint32_t)k * kRow + (i & 3) * 8;
    swz = (uint32_t)swizzle(k);
    first = (uint32_t)first_col / 16 + (q & 1);
  }
  __device__ int steps() const { return (rows + 63) / 64; }
  __device__ bool ragged() const { return rows % 64 != 0; }
  template <bool TAIL>
  __device__ __forceinline__ void copy(int step, int c, uint32_t lds) const {
    const uint8_t* const from = base + (int64_t)step * 64 * ld;
    if (TAIL) {
      const bool in = step * 64 + c * 4 * kRows + row < rows;
      dma16(in ? (const void*)(from + here(off[c])) : (const void*)&zero_chunk, lds + c * 4096);
    } else {
      dma16_at(from, off[c], lds + c * 4096);
    }
  }
  __device__ __forceinline__ i32x4_t read(const uint8_t* area, int quarter, int f) const {
    const uint32_t a = (uint32_t)(uintptr_t)(const lds_char*)area + at + (((first + 2 * f) ^ swz) & kMask) * 32;
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(a + quarter * 16 * kRow));
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(a + quarter * 16 * kRow + 4 * kRow));
    struct Two {
      s16x4_t a, b;
    };
    return __builtin_bit_cast(i32x4_t, Two{lo, hi});
  }
};

struct Bf16Op {
  static constexpr int kCopies = 0;
  struct Scales {};
  __device__ __forceinline__ void copy(int, int) const {}
  __device__ __forceinline__ void read(int, Scales&) const {}
  template <int QUARTER, int F, int T>
  __device__ __forceinline__ f32x16_t mul(const i32x4_t& a, const i32x4_t& b, const f32x16_t& c, const Scales&) const {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  }
};

// acc[f][t] += rows of q (fragment f, the accumulator's acc_row) times rows of
// p (fragment t, its lane % 32) over `steps` steps, the last of them cut short if
// `ragged`.  `smem` is the ring of 2 slots of T::kSlot; what op copies with
// each step (its scales) it keeps itself.
template <class T, class P, class Q, class Op>
__device__ __forceinline__ void tile_loop(int steps, bool ragged, const P& p, const Q& q, const Op& op,
                                          uint8_t* smem, int wave, f32x16_t (&acc)[T::FN][T::FM]) {
  constexpr int kTiles = T::FN * T::FM, kAll = 2 * kTiles, kOps = T::FM + T::FN, kReads = 2 * kOps;
  constexpr int kCopies = P::kCopies + Q::kCopies + Op::kCopies;
  struct Frags {
    i32x4_t m[2][T::FM], n[2][T::FN];  // two quarters
  };
  Frags r0, r1;
  typename Op::Scales sc, sc_next;
  const uint32_t lds = lds_addr(smem) + wave * 1024;
  auto copy = [&](auto tail, int step, int c) __attribute__((always_inline)) {
    const uint32_t to = lds + (step & 1) * T::kSlot;
    if (c < P::kCopies)
      p.template copy<decltype(tail)::value>(step, c, to);
    else if (c < P::kCopies + Q::kCopies)
      q.template copy<decltype(tail)::value>(step, c - P::kCopies, to + T::kM);
    else
      op.copy(step, c - P::kCopies - Q::kCopies);
  };
  auto copy_all = [&](int step) __attribute__((always_inline)) {
    if (ragged && step == steps - 1) {
#pragma unroll
      for (int c = 0; c < kCopies; ++c) copy(std::true_type{}, step, c);
    } else {
#pragma unroll
      for (int c = 0; c < kCopies; ++c) copy(std::false_type{}, step, c);
    }
  };
  auto read = [&](Frags& r, const uint8_t* slot, int half, int j) __attribute__((always_inline)) {
    const int part = j / kOps, o = j % kOps;
    if (o < T::FN)
      r.n[part][o] = q.read(slot + T::kM, 2 * half + part, o);
    else
      r.m[part][o - T::FN] = p.read(slot, 2 * half + part, o - T::FN);
  };
  // One half: its products, with the next half's reads over the first three
  // quarters of them and a later step's copies between all of them.  The order
  // is pinned.
  auto half = [&](auto h, const Frags& now, Frags& next, const uint8_t* slot, int step) __attribute__((always_inline)) {
    constexpr int H = decltype(h)::value;
    // uniform: copies, none (past the last step), or those of the step that is cut short
    const bool whole = step < steps - (int)ragged, cut = step == steps - 1;
    constexpr int kOver = kAll * 3 / 4 > 0 ? kAll * 3 / 4 : 1;
    static_for<kAll>([&](auto ic) __attribute__((always_inline)) {
      constexpr int i = decltype(ic)::value, part = i / kTiles, t = i % kTiles / T::FN, f = i % T::FN;
      acc[f][t] = op.template mul<2 * H + part, f, t>(now.n[part][f], now.m[part][t], acc[f][t], sc);
      // A product has no side effect, so nothing else would keep it from moving
      // behind the reads, the barrier and the copies that it is to run beside.
      asm volatile("" : "+a"(acc[f][t]));
      __builtin_amdgcn_sched_barrier(0);
      // read j comes after product j kOver / kReads
      constexpr int j0 = i < kOver ? (i * kReads + kOver - 1) / kOver : kReads;
      constexpr int j1 = i + 1 < kOver ? ((i + 1) * kReads + kOver - 1) / kOver : kReads;
      static_for<j1 - j0>([&](auto j) __attribute__((always_inline)) { read(next, slot, 1 - H, j0 + decltype(j)::value); });
      if constexpr (H == 1 && i == 0) op.read(step - 1, sc_next);
      if constexpr (H == 1) {
        constexpr int c0 = i * kCopies / kAll, c1 = (i + 1) * kCopies / kAll;
        if constexpr (c1 > c0) {
          auto some = [&](auto tail) __attribute__((always_inline)) {
            static_for<c1 - c0>([&](auto c) __attribute__((always_inline)) { copy(tail, step, c0 + decltype(c)::value); });
          };
          if (whole)
            some(std::false_type{});
          else if (cut)
            some(std::true_type{});
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  copy_all(0);
  if (steps > 1) {
    copy_all(1);
    vm_wait<kCopies>();
  } else {
    vm_wait<0>();
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kReads; ++j) read(r0, smem, 0, j);
  op.read(0, sc);
#pragma unroll 1
  for (int s = 0; s < steps; ++s) {
    half(std::integral_constant<int, 0>{}, r0, r1, smem + (s & 1) * T::kSlot, 0);
    vm_wait<0>();      // this wave's copies for step s + 1 are there
    __syncthreads();   // everyone's are, and everyone has read slot s
    half(std::integral_constant<int, 1>{}, r1, r0, smem + ((s + 1) & 1) * T::kSlot, s + 2);
    sc = sc_next;
  }
  // The accumulators stay where they are until each is read: without this the
  // compiler moves all of them at once, which takes more registers than there are.
#pragma unroll
  for (int f = 0; f < T::FN; ++f)
#pragma unroll
    for (int t = 0; t < T::FM; ++t) asm volatile("" : "+a"(acc[f][t]));
}

// The wave's outputs as bf16 rows: row m of its part starts at out + m * ld,
// T::FN * 32 outputs (HALF: half of them) of which
// the first `cols` (a multiple of 8, may be 0 or less) and rows below `rows`
// are stored.  They are turned round in the wave's own part of the LDS, so that
// it stores whole rows; 16-byte chunk c of row r lies at c ^ (r % chunks).
// value(f, t, i): the output of accumulator i of fragments f, t (HALF: i < 8).
template <class T, bool HALF, class Value>
__device__ __forceinline__ void store_rows(uint8_t* smem, int wave, int lane, uint16_t* out, int64_t ld, int64_t rows,
                                           int64_t cols, Value value) {
  constexpr int kQuads = HALF ? 2 : 4;  // groups of 8 outputs of a fragment
  constexpr int kRow = T::FN * kQuads * 16, kPer = kRow / 16;
  static_assert(4 * T::FM * 32 * kRow <= 2 * T::kSlot, "the waves' parts");
  uint8_t* const mine = smem + wave * T::FM * 32 * kRow;
  const int r = lane & 31, h = lane >> 5;
#pragma unroll
  for (int t = 0; t < T::FM; ++t) {
    __builtin_amdgcn_sched_barrier(0);  // a fragment row at a time: its values out of the accumulators, no more
#pragma unroll
    for (int f = 0; f < T::FN; ++f)
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        const int c = f * kQuads + q;
        *(uint2*)(mine + (32 * t + r) * kRow + (c ^ (r % kPer)) * 16 + h * 8) =
            make_uint2(pack_bf16(value(f, t, 4 * q), value(f, t, 4 * q + 1)),
                       pack_bf16(value(f, t, 4 * q + 2), value(f, t, 4 * q + 3)));
      }
  }
  wave_sync();
  constexpr int kAtOnce = 64 / kPer > 0 ? 64 / kPer : 1;
  lane = here(threadIdx.x) & 63;  // what is derived of it starts here: the accumulators fill the registers above
  const int c = lane % kPer;
#pragma unroll 4
  for (int i = 0; i < T::FM * 32 / kAtOnce; ++i) {
    const int row = i * kAtOnce + lane / kPer;
    const uint4 v = *(const uint4*)(mine + row * kRow + (c ^ row % kPer) * 16);
    if (row < rows && c * 8 < cols) *(uint4*)(out + row * ld + c * 8) = v;
  }
}

}  // namespace moe
