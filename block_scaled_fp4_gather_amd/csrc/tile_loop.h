// Main loop of the products of many rows (grouped.hip, fp4_linear.hip): a
// workgroup of 4 waves computes one tile of BM x BN outputs after the other,
// each wave BM / WM x BN / WN of them from 32 x 32 matrix instructions whose
// operands are 32 bytes of a row: 16 bf16 or 64 E2M1 values, 16 bytes a lane.  A
// step is 128 bytes of the contraction, two halves of two such quarters.
//
// Both operands come to LDS by direct copies, in rings of PS and of QS slots,
// and from there to registers half a step before they are multiplied:
//   half 0 of step s   multiply half 0; read half 1
//   barrier            the slots of step s are read, and step s + 1 is there
//   half 1             multiply half 1; copy steps s + PS and s + QS over those of
//                      step s; read half 0 of step s + 1
// so that a copy has a step (2048 cycles of the matrix cores at 256 x 256) to
// arrive with two slots, and with three two: enough for the way from HBM, which
// an operand takes that few tiles share (weights); the other one comes from the
// L2 mostly.  Where a CU has one small tile, of 512 cycles a step, all of its LDS
// is slots.
// An LDS read has half a step, and there is one barrier a step.  The steps of a
// tile and those of the next follow each other without a gap: what is copied
// runs ahead of what is multiplied across tiles, and the outputs go from the
// accumulators to memory beside it.
// One wave per SIMD keeps its matrix core busy by itself; a wave's 128 x 128
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

template <int BM_, int BN_, int WM_, int WN_, int QS_, int PS_ = 2>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int QS = QS_, PS = PS_;  // slots of the second operand, and of the first
  static constexpr int FM = BM / 32 / WM, FN = BN / 32 / WN;  // a wave's fragments of 32 rows
  static constexpr int kM = BM * 128, kN = BN * 128;  // bytes of a slot
  static constexpr int kRing = PS * kM + QS * kN;
  // workgroups of a launch: as many as run at once on the 256 CUs, and of them on an XCD
  static constexpr int kPerCu = kRing <= 81920 ? 2 : 1, kGrid = 256 * kPerCu;
  static_assert(WM * WN == 4 && BM % 32 == 0 && BN % 32 == 0 && FM > 0 && FN > 0, "4 waves, whole copies");
};

__device__ __forceinline__ const uint8_t* uniform(const void* p) {
  const uint64_t v = (uint64_t)p;
  return (const uint8_t*)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v) |
                          (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)) << 32);
}

// `bytes` of memory as a buffer: loads at or past its end give zeros, stores do
// nothing.
__device__ __forceinline__ i32x4_t buffer_of(const uint8_t* p, uint32_t bytes) {
  const uint64_t v = (uint64_t)p;
  return i32x4_t{(int)(uint32_t)v, (int)(uint32_t)(v >> 32), __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}
// The same in scalar registers, wherever it has been kept.
__device__ __forceinline__ i32x4_t scalar(const i32x4_t& b) {
  return i32x4_t{__builtin_amdgcn_readfirstlane(b[0]), __builtin_amdgcn_readfirstlane(b[1]),
                 __builtin_amdgcn_readfirstlane(b[2]), __builtin_amdgcn_readfirstlane(b[3])};
}
// Offsets into a buffer are 32 bits wide, and kOutside has to be past its end:
// whoever makes one keeps it within that many bytes.
constexpr uint32_t kOutside = 0x80000000u;

// Direct copy as in gemm_util.h from a buffer: lane l's 16 bytes at off + scalar
// land at LDS byte lds + 16 l.  One wave of a SIMD has to issue all of its own
// copies beside its products, so m0 is neither saved nor restored: nothing else
// in the kernels of this loop uses it.
__device__ __forceinline__ void copy16(const i32x4_t& buffer, uint32_t off, uint32_t scalar, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :
               : "v"(off), "s"(buffer), "s"(scalar), "s"(lds));
}

// A wave's value that waits in a vector register, of which there are some left.
struct Parked {
  int v;
  __device__ __forceinline__ void operator=(int x) {
    v = x;
    asm volatile("" : "+v"(v));
  }
  __device__ __forceinline__ operator int() const { return __builtin_amdgcn_readfirstlane(v); }
};

// What a workgroup's tiles are, from when they are first copied until they are
// multiplied (up to QS + 1 tiles later): 8 numbers each, in the lanes of a register.
struct Places {
  int lanes;
  __device__ __forceinline__ void put(int i, int field, int v) {
    lanes = (int)(threadIdx.x & 63) == i % 8 * 8 + field ? v : lanes;
  }
  __device__ __forceinline__ void clear(int i) { lanes = (int)(threadIdx.x & 63) / 8 == i % 8 ? 0 : lanes; }
  __device__ __forceinline__ int get(int i, int field) const {
    return __builtin_amdgcn_readlane(lanes, __builtin_amdgcn_readfirstlane(i % 8 * 8 + field));
  }
};

// Memory that no one writes while the kernel runs, read through the scalar
// cache: a load among the copies would wait for all of those before it.
template <class V>
__device__ __forceinline__ V constant(const V* p) {
  return *(const __attribute__((address_space(4))) V*)(uint64_t)p;
}

// A kernel's arguments (one struct) where they are used: read again each time, so
// that the loop's scalar registers do not hold what a tile needs once.
template <class A>
__device__ __forceinline__ const __attribute__((address_space(4))) A& kernel_args() {
  auto p = (const __attribute__((address_space(4))) A*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *p;
}

// Rows whose contraction is contiguous (bf16): a slot holds ROWS x 128 bytes,
// 16-byte chunk c of row r at position c ^ row_swz(r).  Rows past the last and
// contraction past its end are zero.  A wave's fragments are STRIDE fragments
// apart.
template <int ROWS, int STRIDE>
struct RowSource {
  static constexpr int kCopies = ROWS / 32;
  i32x4_t buffer, now;  // kept, and for the next copies
  uint32_t bytes;      // of the contraction, and of a row
  uint32_t off, last;  // this lane's row and chunk of copy 0 (8 rows a wave, 32 a workgroup); the same in the cut step
  uint32_t voff, soff, gap;  // of the next copy; from one to the next
  int row, chunk;
  uint32_t at;         // of this lane's chunk of quarter 0 in fragment 0

  // first: the wave's first fragment
  __device__ void lanes(int first, int wave, int lane) {
    row = wave * 8 + lane / 8;
    chunk = ((lane & 7) ^ row_swz<128>(row)) * 16;
    const int r = lane & 31, h = lane >> 5;
    at = (uint32_t)(first * 32 + r) * 128 + (h ^ row_swz<128>(r)) * 16;
  }
  __device__ void set(const void* p, int rows, int k) {
    bytes = __builtin_amdgcn_readfirstlane(2 * k);
    buffer = buffer_of(uniform(p), (uint32_t)min(rows, ROWS) * bytes);
    off = (uint32_t)row * bytes + chunk;
    last = (bytes & ~127u) + chunk < bytes ? off : kOutside;
  }
  __device__ __forceinline__ void start(int step) {
    now = scalar(buffer);
    soff = (uint32_t)__builtin_amdgcn_readfirstlane(step * 128);
    gap = (uint32_t)__builtin_amdgcn_readfirstlane((int)(32 * bytes));
    voff = soff + 128 > bytes ? last : off;
  }
  __device__ __forceinline__ void copy(int c, uint32_t lds) {
    copy16(now, voff, soff, lds + c * 4096);
    soff += gap;
  }
  __device__ __forceinline__ i32x4_t read(const uint8_t* area, int quarter, int f) const {
    return *(const i32x4_t*)(area + (at ^ (quarter * 32)) + f * (STRIDE * 4096));
  }
};

// Operands whose contraction is the memory's row (bf16): a slot holds 64 rows
// of COLS values, and the transposing LDS read gives a lane 4 consecutive
// contraction values of one column.  It takes 4 rows x 32 bytes per 16 lanes;
// 32-byte chunk c of row k is at c ^ (2 (k % 4) + 8 (k / 8 % 2)), so that the 4
// rows and the 2 chunks next to each other of 32 lanes lie in different banks.
// Columns past the last chunk are that chunk again; rows past the last are zero.
template <int COLS, int STRIDE>
struct ColSource {
  static constexpr int kCopies = COLS / 32;
  static constexpr int kRow = COLS * 2, kLanes = kRow / 16, kRows = 64 / kLanes;  // a copy's lanes per row, and rows
  static constexpr int kMask = kRow / 32 - 1;
  static constexpr int kSwaps = COLS == 256 ? 2 : 1;  // places of a lane's chunk: copies of 8 rows differ in k / 8 % 2
  static_assert(COLS == 256 || COLS == 128, "rows of a copy");
  const uint8_t* base;
  uint32_t ld;             // bytes of a row
  int rows;                // of the contraction
  i32x4_t buffer;
  uint32_t soff, gap;      // of the next copy; from one to the next
  int row;                 // this lane's row of copy 0
  uint32_t off[kSwaps];    // and its chunk there, and in copy 1
  uint32_t at;             // this lane's row and place in a 32-byte chunk
  uint32_t swz, chunk;     // of its row; its chunk in fragment 0

  __device__ static int swizzle(int k) { return ((k & 3) << 1 | (k & 8)) & kMask; }
  __device__ void lanes(int first, int wave, int lane) {
    row = wave * kRows + lane / kLanes;
    const int i = lane & 15, q = lane >> 4;
    const int k = 8 * (q >> 1) + (i >> 2);
    at = (uint32_t)k * kRow + (i & 3) * 8;
    swz = (uint32_t)swizzle(k);
    chunk = (uint32_t)first * 2 + (q & 1);
  }
  // n rows of the contraction (0: all zero), from a column on of which the matrix has `cols` to its end
  __device__ void set(const void* p, int ld_bytes, int n, int cols, int lane) {
    base = uniform(p);
    ld = __builtin_amdgcn_readfirstlane(ld_bytes);
    rows = __builtin_amdgcn_readfirstlane(n);
#pragma unroll
    for (int c = 0; c < kSwaps; ++c)
      off[c] = (uint32_t)row * ld +
               (uint32_t)min((lane % kLanes) ^ (swizzle(c * 4 * kRows + row) << 1), cols / 8 - 1) * 16;
  }
  __device__ __forceinline__ void start(int step) {
    const int left = rows - 64 * step;
    buffer = scalar(buffer_of(base + (uint64_t)(uint32_t)(64 * step) * ld, left > 0 ? (uint32_t)min(left, 64) * ld : 0u));
    soff = 0;
    gap = (uint32_t)__builtin_amdgcn_readfirstlane((int)(4 * kRows * ld));
  }
  __device__ __forceinline__ void copy(int c, uint32_t lds) {
    copy16(buffer, off[c % kSwaps], soff, lds + c * 4096);
    soff += gap;
  }
  __device__ __forceinline__ i32x4_t read(const uint8_t* area, int quarter, int f) const {
    const uint32_t a = (uint32_t)(uintptr_t)(const lds_char*)area + at + (((chunk + 2 * STRIDE * f) ^ swz) & kMask) * 32;
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
  __device__ __forceinline__ void start(int, int) {}
  __device__ __forceinline__ void copy(int) {}
  __device__ __forceinline__ void read(int, Scales&) const {}
  template <int QUARTER, int F, int T>
  __device__ __forceinline__ f32x16_t mul(const i32x4_t& a, const i32x4_t& b, const f32x16_t& c, const Scales&) const {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  }
};

// Computes a workgroup's tiles.  `work` has
//   p, q, op      the sources of the first and the second operand, and the
//                 instruction;
//   find(i)       what the workgroup's tile i is, kept for the calls below; its
//                 steps (0: there is none, and tile 0 of all is copied where one
//                 has to be, and not used);
//   steps(i)      the same;
//   set_p(i), set_q(i)  sets p, and q with op, to tile i;
//   begin(i)      tile i is computed; of T::FM fragments of p's rows, how many
//                 have any (at least 1);
//   kStores       stores of a fragment row, in
//   store(acc)    its outputs: acc[f][t] of rows of q (fragment f, the
//                 accumulator's acc_row) and of p (fragment t, lane % 32).
// `smem` is the ring, T::kRing bytes; what op copies it keeps itself.
template <class T, class Work>
__device__ __forceinline__ void tile_loop(Work& work, uint8_t* smem, int wave) {
  using P = decltype(work.p);
  using Q = decltype(work.q);
  using Op = decltype(work.op);
  static_assert(T::PS == T::QS || (T::PS == 2 && T::QS == 3), "what kLater counts");
  static_assert(Op::kCopies == 0 || T::QS == 2, "the instruction's own copies have two slots");
  constexpr int kOps = T::FM + T::FN, kReads = 2 * kOps;
  constexpr int kCopies = P::kCopies + Q::kCopies + Op::kCopies;
  // Copies that may be on their way when a step's have to be there: those for
  // later ones, which came after them.
  constexpr int kLater = (T::PS - 2) * P::kCopies + (T::QS - 2) * Q::kCopies;
  // Stores of a whole tile that may be too: a wave counts 63 operations.
  constexpr int kFullStores = T::FM * Work::kStores + kLater < 60 ? T::FM * Work::kStores + kLater : 60;
  struct Frags {
    i32x4_t m[2][T::FM], n[2][T::FN];  // two quarters
  };
  Frags r0, r1;
  typename Op::Scales sc, sc_next;
  const uint32_t lds = lds_addr(smem) + wave * 1024;

  // What is copied next of each operand: a step of a tile of the workgroup's.
  struct Cursor {
    int tile, step, steps;
  };
  Cursor cp{0, 0, 0}, cq{0, 0, 0};
  if ((cp.steps = cq.steps = work.find(0)) == 0) return;
  work.set_p(0);
  work.set_q(0);
  auto advance_q = [&]() __attribute__((always_inline)) {
    if (cq.steps > 0 && ++cq.step == cq.steps) {
      cq.step = 0;
      cq.steps = work.find(++cq.tile);
      work.set_q(cq.tile);
    }
  };
  auto advance_p = [&]() __attribute__((always_inline)) {
    if (cp.steps > 0 && ++cp.step == cp.steps) {
      cp.step = 0;
      cp.steps = work.steps(++cp.tile);
      work.set_p(cp.tile);
    }
  };
  // Slots: of the step that is multiplied and the next, which is read.
  int slot = 0, snext = 1, qslot = 0, qnext = 1;
  auto area_p = [&](int s) __attribute__((always_inline)) { return smem + s * T::kM; };
  auto area_q = [&](int s) __attribute__((always_inline)) { return smem + T::PS * T::kM + s * T::kN; };
  // Copy c into slots s and t, the first operand's copies first.
  auto copy = [&](int s, int t, int c) __attribute__((always_inline)) {
    if (c < P::kCopies)
      work.p.copy(c, lds + s * T::kM);
    else if (c < P::kCopies + Q::kCopies)
      work.q.copy(c - P::kCopies, lds + T::PS * T::kM + t * T::kN);
    else
      work.op.copy(c - P::kCopies - Q::kCopies);
  };
  auto read = [&](Frags& r, const uint8_t* ap, const uint8_t* aq, int half, int j) __attribute__((always_inline)) {
    const int part = j / kOps, o = j % kOps;
    if (o < T::FN)
      r.n[part][o] = work.q.read(aq, 2 * half + part, o);
    else
      r.m[part][o - T::FN] = work.p.read(ap, 2 * half + part, o - T::FN);
  };

  static_for<T::QS>([&](auto sc) __attribute__((always_inline)) {
    constexpr int s = decltype(sc)::value, c0 = s < T::PS ? 0 : P::kCopies;
    if constexpr (s < T::PS) work.p.start(cp.step);
    work.q.start(cq.step);
    work.op.start(cq.step, s);
    static_for<kCopies - c0>([&](auto c) __attribute__((always_inline)) { copy(s, s, c0 + decltype(c)::value); });
    advance_q();
    if constexpr (s < T::PS) advance_p();
  });
  vm_wait<kCopies + kLater>();
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kReads; ++j) read(r0, area_p(0), area_q(0), 0, j);
  work.op.read(0, sc);

  int stored = 0;  // fragment rows that the tile before stored
  // A tile with rows in the first A fragments of each wave.
  auto run = [&](auto active, int n) __attribute__((always_inline)) {
    constexpr int A = decltype(active)::value, kTiles = T::FN * A, kAll = 2 * kTiles;
    f32x16_t acc[T::FN][A];
#pragma unroll
    for (int f = 0; f < T::FN; ++f)
#pragma unroll
      for (int t = 0; t < A; ++t) acc[f][t] = f32x16_t{};
    // One half: its products, with the next half's reads over the first three
    // quarters of them and, in the second, a later step's copies between all of
    // them.  The order is pinned.
    auto half = [&](auto h, const Frags& now, Frags& next, const uint8_t* ap, const uint8_t* aq)
                    __attribute__((always_inline)) {
      constexpr int H = decltype(h)::value;
      constexpr int kOver = kAll * 3 / 4 > 0 ? kAll * 3 / 4 : 1;
      static_for<kAll>([&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value, part = i / kTiles, t = i % kTiles / T::FN, f = i % T::FN;
        acc[f][t] = work.op.template mul<2 * H + part, f, t>(now.n[part][f], now.m[part][t], acc[f][t], sc);
        // A product has no side effect, so nothing else would keep it from moving
        // behind the reads, the barrier and the copies that it is to run beside.
        asm volatile("" : "+a"(acc[f][t]));
        __builtin_amdgcn_sched_barrier(0);
        // read j comes after product j kOver / kReads
        constexpr int j0 = i < kOver ? (i * kReads + kOver - 1) / kOver : kReads;
        constexpr int j1 = i + 1 < kOver ? ((i + 1) * kReads + kOver - 1) / kOver : kReads;
        static_for<j1 - j0>([&](auto j) __attribute__((always_inline)) {
          read(next, ap, aq, 1 - H, j0 + decltype(j)::value);
        });
        if constexpr (H == 1) {
          if constexpr (i == 0) {
            work.op.read(slot ^ 1, sc_next);
            work.p.start(cp.step);
            work.q.start(cq.step);
            work.op.start(cq.step, slot);
          }
          constexpr int c0 = i * kCopies / kAll, c1 = (i + 1) * kCopies / kAll;
          static_for<c1 - c0>([&](auto c) __attribute__((always_inline)) { copy(slot, qslot, c0 + decltype(c)::value); });
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    };
#pragma unroll 1
    do {
      half(std::integral_constant<int, 0>{}, r0, r1, area_p(slot), area_q(qslot));
      // This wave's copies for the next step are there; in a tile's first step the
      // stores of the one before, which came after them, may not be.
      if (stored == T::FM)
        vm_wait<kFullStores>();
      else if (stored > 0)
        vm_wait<Work::kStores + kLater>();
      else
        vm_wait<kLater>();
      stored = 0;
      __syncthreads();  // everyone's are, and everyone has read these slots
      half(std::integral_constant<int, 1>{}, r1, r0, area_p(T::PS == 2 ? slot ^ 1 : snext), area_q(qnext));
      sc = sc_next;
      if constexpr (T::PS == 2) {
        slot ^= 1;
      } else {
        slot = snext;
        snext = snext + 1 == T::PS ? 0 : snext + 1;
      }
      qslot = qnext;
      qnext = qnext + 1 == T::QS ? 0 : qnext + 1;
      advance_q();
      advance_p();
    } while (--n > 0);
    work.template store<A>(acc);
    stored = A;
  };
#pragma unroll 1
  for (int i = 0;; ++i) {
    const int n = work.steps(i);
    if (n == 0) break;
    const int active = work.begin(i);
    if constexpr (T::FM > 2) {
      if (active > 3) run(std::integral_constant<int, 4>{}, n);
      else if (active == 3) run(std::integral_constant<int, 3>{}, n);
    }
    if (T::FM <= 2 ? active > 1 : active == 2) run(std::integral_constant<int, 2>{}, n);
    else if (active == 1) run(std::integral_constant<int, 1>{}, n);
  }
  vm_wait<0>();  // no copy may land after the workgroup's LDS is released
}

// A fragment row's accumulators stay where they are up to here: without this the
// compiler moves all of them at once, which takes more registers than there are.
template <class T, int A>
__device__ __forceinline__ void hold(f32x16_t (&acc)[T::FN][A], int t) {
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int f = 0; f < T::FN; ++f) asm volatile("" : "+a"(acc[f][t]));
}

// A tile's outputs, rows of `ld` bytes from its first on (rows * ld: kOutside at
// most): stores past the last row or the matrix's last column do nothing.
struct TileOut {
  __amdgpu_buffer_rsrc_t buffer;
  uint32_t ld;
  __device__ TileOut(const void* first, int64_t ld_bytes, int rows) : ld((uint32_t)ld_bytes) {
    // (a size that the compiler does not know to be uniform would cost a loop at each store)
    buffer = __builtin_amdgcn_make_buffer_rsrc((void*)uniform(first), 0,
                                               __builtin_amdgcn_readfirstlane((int)((uint32_t)rows * ld)), 0x00020000);
  }
  __device__ __forceinline__ void put(const u32x4& v, uint32_t off) const {
    __builtin_amdgcn_raw_buffer_store_b128(v, buffer, off, 0, 0);
  }
};

// Rows of 32 that a wave turns in LDS, so that its stores are of whole rows of
// ROW bytes: a lane has parts of one row, and 16 bytes of 32 rows at a time are
// no whole lines.  16-byte chunk c of row r at position c ^ r.
template <int ROW>
struct Turn {
  static constexpr int kChunks = ROW / 16;
  uint8_t* area;  // of the wave, 32 ROW bytes
  __device__ __forceinline__ void put(const u32x4& v, int c) const {
    const int r = threadIdx.x & 31;
    *(u32x4*)(area + r * ROW + ((c ^ r) % kChunks) * 16) = v;
  }
  // Rows row .. row + 31 of the tile, their first `bytes` (a multiple of 16) from byte `off` on.
  __device__ __forceinline__ void store(const TileOut& out, int row, uint32_t off, int bytes) const {
    const int lane = threadIdx.x & 63, c = lane % kChunks, r0 = lane / kChunks;
    __builtin_amdgcn_wave_barrier();  // the wave's own LDS operations are in order
    u32x4 v[kChunks / 2];
#pragma unroll
    for (int i = 0; i < kChunks / 2; ++i) {
      const int r = r0 + i * (64 / kChunks);
      v[i] = *(const u32x4*)(area + r * ROW + ((c ^ r) % kChunks) * 16);
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < kChunks / 2; ++i)
      out.put(v[i], 16 * c < bytes ? (uint32_t)(row + r0 + i * (64 / kChunks)) * out.ld + off + 16 * c : kOutside);
  }
};

// put(v, c) for the 16-byte chunks c of a row's 32 outputs as bf16 (of 16, for 2
// `quads`) that this lane gets: it has 4 of every 8 of row lane % 32, and the two
// lanes of a row swap, so that the lower has chunks 0 and 2, the upper 1 and 3.
template <class Value, class Put>
__device__ __forceinline__ void row_chunks(int quads, Value value, Put put) {
  const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
  for (int q = 0; q < 4; q += 2) {
    if (q >= quads) break;
    uint32_t v[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) v[i][e] = pack_bf16(value(4 * (q + i) + 2 * e), value(4 * (q + i) + 2 * e + 1));
    const auto lo = __builtin_amdgcn_permlane32_swap(v[0][0], v[1][0], false, false);
    const auto hi = __builtin_amdgcn_permlane32_swap(v[0][1], v[1][1], false, false);
    put(u32x4{lo[0], hi[0], lo[1], hi[1]}, q + h);
  }
}

// Stores such a row's first `cols` (a multiple of 8) outputs at byte `off` of the tile.
template <class Value>
__device__ __forceinline__ void store_fragment(const TileOut& out, uint32_t off, int cols, int quads, Value value) {
  row_chunks(quads, value, [&](const u32x4& v, int c) { out.put(v, 8 * c < cols ? off + 16 * c : kOutside); });
}

}  // namespace moe
