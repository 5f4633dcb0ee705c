// Host-side interface of the kernels that lead from 16- and 32-bit experts
// to FP4 ones and run beside them: FP4 quantisation (fp4_quant.hip), the
// MXFP4 linear map (fp4_linear.hip), products grouped by expert
// (grouped.hip) and the routes' grouping (routes.hip).  Arguments have been
// checked by experts_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "block.h"
#include "layout.h"

namespace moe {

constexpr int kMaxCols = 1 << 20;  // values of a row that is quantised or multiplied

// ---------------------------------------------------------------- quantisation

struct QuantArgs {
  const void* x;        // [experts][rows][K], rows `ld` elements apart, bf16 or fp32
  uint8_t* codes;       // [experts][rows][K / 2]
  uint8_t* scales;      // [experts][rows][K / G]
  const float* global;  // [experts], NVFP4; null: g_out is filled from the data
  float* g_out;
  uint32_t* partial;    // [experts][kQuantParts] where g_out is filled
  int64_t experts, rows, ld;
  int K;
  bool nvfp4, f32;
};

// Workgroups that look for an expert's largest magnitude, at most.
constexpr int kQuantParts = 256;

hipError_t launch_fp4_quantize(const QuantArgs& a, hipStream_t st);

struct DequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* global;  // NVFP4
  void* out;            // [experts][rows][K], bf16 or fp32
  int64_t experts, rows;
  int K;
  bool nvfp4, f32;
};

hipError_t launch_fp4_dequantize(const DequantArgs& a, hipStream_t st);

// ---------------------------------------------------------------- routes

constexpr int kGroupMaxExperts = 4096;
constexpr int64_t kGroupMaxRoutes = (int64_t)1 << 22;

int64_t group_routes_workspace(int64_t routes, int E);
hipError_t launch_group_routes(const void* ids, bool i64, int64_t routes, int E, int32_t* offsets, int32_t* order,
                               int32_t* place, uint8_t* ws, hipStream_t st);
hipError_t launch_gather_routes(const uint16_t* x, const int32_t* order, int64_t routes, int k, int H, uint16_t* out,
                                hipStream_t st);
hipError_t launch_combine_routes(const uint16_t* y, const int32_t* place, const float* w, int64_t tokens, int k, int H,
                                 uint16_t* out, hipStream_t st);
hipError_t launch_combine_routes_grad(const uint16_t* dout, const uint16_t* y, const int32_t* place,
                                      const int32_t* order, const float* w, int64_t tokens, int k, int H, uint16_t* dy,
                                      float* dw, hipStream_t st);

// ---------------------------------------------------------------- MXFP4 linear

// Shape of an MXFP4 linear map and the layout of its prepared weights, which
// the quantised tokens share.  A subtile is 16 rows; with a gated activation
// subtile 2p holds gate rows 16p.. and subtile 2p + 1 the up rows 16p.., so
// that one lane of the accumulators gets the gate and the up of the same
// output.
//   codes  [subtile][K block of 128][lane][16 B]: lane l holds row l % 16, K
//          values 128 b + 32 (l / 16) .. + 31, the operand of
//          v_mfma_scale_f32_16x16x128_f8f6f4 and one scale block
//   scales [K step of 256][pair of subtiles][lane] dwords: lane l has row
//          l % 32 of the pair, its byte q the scale of the 32 values from
//          256 step + 64 q + 32 (l / 32) on, the scale operands of v_mfma_scale_
//          f32_32x32x64_f8f6f4 for a step
// K is padded to whole steps and rows to whole pairs of subtiles with zero
// codes and scale bytes; the scales' pairs to `pair_cols`, so that
// a tile of 256 rows can copy its 8 pairs from any of its starts.
struct Fp4Shape {
  int K, N;
  bool gated;
  ActParams act;
  bool has_act;

  MOE_HD int halves() const { return gated ? 2 : 1; }
  MOE_HD int subtiles() const { return halves() * ((N + 15) / 16); }
  MOE_HD int ksteps() const { return (K + 255) / 256; }
  MOE_HD int kblocks() const { return 2 * ksteps(); }
  MOE_HD static int64_t pair_cols(int64_t subtiles) { return (subtiles + 15) / 16 * 8; }
  MOE_HD static int64_t padded(int64_t subtiles) { return (subtiles + 1) / 2 * 2; }
  MOE_HD int64_t codes_bytes(int64_t subs) const { return padded(subs) * kblocks() * 1024; }
  MOE_HD int64_t scales_bytes(int64_t subs) const { return pair_cols(subs) * ksteps() * 256; }
  MOE_HD int64_t prepared_bytes() const { return align256(codes_bytes(subtiles()) + scales_bytes(subtiles())); }
};

// Workspace for calls of up to max_tokens tokens.
int64_t fp4_workspace(const Fp4Shape& s, int64_t max_tokens);
hipError_t launch_fp4_prepare(const Fp4Shape& s, const uint8_t* codes, const uint8_t* scales, uint8_t* prepared,
                              hipStream_t st);
// x, or where it is null the tokens' codes [M][K / 2] and scales [M][K / 32].
hipError_t launch_fp4_linear(const Fp4Shape& s, const uint8_t* prepared, const uint16_t* x, const uint8_t* xcodes,
                             const uint8_t* xscales, int M, uint16_t* out, uint8_t* ws, hipStream_t st);

// ---------------------------------------------------------------- grouped products

struct GroupedArgs {
  const uint16_t* x;       // [rows][K]
  const uint16_t* w;       // [E][N][K], or [E][K][N] with w_kn
  const int32_t* offsets;  // [E + 1]
  uint16_t* y;             // [rows][N]
  int64_t rows;
  int E, K, N;
  bool w_kn;
};

hipError_t launch_grouped(const GroupedArgs& a, hipStream_t st);

struct GroupedGradArgs {
  const uint16_t* dy;      // [rows][N]
  const uint16_t* x;       // [rows][K]
  const int32_t* offsets;  // [E + 1]
  void* dw;                // [E][N][K], bf16 or fp32
  int64_t rows;
  int E, K, N;
  bool f32;
};

hipError_t launch_grouped_weight_grad(const GroupedGradArgs& a, hipStream_t st);

}  // namespace moe
