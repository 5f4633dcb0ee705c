// Host-side interface of the kernels around the expert layer: the router
// (router.hip), the FP8 block-scaled linear map (fp8_linear.hip) and the
// fused block norms (block_norm.hip).  Arguments have been checked by
// block_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "layout.h"

namespace moe {

MOE_HD constexpr int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// ---------------------------------------------------------------- router

// Shape of a router and the layout of its prepared weights:
//   codes [plane][expert subtile of 16][K block of 32][lane][16 B]: lane l of
//         a wave holds expert 16 s + l % 16, K values 32 b + 8 (l / 16) .. + 7
//         in bf16, the A operand of v_mfma_f32_16x16x32_bf16.  fp32 weights
//         are three bf16 planes whose sum is the weight exactly
//         (24 = 3 x 8 significant bits).  K blocks past H are zero, up to a
//         multiple of kPadBlocks.
//   norms f32[E]: the experts' 2-norms, rounded up.
//   rows  [E][H]: the weights as they came.
struct RouterShape {
  int E, H, k, groups, top_groups;
  int planes;    // 1 (bf16 weights) or 3 (fp32)
  bool sigmoid;  // else softmax
  bool renorm;
  float scale;

  MOE_HD int subtiles() const { return (E + 15) / 16; }
  static constexpr int kPadBlocks = 8;
  MOE_HD int blocks() const { return (H + 31) / 32; }
  MOE_HD int kblocks() const { return (blocks() + kPadBlocks - 1) / kPadBlocks * kPadBlocks; }
  MOE_HD int64_t plane_bytes() const { return (int64_t)subtiles() * kblocks() * 1024; }
  MOE_HD int64_t norms_offset() const { return planes * plane_bytes(); }
  MOE_HD int64_t rows_offset() const { return align256(norms_offset() + 4ll * E); }
  MOE_HD int64_t prepared_bytes() const { return align256(rows_offset() + (planes == 1 ? 2ll : 4ll) * E * H); }
};

constexpr int kRouterMaxExperts = 512;
constexpr int kRouterMaxTopK = 64;
constexpr int kRouterMaxGroups = 64;

// Workspace for calls of up to max_tokens tokens.
int64_t router_workspace(const RouterShape& s, int64_t max_tokens);
hipError_t launch_router_prepare(const RouterShape& s, const void* weight, uint8_t* prepared, hipStream_t st);
hipError_t launch_route(const RouterShape& s, const uint8_t* prepared, const uint16_t* x, int M, const float* bias,
                        int32_t* ids, float* w, float* logits, uint8_t* ws, hipStream_t st);

// ---------------------------------------------------------------- FP8 linear

// Shape of an FP8 linear map and the layout of its prepared weights.  A
// subtile is 16 weight rows; with a gated activation subtile 2p holds gate
// rows 16p.. and subtile 2p + 1 the up rows 16p.., so that one lane of the
// accumulators gets the gate and the up of the same output.
//   codes  [subtile][K block of 128][half][lane][16 B]: lane l holds row
//          l % 16, K values 128 b + 64 half + 16 (l / 16) .. + 15
//   scales f32 [K block][scale_cols]: the scale of each subtile's 128-row
//          block (128 is a multiple of 16, so a subtile has one); rows are
//          long enough to read 64 from any subtile
// Rows past N and K values past K are zero.
struct Fp8Shape {
  int K, N;
  bool gated;
  ActParams act;
  bool has_act;

  MOE_HD int halves() const { return gated ? 2 : 1; }
  MOE_HD int subtiles() const { return halves() * ((N + 15) / 16); }
  MOE_HD int kblocks() const { return (K + 127) / 128; }
  MOE_HD int64_t codes_bytes() const { return (int64_t)subtiles() * kblocks() * 2048; }
  MOE_HD int64_t prepared_bytes() const { return align256(codes_bytes() + 4ll * scale_cols() * kblocks()); }
  MOE_HD int scale_cols() const { return (subtiles() + 63) / 64 * 64 + 64; }
  // Quantised activations: codes as the weights', [16 tokens][K block][half]
  // [lane][16 B], zeros past the last token; then one scale byte per token and
  // K block, as dwords of 4 K blocks: [kblocks / 4][scale_rows].  (Rows of K
  // bytes would put the rows that a tile takes of a K block on few of the L2's
  // channels where K is a multiple of a large power of two.)
  MOE_HD int64_t scale_rows(int64_t M) const { return (M + 255) / 256 * 256; }
  MOE_HD int64_t code_bytes(int64_t M) const { return (M + 15) / 16 * kblocks() * 2048; }
};

// Workspace for calls of up to max_tokens tokens.
int64_t fp8_workspace(const Fp8Shape& s, int64_t max_tokens);
hipError_t launch_fp8_prepare(const Fp8Shape& s, const uint8_t* codes, const float* scales, uint8_t* prepared,
                              hipStream_t st);
hipError_t launch_fp8_linear(const Fp8Shape& s, const uint8_t* prepared, const uint16_t* x, int M, uint16_t* out,
                             uint8_t* ws, hipStream_t st);

// ---------------------------------------------------------------- block norm

struct NormArgs {
  const void* h;       // residual [M][H], bf16 or fp32
  const uint16_t* y;   // branch output [M][H] or null
  const uint16_t* y2;  // second branch output or null
  const void* gate;    // null, a value per token, or (gate_vector) H per row of stride gate_row (0: all rows
                       // alike), of the weights' type
  const void* post_w;  // [H] or null
  const void* pre_w;   // [H] or null
  void* h_out;         // of the residual's type, or null
  uint16_t* x_out;     // bf16 or null
  int M, H;
  int64_t row0;  // first row of a launch
  int64_t gate_row;
  bool gate_vector, gate_sigmoid, h_f32, w_f32;
  float eps, residual_scale, branch_scale, weight_offset;
};

constexpr int kNormMaxHidden = 32768;

hipError_t launch_block_norm(const NormArgs& a, hipStream_t st);

}  // namespace moe
