// C-ABI of the operators from 16- and 32-bit experts to FP4 ones and beside
// them (the last part of include/moe_fp4.h): argument checks, sizing and the
// launches.  Every check runs before any HIP call.
#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>

#include "../../include/moe_fp4.h"
#include "experts.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

moe_fp4_status from_hip(hipError_t e) { return e == hipSuccess ? MOE_FP4_OK : MOE_FP4_EHIP; }

// Memory of a call; null is none.
struct Range {
  const void* p;
  int64_t bytes;
  bool meets(const Range& o) const {
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)o.p;
    return p && o.p && a < b + (uintptr_t)o.bytes && b < a + (uintptr_t)bytes;
  }
};

// Whether anything that is written lies on something that is read or written.
bool overlapping(std::initializer_list<Range> in, std::initializer_list<Range> out) {
  for (const Range* o = out.begin(); o != out.end(); ++o) {
    for (const Range& i : in)
      if (o->meets(i)) return true;
    for (const Range* q = out.begin(); q != o; ++q)
      if (o->meets(*q)) return true;
  }
  return false;
}

bool format_ok(int32_t f) { return f == MOE_FP4_MXFP4 || f == MOE_FP4_NVFP4; }
bool type_ok(int32_t t) { return t == MOE_FP4_TYPE_BF16 || t == MOE_FP4_TYPE_F32; }

constexpr int64_t kMaxValues = (int64_t)1 << 40;  // of a quantised tensor

// experts * rows * stride without overflow, or -1 where it passes kMaxValues.
int64_t values(int64_t experts, int64_t rows, int64_t stride) {
  if (experts == 0 || rows == 0) return 0;
  if (experts > kMaxValues || rows > kMaxValues / experts || stride > kMaxValues / (experts * rows)) return -1;
  return experts * rows * stride;
}

constexpr int kMaxTokens = 1 << 20;
constexpr int kMaxOutFeatures = 1 << 26;

moe_fp4_status linear_shape(const moe_fp4_linear_desc* d, moe::Fp4Shape* s) {
  if (!d) return MOE_FP4_EINVAL;
  if (d->in_features <= 0 || d->out_features <= 0 || d->max_tokens < 0) return MOE_FP4_EINVAL;
  if (d->in_features % 32 || d->out_features % 8) return MOE_FP4_EINVAL;
  if (d->act_fn < MOE_FP4_FN_NONE || d->act_fn > MOE_FP4_FN_RELU2) return MOE_FP4_EINVAL;
  if (d->act_fn == MOE_FP4_FN_SWIGLUOAI &&
      (!std::isfinite(d->act_alpha) || !std::isfinite(d->act_beta) || !(d->act_limit > 0.0f)))
    return MOE_FP4_EINVAL;
  if (d->in_features > moe::kMaxCols || d->out_features > kMaxOutFeatures ||
      (int64_t)d->in_features * d->out_features > (int64_t)1 << 31 || d->max_tokens > kMaxTokens)
    return MOE_FP4_EUNSUPPORTED;
  const bool act = d->act_fn != MOE_FP4_FN_NONE;
  *s = moe::Fp4Shape{d->in_features, d->out_features, act && d->act_fn != MOE_FP4_FN_RELU2,
                     moe::ActParams{act ? d->act_fn : 0, d->act_alpha, d->act_beta, d->act_limit}, act};
  return MOE_FP4_OK;
}

moe_fp4_status linear(const moe_fp4_linear_desc* desc, const void* prepared, const uint16_t* x, const uint8_t* codes,
                      const uint8_t* scales, int32_t M, uint16_t* out, void* workspace, size_t workspace_bytes,
                      void* stream) {
  moe::Fp4Shape s;
  const moe_fp4_status st = linear_shape(desc, &s);
  if (st != MOE_FP4_OK) return st;
  if (M < 0 || M > desc->max_tokens) return MOE_FP4_EINVAL;
  if (M == 0) return MOE_FP4_OK;
  if (!prepared || !(x || (codes && scales)) || !out || !workspace) return MOE_FP4_EINVAL;
  if (!aligned(prepared, 256) || !aligned(x, 16) || !aligned(codes, 16) || !aligned(out, 16) ||
      !aligned(workspace, 256))
    return MOE_FP4_EINVAL;
  const int64_t need = moe::fp4_workspace(s, desc->max_tokens);
  if (overlapping({{x, 2ll * M * s.K}, {codes, (int64_t)M * s.K / 2}, {scales, (int64_t)M * s.K / 32},
                   {prepared, s.prepared_bytes()}},
                  {{out, 2ll * M * s.N}, {workspace, need}}))
    return MOE_FP4_EINVAL;
  if ((int64_t)workspace_bytes < need) return MOE_FP4_EWORKSPACE;
  return from_hip(moe::launch_fp4_linear(s, (const uint8_t*)prepared, x, codes, scales, M, out, (uint8_t*)workspace,
                                         (hipStream_t)stream));
}

moe_fp4_status routes_shape(int32_t tokens, int32_t k, int32_t E) {
  if (tokens < 0 || k <= 0 || E <= 0) return MOE_FP4_EINVAL;
  if ((int64_t)tokens * k > moe::kGroupMaxRoutes || E > moe::kGroupMaxExperts) return MOE_FP4_EUNSUPPORTED;
  return MOE_FP4_OK;
}

moe_fp4_status group_routes(const void* ids, int size, int32_t tokens, int32_t k, int32_t E, int32_t* offsets,
                            int32_t* order, int32_t* place, void* workspace, size_t workspace_bytes, void* stream) {
  const moe_fp4_status st = routes_shape(tokens, k, E);
  if (st != MOE_FP4_OK) return st;
  const int64_t R = (int64_t)tokens * k, need = moe::group_routes_workspace(R, E);
  if (!offsets || !workspace || (R && (!ids || !order || !place))) return MOE_FP4_EINVAL;
  if (!aligned(ids, size) || !aligned(offsets, 4) || !aligned(order, 4) || !aligned(place, 4) ||
      !aligned(workspace, 256))
    return MOE_FP4_EINVAL;
  if (overlapping({{ids, R * size}}, {{offsets, 4ll * (E + 1)}, {order, 4 * R}, {place, 4 * R}, {workspace, need}}))
    return MOE_FP4_EINVAL;
  if ((int64_t)workspace_bytes < need) return MOE_FP4_EWORKSPACE;
  return from_hip(moe::launch_group_routes(ids, size == 8, R, E, offsets, order, place, (uint8_t*)workspace,
                                           (hipStream_t)stream));
}

// Sizes of the calls on rows of routes.
moe_fp4_status rows_shape(int32_t tokens, int32_t k, int32_t hidden) {
  if (tokens < 0 || k <= 0 || hidden <= 0 || hidden % 8) return MOE_FP4_EINVAL;
  if ((int64_t)tokens * k > moe::kGroupMaxRoutes || hidden > 1 << 15) return MOE_FP4_EUNSUPPORTED;
  return MOE_FP4_OK;
}

moe_fp4_status grouped_shape(const moe_fp4_grouped_desc* d, int32_t rows) {
  if (!d || d->num_experts <= 0 || d->in_features <= 0 || d->out_features <= 0 || d->in_features % 8 ||
      d->out_features % 8 || rows < 0)
    return MOE_FP4_EINVAL;
  if (d->weight_layout != MOE_FP4_WEIGHT_OUT_IN && d->weight_layout != MOE_FP4_WEIGHT_IN_OUT) return MOE_FP4_EINVAL;
  if (d->num_experts > moe::kGroupMaxExperts || d->in_features > moe::kMaxCols || d->out_features > moe::kMaxCols ||
      rows > moe::kGroupMaxRoutes)
    return MOE_FP4_EUNSUPPORTED;
  return MOE_FP4_OK;
}

}  // namespace

extern "C" {

moe_fp4_status moe_fp4_quantize_workspace_bytes(int32_t format, int64_t experts, size_t* bytes) {
  if (!format_ok(format) || experts < 0 || !bytes) return MOE_FP4_EINVAL;
  if (experts > kMaxValues) return MOE_FP4_EUNSUPPORTED;
  *bytes = format == MOE_FP4_NVFP4 ? (size_t)experts * moe::kQuantParts * 4 : 0;
  return MOE_FP4_OK;
}

moe_fp4_status moe_fp4_quantize(int32_t format, int32_t type, const void* x, int64_t experts, int64_t rows,
                                int32_t cols, int64_t row_stride, uint8_t* codes, uint8_t* scales,
                                const float* global_scale, float* global_out, void* workspace, size_t workspace_bytes,
                                void* stream) {
  if (!format_ok(format) || !type_ok(type) || experts < 0 || rows < 0 || cols <= 0) return MOE_FP4_EINVAL;
  const bool nv = format == MOE_FP4_NVFP4, f32 = type == MOE_FP4_TYPE_F32;
  const int G = nv ? 16 : 32, size = f32 ? 4 : 2;
  if (cols % G || row_stride < cols || row_stride % (16 / size)) return MOE_FP4_EINVAL;
  if (nv ? (global_scale != nullptr) == (global_out != nullptr) : global_scale || global_out) return MOE_FP4_EINVAL;
  const int64_t n = values(experts, rows, row_stride);
  if (cols > moe::kMaxCols || n < 0) return MOE_FP4_EUNSUPPORTED;
  if (n == 0) return MOE_FP4_OK;
  if (!x || !codes || !scales || !aligned(x, 16) || !aligned(codes, 16) || !aligned(global_scale, 4) ||
      !aligned(global_out, 4))
    return MOE_FP4_EINVAL;
  const int64_t need = global_out ? experts * moe::kQuantParts * 4 : 0;
  if (need && (!workspace || !aligned(workspace, 256))) return MOE_FP4_EINVAL;
  const int64_t held = experts * rows * cols;
  if (overlapping({{x, (n - row_stride + cols) * size}, {global_scale, 4 * experts}},
                  {{codes, held / 2}, {scales, held / G}, {global_out, 4 * experts}, {need ? workspace : nullptr, need}}))
    return MOE_FP4_EINVAL;
  if ((int64_t)workspace_bytes < need) return MOE_FP4_EWORKSPACE;
  moe::QuantArgs a;
  a.x = x;
  a.codes = codes;
  a.scales = scales;
  a.global = global_scale;
  a.g_out = global_out;
  a.partial = global_out ? (uint32_t*)workspace : nullptr;
  a.experts = experts;
  a.rows = rows;
  a.ld = row_stride;
  a.K = cols;
  a.nvfp4 = nv;
  a.f32 = f32;
  return from_hip(moe::launch_fp4_quantize(a, (hipStream_t)stream));
}

moe_fp4_status moe_fp4_dequantize(int32_t format, int32_t type, const uint8_t* codes, const uint8_t* scales,
                                  const float* global_scale, int64_t experts, int64_t rows, int32_t cols, void* out,
                                  void* stream) {
  if (!format_ok(format) || !type_ok(type) || experts < 0 || rows < 0 || cols <= 0) return MOE_FP4_EINVAL;
  const bool nv = format == MOE_FP4_NVFP4, f32 = type == MOE_FP4_TYPE_F32;
  const int G = nv ? 16 : 32;
  if (cols % G || nv != (global_scale != nullptr)) return MOE_FP4_EINVAL;
  const int64_t n = values(experts, rows, cols);
  if (cols > moe::kMaxCols || n < 0) return MOE_FP4_EUNSUPPORTED;
  if (n == 0) return MOE_FP4_OK;
  if (!codes || !scales || !out || !aligned(codes, 16) || !aligned(out, 16) || !aligned(global_scale, 4))
    return MOE_FP4_EINVAL;
  if (overlapping({{codes, n / 2}, {scales, n / G}, {global_scale, 4 * experts}}, {{out, n * (f32 ? 4 : 2)}}))
    return MOE_FP4_EINVAL;
  return from_hip(moe::launch_fp4_dequantize(moe::DequantArgs{codes, scales, global_scale, out, experts, rows, cols, nv, f32},
                                             (hipStream_t)stream));
}

moe_fp4_status moe_fp4_linear_prepared_bytes(const moe_fp4_linear_desc* desc, size_t* bytes) {
  moe::Fp4Shape s;
  const moe_fp4_status st = linear_shape(desc, &s);
  if (st != MOE_FP4_OK) return st;
  if (!bytes) return MOE_FP4_EINVAL;
  *bytes = (size_t)s.prepared_bytes();
  return MOE_FP4_OK;
}

moe_fp4_status moe_fp4_linear_prepare(const moe_fp4_linear_desc* desc, const uint8_t* codes, const uint8_t* scales,
                                      void* prepared, size_t prepared_bytes, void* stream) {
  moe::Fp4Shape s;
  const moe_fp4_status st = linear_shape(desc, &s);
  if (st != MOE_FP4_OK) return st;
  if (!codes || !scales || !prepared || !aligned(codes, 16) || !aligned(prepared, 256)) return MOE_FP4_EINVAL;
  const int64_t n = (int64_t)s.halves() * s.N * s.K;
  if (overlapping({{codes, n / 2}, {scales, n / 32}}, {{prepared, s.prepared_bytes()}})) return MOE_FP4_EINVAL;
  if ((int64_t)prepared_bytes < s.prepared_bytes()) return MOE_FP4_EWORKSPACE;
  return from_hip(moe::launch_fp4_prepare(s, codes, scales, (uint8_t*)prepared, (hipStream_t)stream));
}

moe_fp4_status moe_fp4_linear_workspace_bytes(const moe_fp4_linear_desc* desc, int32_t M, size_t* bytes) {
  moe::Fp4Shape s;
  const moe_fp4_status st = linear_shape(desc, &s);
  if (st != MOE_FP4_OK) return st;
  if (!bytes || M < 0 || M > desc->max_tokens) return MOE_FP4_EINVAL;
  *bytes = (size_t)moe::fp4_workspace(s, desc->max_tokens);
  return MOE_FP4_OK;
}

moe_fp4_status moe_fp4_linear(const moe_fp4_linear_desc* desc, const void* prepared, const uint16_t* x, int32_t M,
                              uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  return linear(desc, prepared, x, nullptr, nullptr, M, out, workspace, workspace_bytes, stream);
}

moe_fp4_status moe_fp4_linear_quantized(const moe_fp4_linear_desc* desc, const void* prepared, const uint8_t* codes,
                                        const uint8_t* scales, int32_t M, uint16_t* out, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  return linear(desc, prepared, nullptr, codes, scales, M, out, workspace, workspace_bytes, stream);
}

moe_fp4_status moe_fp4_group_routes_workspace_bytes(int32_t tokens, int32_t top_k, int32_t num_experts,
                                                    size_t* bytes) {
  const moe_fp4_status st = routes_shape(tokens, top_k, num_experts);
  if (st != MOE_FP4_OK) return st;
  if (!bytes) return MOE_FP4_EINVAL;
  *bytes = (size_t)moe::group_routes_workspace((int64_t)tokens * top_k, num_experts);
  return MOE_FP4_OK;
}

moe_fp4_status moe_fp4_group_routes(const int32_t* topk_ids, int32_t tokens, int32_t top_k, int32_t num_experts,
                                    int32_t* offsets, int32_t* order, int32_t* place, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  return group_routes(topk_ids, 4, tokens, top_k, num_experts, offsets, order, place, workspace, workspace_bytes, stream);
}

moe_fp4_status moe_fp4_group_routes_i64(const int64_t* topk_ids, int32_t tokens, int32_t top_k, int32_t num_experts,
                                        int32_t* offsets, int32_t* order, int32_t* place, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  return group_routes(topk_ids, 8, tokens, top_k, num_experts, offsets, order, place, workspace, workspace_bytes, stream);
}

moe_fp4_status moe_fp4_gather_routes(const uint16_t* x, const int32_t* order, int32_t tokens, int32_t top_k,
                                     int32_t hidden, uint16_t* out, void* stream) {
  const moe_fp4_status st = rows_shape(tokens, top_k, hidden);
  if (st != MOE_FP4_OK) return st;
  if (tokens == 0) return MOE_FP4_OK;
  if (!x || !order || !out || !aligned(x, 16) || !aligned(order, 4) || !aligned(out, 16)) return MOE_FP4_EINVAL;
  const int64_t R = (int64_t)tokens * top_k;
  if (overlapping({{x, 2ll * tokens * hidden}, {order, 4 * R}}, {{out, 2 * R * hidden}})) return MOE_FP4_EINVAL;
  return from_hip(moe::launch_gather_routes(x, order, R, top_k, hidden, out, (hipStream_t)stream));
}

moe_fp4_status moe_fp4_combine_routes(const uint16_t* y, const int32_t* place, const float* w, int32_t tokens,
                                      int32_t top_k, int32_t hidden, uint16_t* out, void* stream) {
  const moe_fp4_status st = rows_shape(tokens, top_k, hidden);
  if (st != MOE_FP4_OK) return st;
  if (tokens == 0) return MOE_FP4_OK;
  if (!y || !place || !out || !aligned(y, 16) || !aligned(place, 4) || !aligned(w, 4) || !aligned(out, 16))
    return MOE_FP4_EINVAL;
  const int64_t R = (int64_t)tokens * top_k;
  if (overlapping({{y, 2 * R * hidden}, {place, 4 * R}, {w, 4 * R}}, {{out, 2ll * tokens * hidden}}))
    return MOE_FP4_EINVAL;
  return from_hip(moe::launch_combine_routes(y, place, w, tokens, top_k, hidden, out, (hipStream_t)stream));
}

moe_fp4_status moe_fp4_combine_routes_grad(const uint16_t* dout, const uint16_t* y, const int32_t* place,
                                           const int32_t* order, const float* w, int32_t tokens, int32_t top_k,
                                           int32_t hidden, uint16_t* dy, float* dw, void* stream) {
  const moe_fp4_status st = rows_shape(tokens, top_k, hidden);
  if (st != MOE_FP4_OK) return st;
  if (tokens == 0) return MOE_FP4_OK;
  if (!dout || !y || !place || !order || !w || !dy || !dw) return MOE_FP4_EINVAL;
  if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(place, 4) || !aligned(order, 4) || !aligned(w, 4) ||
      !aligned(dy, 16) || !aligned(dw, 4))
    return MOE_FP4_EINVAL;
  const int64_t R = (int64_t)tokens * top_k;
  if (overlapping({{dout, 2ll * tokens * hidden}, {y, 2 * R * hidden}, {place, 4 * R}, {order, 4 * R}, {w, 4 * R}},
                  {{dy, 2 * R * hidden}, {dw, 4 * R}}))
    return MOE_FP4_EINVAL;
  return from_hip(moe::launch_combine_routes_grad(dout, y, place, order, w, tokens, top_k, hidden, dy, dw,
                                                  (hipStream_t)stream));
}

moe_fp4_status moe_fp4_grouped_linear(const moe_fp4_grouped_desc* desc, const uint16_t* x, int32_t rows,
                                      const uint16_t* weight, const int32_t* offsets, uint16_t* y, void* stream) {
  const moe_fp4_status st = grouped_shape(desc, rows);
  if (st != MOE_FP4_OK) return st;
  if (rows == 0) return MOE_FP4_OK;
  if (!x || !weight || !offsets || !y) return MOE_FP4_EINVAL;
  if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(offsets, 4) || !aligned(y, 16)) return MOE_FP4_EINVAL;
  const int E = desc->num_experts, K = desc->in_features, N = desc->out_features;
  if (overlapping({{x, 2ll * rows * K}, {weight, 2ll * E * N * K}, {offsets, 4ll * (E + 1)}}, {{y, 2ll * rows * N}}))
    return MOE_FP4_EINVAL;
  const moe::GroupedArgs a{x, weight, offsets, y, rows, E, K, N, desc->weight_layout == MOE_FP4_WEIGHT_IN_OUT};
  return from_hip(moe::launch_grouped(a, (hipStream_t)stream));
}

moe_fp4_status moe_fp4_grouped_weight_grad(const moe_fp4_grouped_desc* desc, int32_t type, const uint16_t* dy,
                                           const uint16_t* x, int32_t rows, const int32_t* offsets, void* dw,
                                           void* stream) {
  const moe_fp4_status st = grouped_shape(desc, rows);
  if (st != MOE_FP4_OK) return st;
  if (!type_ok(type) || desc->weight_layout != MOE_FP4_WEIGHT_OUT_IN) return MOE_FP4_EINVAL;
  if (!offsets || !dw || (rows && (!dy || !x))) return MOE_FP4_EINVAL;
  if (!aligned(x, 16) || !aligned(dy, 16) || !aligned(offsets, 4) || !aligned(dw, 16)) return MOE_FP4_EINVAL;
  const int E = desc->num_experts, K = desc->in_features, N = desc->out_features;
  const bool f32 = type == MOE_FP4_TYPE_F32;
  if (overlapping({{x, 2ll * rows * K}, {dy, 2ll * rows * N}, {offsets, 4ll * (E + 1)}},
                  {{dw, (f32 ? 4ll : 2ll) * E * N * K}}))
    return MOE_FP4_EINVAL;
  const moe::GroupedGradArgs a{dy, x, offsets, dw, rows, E, K, N, f32};
  return from_hip(moe::launch_grouped_weight_grad(a, (hipStream_t)stream));
}

}  // extern "C"
