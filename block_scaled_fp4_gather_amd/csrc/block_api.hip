// C-ABI of the operators around the expert layer (declared in
// include/moe_fp4.h): argument checks, sizing and the launches.  Every check
// runs before any HIP call.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/moe_fp4.h"
#include "block.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

moe_fp4_status from_hip(hipError_t e) { return e == hipSuccess ? MOE_FP4_OK : MOE_FP4_EHIP; }

// Largest max_tokens of the router and the FP8 map.
constexpr int kMaxTokens = 1 << 20;

// Largest out_features of the FP8 map: the few tokens' kernel takes 16 rows a
// workgroup of 256 threads (K up to 512; N is smaller for larger ones), gate
// and up twice N, and a launch has fewer than 2^32 threads.
constexpr int kMaxOutFeatures = 1 << 26;

// Whether [p, p + n) and [q, q + m) share a byte.
bool overlap(const void* p, int64_t n, const void* q, int64_t m) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return p && q && a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}

moe_fp4_status router_shape(const moe_fp4_router_desc* d, moe::RouterShape* s) {
  if (!d) return MOE_FP4_EINVAL;
  if (d->num_experts <= 0 || d->hidden <= 0 || d->hidden % 8 || d->top_k <= 0 || d->max_tokens < 0)
    return MOE_FP4_EINVAL;
  if (d->weight_type != MOE_FP4_TYPE_BF16 && d->weight_type != MOE_FP4_TYPE_F32) return MOE_FP4_EINVAL;
  if (d->scoring != MOE_FP4_SCORE_SOFTMAX && d->scoring != MOE_FP4_SCORE_SIGMOID) return MOE_FP4_EINVAL;
  if (d->num_groups < 1 || d->num_experts % d->num_groups) return MOE_FP4_EINVAL;
  if (d->num_groups > 1 && d->num_experts / d->num_groups < 2) return MOE_FP4_EINVAL;
  if (d->top_groups < 1 || d->top_groups > d->num_groups) return MOE_FP4_EINVAL;
  if (d->top_k > d->num_experts / d->num_groups * d->top_groups) return MOE_FP4_EINVAL;
  if (d->renormalize != 0 && d->renormalize != 1) return MOE_FP4_EINVAL;
  if (!std::isfinite(d->scale)) return MOE_FP4_EINVAL;
  if (d->num_experts > moe::kRouterMaxExperts || d->top_k > moe::kRouterMaxTopK ||
      d->num_groups > moe::kRouterMaxGroups || d->hidden > 65536 || d->max_tokens > kMaxTokens)
    return MOE_FP4_EUNSUPPORTED;
  *s = moe::RouterShape{d->num_experts,
                        d->hidden,
                        d->top_k,
                        d->num_groups,
                        d->top_groups,
                        d->weight_type == MOE_FP4_TYPE_F32 ? 3 : 1,
                        d->scoring == MOE_FP4_SCORE_SIGMOID,
                        d->renormalize != 0,
                        d->scale};
  return MOE_FP4_OK;
}

moe_fp4_status fp8_shape(const moe_fp4_fp8_desc* d, moe::Fp8Shape* s) {
  if (!d) return MOE_FP4_EINVAL;
  if (d->in_features <= 0 || d->out_features <= 0 || d->max_tokens < 0) return MOE_FP4_EINVAL;
  if (d->in_features % 8 || d->out_features % 8) return MOE_FP4_EINVAL;
  if (d->act_fn < MOE_FP4_FN_NONE || d->act_fn > MOE_FP4_FN_RELU2) return MOE_FP4_EINVAL;
  if (d->act_fn == MOE_FP4_FN_SWIGLUOAI &&
      (!std::isfinite(d->act_alpha) || !std::isfinite(d->act_beta) || !(d->act_limit > 0.0f)))
    return MOE_FP4_EINVAL;
  if (d->in_features > 1 << 20 || d->out_features > kMaxOutFeatures ||
      (int64_t)d->in_features * d->out_features > (int64_t)1 << 30 || d->max_tokens > kMaxTokens)
    return MOE_FP4_EUNSUPPORTED;
  const bool act = d->act_fn != MOE_FP4_FN_NONE;
  *s = moe::Fp8Shape{d->in_features, d->out_features, act && d->act_fn != MOE_FP4_FN_RELU2,
                     moe::ActParams{act ? d->act_fn : 0, d->act_alpha, d->act_beta, d->act_limit}, act};
  return MOE_FP4_OK;
}

}  // namespace

extern "C" {

moe_fp4_status moe_fp4_router_prepared_bytes(const moe_fp4_router_desc* desc, size_t* bytes) {
  moe::RouterShape s;
  const moe_fp4_status st = router_shape(desc, &s);
  if (st != MOE_FP4_OK) return st;
  if (!bytes) return MOE_FP4_EINVAL;
  *bytes = (size_t)s.prepared_bytes();
  return MOE_FP4_OK;
}

moe_fp4_status moe_fp4_router_prepare(const moe_fp4_router_desc* desc, const void* weight, void* prepared,
                                      size_t prepared_bytes, void* stream) {
  moe::RouterShape s;
  const moe_fp4_status st = router_shape(desc, &s);
  if (st != MOE_FP4_OK) return st;
  if (!weight || !prepared || !aligned(weight, 16) || !aligned(prepared, 256)) return MOE_FP4_EINVAL;
  if ((int64_t)prepared_bytes < s.prepared_bytes()) return MOE_FP4_EWORKSPACE;
  if (overlap(weight, (s.planes == 3 ? 4ll : 2ll) * s.E * s.H, prepared, s.prepared_bytes())) return MOE_FP4_EINVAL;
  return from_hip(moe::launch_router_prepare(s, weight, (uint8_t*)prepared, (hipStream_t)stream));
}

moe_fp4_status moe_fp4_router_workspace_bytes(const moe_fp4_router_desc* desc, int32_t M, size_t* bytes) {
  moe::RouterShape s;
  const moe_fp4_status st = router_shape(desc, &s);
  if (st != MOE_FP4_OK) return st;
  if (!bytes || M < 0 || M > desc->max_tokens) return MOE_FP4_EINVAL;
  *bytes = (size_t)moe::router_workspace(s, desc->max_tokens);
  return MOE_FP4_OK;
}

moe_fp4_status moe_fp4_route(const moe_fp4_router_desc* desc, const void* prepared, const uint16_t* x, int32_t M,
                             const float* bias, int32_t* topk_ids, float* topk_w, float* logits, void* workspace,
                             size_t workspace_bytes, void* stream) {
  moe::RouterShape s;
  const moe_fp4_status st = router_shape(desc, &s);
  if (st != MOE_FP4_OK) return st;
  if (M < 0 || M > desc->max_tokens) return MOE_FP4_EINVAL;
  if (M == 0) return MOE_FP4_OK;
  if (!prepared || !x || !topk_ids || !topk_w || !workspace) return MOE_FP4_EINVAL;
  if (!aligned(prepared, 256) || !aligned(x, 16) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) ||
      !aligned(bias, 4) || !aligned(logits, 4) || !aligned(workspace, 256))
    return MOE_FP4_EINVAL;
  const int64_t need = moe::router_workspace(s, desc->max_tokens);
  const struct {
    const void* p;
    int64_t bytes;
  } in[] = {{x, 2ll * M * s.H}, {bias, 4ll * s.E}, {prepared, s.prepared_bytes()}, {workspace, need}},
    out[] = {{topk_ids, 4ll * M * s.k}, {topk_w, 4ll * M * s.k}, {logits, 4ll * M * s.E}};
  for (int i = 0; i < 3; ++i)
    if (overlap(in[i].p, in[i].bytes, workspace, need)) return MOE_FP4_EINVAL;
  for (int o = 0; o < 3; ++o) {
    for (const auto& i : in)
      if (overlap(out[o].p, out[o].bytes, i.p, i.bytes)) return MOE_FP4_EINVAL;
    for (int q = 0; q < o; ++q)
      if (overlap(out[o].p, out[o].bytes, out[q].p, out[q].bytes)) return MOE_FP4_EINVAL;
  }
  if ((int64_t)workspace_bytes < need) return MOE_FP4_EWORKSPACE;
  return from_hip(moe::launch_route(s, (const uint8_t*)prepared, x, M, bias, topk_ids, topk_w, logits,
                                    (uint8_t*)workspace, (hipStream_t)stream));
}

moe_fp4_status moe_fp4_fp8_prepared_bytes(const moe_fp4_fp8_desc* desc, size_t* bytes) {
  moe::Fp8Shape s;
  const moe_fp4_status st = fp8_shape(desc, &s);
  if (st != MOE_FP4_OK) return st;
  if (!bytes) return MOE_FP4_EINVAL;
  *bytes = (size_t)s.prepared_bytes();
  return MOE_FP4_OK;
}

moe_fp4_status moe_fp4_fp8_prepare(const moe_fp4_fp8_desc* desc, const uint8_t* codes, const float* scales,
                                   void* prepared, size_t prepared_bytes, void* stream) {
  moe::Fp8Shape s;
  const moe_fp4_status st = fp8_shape(desc, &s);
  if (st != MOE_FP4_OK) return st;
  if (!codes || !scales || !prepared || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(prepared, 256))
    return MOE_FP4_EINVAL;
  if ((int64_t)prepared_bytes < s.prepared_bytes()) return MOE_FP4_EWORKSPACE;
  const int64_t nb = (s.N + 127) / 128;
  if (overlap(codes, (int64_t)s.halves() * s.N * s.K, prepared, s.prepared_bytes()) ||
      overlap(scales, 4 * s.halves() * nb * s.kblocks(), prepared, s.prepared_bytes()))
    return MOE_FP4_EINVAL;
  return from_hip(moe::launch_fp8_prepare(s, codes, scales, (uint8_t*)prepared, (hipStream_t)stream));
}

moe_fp4_status moe_fp4_fp8_workspace_bytes(const moe_fp4_fp8_desc* desc, int32_t M, size_t* bytes) {
  moe::Fp8Shape s;
  const moe_fp4_status st = fp8_shape(desc, &s);
  if (st != MOE_FP4_OK) return st;
  if (!bytes || M < 0 || M > desc->max_tokens) return MOE_FP4_EINVAL;
  *bytes = (size_t)moe::fp8_workspace(s, desc->max_tokens);
  return MOE_FP4_OK;
}

moe_fp4_status moe_fp4_fp8_linear(const moe_fp4_fp8_desc* desc, const void* prepared, const uint16_t* x, int32_t M,
                                  uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  moe::Fp8Shape s;
  const moe_fp4_status st = fp8_shape(desc, &s);
  if (st != MOE_FP4_OK) return st;
  if (M < 0 || M > desc->max_tokens) return MOE_FP4_EINVAL;
  if (M == 0) return MOE_FP4_OK;
  if (!prepared || !x || !out || !workspace) return MOE_FP4_EINVAL;
  if (!aligned(prepared, 256) || !aligned(x, 16) || !aligned(out, 16) || !aligned(workspace, 256))
    return MOE_FP4_EINVAL;
  const int64_t need = moe::fp8_workspace(s, desc->max_tokens), out_bytes = 2ll * M * s.N;
  if (overlap(out, out_bytes, x, 2ll * M * s.K) || overlap(out, out_bytes, prepared, s.prepared_bytes()) ||
      overlap(out, out_bytes, workspace, need) || overlap(x, 2ll * M * s.K, workspace, need) ||
      overlap(prepared, s.prepared_bytes(), workspace, need))
    return MOE_FP4_EINVAL;
  if ((int64_t)workspace_bytes < need) return MOE_FP4_EWORKSPACE;
  return from_hip(moe::launch_fp8_linear(s, (const uint8_t*)prepared, x, M, out, (uint8_t*)workspace,
                                         (hipStream_t)stream));
}

moe_fp4_status moe_fp4_block_norm(const moe_fp4_norm_desc* desc, int32_t M, const void* h, const uint16_t* y,
                                  const uint16_t* y2, const void* gate, const void* post_weight,
                                  const void* pre_weight, void* h_out, uint16_t* x_out, void* stream) {
  if (!desc) return MOE_FP4_EINVAL;
  const moe_fp4_norm_desc& d = *desc;
  if (d.hidden <= 0 || d.hidden % 8 || M < 0) return MOE_FP4_EINVAL;
  if (d.residual_type != MOE_FP4_TYPE_BF16 && d.residual_type != MOE_FP4_TYPE_F32) return MOE_FP4_EINVAL;
  if (d.weight_type != MOE_FP4_TYPE_BF16 && d.weight_type != MOE_FP4_TYPE_F32) return MOE_FP4_EINVAL;
  if (d.gate < MOE_FP4_GATE_NONE || d.gate > MOE_FP4_GATE_FULL) return MOE_FP4_EINVAL;
  if (d.gate_sigmoid != 0 && d.gate_sigmoid != 1) return MOE_FP4_EINVAL;
  if (!(d.eps >= 0.0f) || !std::isfinite(d.eps) || !std::isfinite(d.residual_scale) ||
      !std::isfinite(d.branch_scale) || !std::isfinite(d.weight_offset))
    return MOE_FP4_EINVAL;
  if (d.hidden > moe::kNormMaxHidden) return MOE_FP4_EUNSUPPORTED;
  if (M == 0) return MOE_FP4_OK;
  // a branch writes a residual; a norm has its weight and its output; there
  // is something to do
  if (!h || (y != nullptr) != (h_out != nullptr) || (pre_weight != nullptr) != (x_out != nullptr))
    return MOE_FP4_EINVAL;
  if (!y && (y2 || post_weight || d.gate != MOE_FP4_GATE_NONE)) return MOE_FP4_EINVAL;
  if (!y && !x_out) return MOE_FP4_EINVAL;
  if ((d.gate != MOE_FP4_GATE_NONE) != (gate != nullptr)) return MOE_FP4_EINVAL;
  const uintptr_t gate_align = d.gate == MOE_FP4_GATE_TOKEN ? (d.weight_type == MOE_FP4_TYPE_F32 ? 4 : 2) : 16;
  if (!aligned(h, 16) || !aligned(y, 16) || !aligned(y2, 16) || !aligned(gate, gate_align) ||
      !aligned(post_weight, 16) || !aligned(pre_weight, 16) || !aligned(h_out, 16) || !aligned(x_out, 16))
    return MOE_FP4_EINVAL;
  // h, y and y2 are read, a row whole, before it is written, so an output may
  // take their place row for row (same address and type); the gate and the
  // norms' weights are read in between
  const int64_t rb = d.residual_type == MOE_FP4_TYPE_F32 ? 4 : 2, wb = d.weight_type == MOE_FP4_TYPE_F32 ? 4 : 2;
  const int64_t n = (int64_t)M * d.hidden;
  const int64_t gate_n = d.gate == MOE_FP4_GATE_FULL ? n : d.gate == MOE_FP4_GATE_TOKEN ? M : d.hidden;
  const struct {
    const void* p;
    int64_t bytes, size;
  } in[] = {{h, n * rb, rb}, {y, n * 2, 2}, {y2, n * 2, 2}, {gate, gate_n * wb, 0},
            {post_weight, d.hidden * wb, 0}, {pre_weight, d.hidden * wb, 0}},
    out[] = {{h_out, n * rb, rb}, {x_out, n * 2, 2}};
  for (const auto& o : out)
    for (const auto& i : in)
      if (overlap(o.p, o.bytes, i.p, i.bytes) && !(o.p == i.p && o.size == i.size)) return MOE_FP4_EINVAL;
  if (overlap(h_out, n * rb, x_out, n * 2)) return MOE_FP4_EINVAL;
  moe::NormArgs a;
  a.h = h;
  a.y = y;
  a.y2 = y2;
  a.gate = gate;
  a.post_w = post_weight;
  a.pre_w = pre_weight;
  a.h_out = h_out;
  a.x_out = x_out;
  a.M = M;
  a.H = d.hidden;
  a.gate_row = d.gate == MOE_FP4_GATE_FULL ? d.hidden : 0;
  a.gate_vector = d.gate == MOE_FP4_GATE_CHANNEL || d.gate == MOE_FP4_GATE_FULL;
  a.gate_sigmoid = d.gate_sigmoid != 0;
  a.h_f32 = d.residual_type == MOE_FP4_TYPE_F32;
  a.w_f32 = d.weight_type == MOE_FP4_TYPE_F32;
  a.eps = d.eps;
  a.residual_scale = d.residual_scale;
  a.branch_scale = d.branch_scale;
  a.weight_offset = d.weight_offset;
  return from_hip(moe::launch_block_norm(a, (hipStream_t)stream));
}

}  // extern "C"
