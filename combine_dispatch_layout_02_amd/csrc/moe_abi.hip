// moe_abi.hip -- the C ABI of the router, the experts' products and the
// combine's backward pass (declared in include/ep.h): argument validation on
// the host, then one kernel launch on the caller's stream.  Nothing here
// allocates or synchronizes.
#include "ep.h"
#include "moe.h"

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? EP_OK : EP_EHIP; }

int check_router(const ep_router *r, int64_t T, ep::Router *out) {
    if (!r) return EP_EINVAL;
    if (r->num_experts < 1 || r->num_experts > 4096) return EP_EINVAL;
    if (r->num_topk < 1 || r->num_topk > 32 || r->num_topk > r->num_experts) return EP_EINVAL;
    if (T < 0 || T >= (int64_t(1) << 26) || T * (int64_t)r->num_topk >= (int64_t(1) << 31)) return EP_EINVAL;
    if (r->score != EP_SCORE_SOFTMAX && r->score != EP_SCORE_SIGMOID) return EP_EINVAL;
    if (r->num_groups < 1 || r->num_groups > 64 || r->num_experts % r->num_groups != 0) return EP_EINVAL;
    if (r->topk_groups < 1 || r->topk_groups > r->num_groups) return EP_EINVAL;
    const int per = r->num_experts / r->num_groups;
    if (r->group_top < 1 || r->group_top > 2 || (r->num_groups > 1 && r->group_top > per)) return EP_EINVAL;
    if ((int64_t)r->topk_groups * per < r->num_topk) return EP_EINVAL;
    if (r->renormalize != 0 && r->renormalize != 1) return EP_EINVAL;
    if (r->logits_bf16 != 0 && r->logits_bf16 != 1) return EP_EINVAL;
    if (!(r->scale - r->scale == 0.0f)) return EP_EINVAL;   // finite
    out->T = T;
    out->E = r->num_experts;
    out->k = r->num_topk;
    out->softmax = r->score == EP_SCORE_SOFTMAX;
    out->G = r->num_groups;
    out->Gk = r->topk_groups;
    out->gtop = r->group_top;
    out->renorm = r->renormalize == 1;
    out->bf16 = r->logits_bf16 == 1;
    out->scale = r->scale;
    return EP_OK;
}

int check_expert(const ep_expert_shape *s, bool gated, ep::ExpertShape *out) {
    if (!s) return EP_EINVAL;
    if (s->rows < 0 || s->rows >= (int64_t(1) << 30)) return EP_EINVAL;
    if (s->num_experts < 1 || s->num_experts > 4096) return EP_EINVAL;
    if (s->in_features < 128 || s->in_features % 128 != 0) return EP_EINVAL;
    if (s->out_features < 8 || s->out_features % (gated ? 128 : 8) != 0) return EP_EINVAL;
    if (s->in_features > (1 << 20) || s->out_features > (1 << 20)) return EP_EINVAL;
    if (s->rank_capacity < 0) return EP_EINVAL;
    if (s->num_ranks < 1 || s->num_ranks > 64 || s->num_experts % s->num_ranks != 0) return EP_EINVAL;
    if (s->rank_capacity > 0 && (int64_t)s->num_ranks * s->rank_capacity != s->rows) return EP_EINVAL;
    out->rows = s->rows;
    out->E = s->num_experts;
    out->K = s->in_features;
    out->N = s->out_features;
    out->R = s->num_ranks;
    out->M = s->rank_capacity;
    return ep::expert_grid_fits(*out, gated) ? EP_OK : EP_EINVAL;
}

int check_expert_inputs(const int32_t *offset, const void *a, const float *as, const void *w, const float *ws) {
    if (!offset || !a || !as || !w || !ws) return EP_EINVAL;
    return (aligned(a, 16) && aligned(w, 16)) ? EP_OK : EP_EALIGN;
}

}  // namespace

extern "C" {

int ep_route(const ep_router *router, int64_t num_tokens, const void *logits, const float *bias,
             int64_t *topk_idx, float *topk_w, void *stream) {
    ep::Router r;
    const int rc = check_router(router, num_tokens, &r);
    if (rc != EP_OK) return rc;
    if (r.T == 0) return EP_OK;
    if (!logits || !topk_idx || !topk_w) return EP_EINVAL;
    return hip_status(ep::launch_route(r, logits, bias, topk_idx, topk_w, static_cast<hipStream_t>(stream)));
}

int ep_route_backward(const ep_router *router, int64_t num_tokens, const void *logits, const int64_t *topk_idx,
                      const float *grad_topk_w, void *grad_logits, void *stream) {
    ep::Router r;
    const int rc = check_router(router, num_tokens, &r);
    if (rc != EP_OK) return rc;
    if (r.T == 0) return EP_OK;
    if (!logits || !topk_idx || !grad_topk_w || !grad_logits) return EP_EINVAL;
    return hip_status(ep::launch_route_backward(r, logits, topk_idx, grad_topk_w, grad_logits,
                                                static_cast<hipStream_t>(stream)));
}

int ep_expert_gemm(const ep_expert_shape *shape, const int32_t *expert_offset, const uint8_t *a,
                   const float *a_scales, const uint8_t *w, const float *w_scales, uint16_t *out, void *stream) {
    ep::ExpertShape s;
    int rc = check_expert(shape, false, &s);
    if (rc != EP_OK) return rc;
    if (s.rows == 0) return EP_OK;
    rc = check_expert_inputs(expert_offset, a, a_scales, w, w_scales);
    if (rc != EP_OK) return rc;
    if (!out) return EP_EINVAL;
    if (!aligned(out, 16)) return EP_EALIGN;
    return hip_status(ep::launch_expert_gemm(s, expert_offset, a, a_scales, w, w_scales, out,
                                             static_cast<hipStream_t>(stream)));
}

int ep_expert_gated(const ep_expert_shape *shape, const int32_t *expert_offset, const uint8_t *a,
                    const float *a_scales, const uint8_t *w, const float *w_scales, uint8_t *out_q,
                    float *out_scales, void *stream) {
    ep::ExpertShape s;
    int rc = check_expert(shape, true, &s);
    if (rc != EP_OK) return rc;
    if (s.rows == 0) return EP_OK;
    rc = check_expert_inputs(expert_offset, a, a_scales, w, w_scales);
    if (rc != EP_OK) return rc;
    if (!out_q || !out_scales) return EP_EINVAL;
    if (!aligned(out_q, 16)) return EP_EALIGN;
    return hip_status(ep::launch_expert_gated(s, expert_offset, a, a_scales, w, w_scales, out_q, out_scales,
                                              static_cast<hipStream_t>(stream)));
}

int ep_combine_backward(const ep_shape *shape, const uint16_t *dy, const uint16_t *expert_out,
                        const int32_t *token_slot, const float *topk_w, uint16_t *grad_expert_out,
                        float *grad_topk_w, void *stream) {
    const int rc = ep_validate_shape(shape);
    if (rc != EP_OK) return rc;
    if (shape->y_format != EP_FMT_BF16) return EP_EINVAL;
    if (shape->num_tokens == 0) return EP_OK;
    ep::Shape s;
    s.T = shape->num_tokens;
    s.H = shape->hidden;
    s.E = shape->num_experts;
    s.R = shape->num_ranks;
    s.N = shape->num_nodes;
    s.k = shape->num_topk;
    s.x_fmt = shape->x_format;
    s.y_fmt = shape->y_format;
    s.M = shape->rank_capacity;
    s.rank_rows = shape->rank_rows;
    if (!dy || !expert_out || !token_slot || !topk_w || !grad_expert_out || !grad_topk_w) return EP_EINVAL;
    if (!aligned(dy, 16) || !aligned(expert_out, 16) || !aligned(grad_expert_out, 16)) return EP_EALIGN;
    return hip_status(ep::launch_combine_backward(s, dy, expert_out, token_slot, topk_w, grad_expert_out,
                                                  grad_topk_w, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
