// dense_abi.hip -- the C ABI of the experts' layer for a few tokens and of the
// matrix product with its backward pass (declared in include/ep.h): argument
// validation on the host, then launches on the caller's stream.  Nothing here
// allocates or synchronizes.
#include "dense.h"
#include "ep.h"

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? EP_OK : EP_EHIP; }

int check_few(const ep_few_shape *s, ep::FewShape *out) {
    static_assert(EP_FEW_TOKENS == ep::kFewTokens, "the limit the kernels assume");
    if (!s) return EP_EINVAL;
    if (s->num_tokens < 0 || s->num_tokens > EP_FEW_TOKENS) return EP_EINVAL;
    if (s->num_experts < 1 || s->num_experts > 4096 || s->num_topk < 1 || s->num_topk > 32) return EP_EINVAL;
    if (s->w_format != EP_FMT_BF16 && s->w_format != EP_FMT_FP8_S128) return EP_EINVAL;
    const int unit = s->w_format == EP_FMT_BF16 ? 8 : 128;
    if (s->hidden < unit || s->hidden % unit != 0 || s->hidden > (1 << 20)) return EP_EINVAL;
    if (s->intermediate < unit || s->intermediate % unit != 0 || s->intermediate > (1 << 20)) return EP_EINVAL;
    if ((int64_t)s->num_tokens * s->num_topk * s->intermediate >= (int64_t(1) << 28)) return EP_EINVAL;
    out->T = s->num_tokens;
    out->H = s->hidden;
    out->I = s->intermediate;
    out->E = s->num_experts;
    out->k = s->num_topk;
    out->f8 = s->w_format == EP_FMT_FP8_S128;
    return EP_OK;
}

int check_linear(const ep_linear_shape *s, ep::LinearShape *out) {
    if (!s) return EP_EINVAL;
    if (s->rows < 0 || s->rows >= (int64_t(1) << 40)) return EP_EINVAL;
    if (s->in_features < 8 || s->in_features % 8 != 0 || s->in_features > (1 << 20)) return EP_EINVAL;
    if (s->out_features < 8 || s->out_features % 8 != 0 || s->out_features > (1 << 20)) return EP_EINVAL;
    if (s->activation < EP_ACT_NONE || s->activation > EP_ACT_GELU_TANH) return EP_EINVAL;
    for (int32_t flag : {s->gated, s->y_f32, s->grad_w_f32})
        if (flag != 0 && flag != 1) return EP_EINVAL;
    out->M = s->rows;
    out->K = s->in_features;
    out->N = s->out_features;
    out->act = s->activation;
    out->gated = s->gated == 1;
    out->f32 = s->y_f32 == 1;
    out->w32 = s->grad_w_f32 == 1;
    const int64_t m = s->rows / 64 + 1, k = out->K / 64 + 1, n = out->wide() / 64 + 1, limit = int64_t(1) << 23;
    return m * k < limit && m * n < limit && n * k < limit ? EP_OK : EP_EINVAL;
}

}  // namespace

extern "C" {

int ep_moe_few_workspace_bytes(const ep_few_shape *shape, size_t *bytes) {
    ep::FewShape s;
    const int rc = check_few(shape, &s);
    if (rc != EP_OK) return rc;
    if (!bytes) return EP_EINVAL;
    *bytes = ep::few_workspace(s);
    return EP_OK;
}

int ep_moe_few(const ep_few_shape *shape, const uint16_t *x, const int64_t *topk_idx, const float *topk_w,
               const void *gate_up, const float *gate_up_scales, const void *down, const float *down_scales,
               const uint16_t *residual, uint16_t *y, void *ws, size_t ws_bytes, void *stream) {
    ep::FewShape s;
    const int rc = check_few(shape, &s);
    if (rc != EP_OK) return rc;
    if (s.T == 0) return EP_OK;
    if (!x || !topk_idx || !topk_w || !gate_up || !down || !y) return EP_EINVAL;
    if (s.f8 ? (!gate_up_scales || !down_scales) : (gate_up_scales || down_scales)) return EP_EINVAL;
    for (const void *p : {(const void *)x, gate_up, down, (const void *)residual, (const void *)y})
        if (!aligned(p, 16)) return EP_EALIGN;
    if (!ws || ws_bytes < ep::few_workspace(s)) return EP_EWORKSPACE;
    if (!aligned(ws, 256)) return EP_EALIGN;
    return hip_status(ep::launch_few(s, x, topk_idx, topk_w, gate_up, gate_up_scales, down, down_scales, residual, y,
                                     static_cast<uint8_t *>(ws), static_cast<hipStream_t>(stream)));
}

int ep_linear(const ep_linear_shape *shape, const uint16_t *x, const uint16_t *w, const float *bias,
              const uint16_t *residual, void *y, uint16_t *z, void *stream) {
    ep::LinearShape s;
    const int rc = check_linear(shape, &s);
    if (rc != EP_OK) return rc;
    if (s.M == 0) return EP_OK;
    if (!x || !w || !y) return EP_EINVAL;
    for (const void *p : {(const void *)x, (const void *)w, (const void *)bias, (const void *)residual, (const void *)y,
                          (const void *)z})
        if (!aligned(p, 16)) return EP_EALIGN;
    return hip_status(ep::launch_linear(s, x, w, bias, residual, y, z, static_cast<hipStream_t>(stream)));
}

int ep_linear_backward_workspace_bytes(const ep_linear_shape *shape, size_t *bytes) {
    ep::LinearShape s;
    const int rc = check_linear(shape, &s);
    if (rc != EP_OK) return rc;
    if (!bytes) return EP_EINVAL;
    *bytes = ep::linear_workspace(s);
    return EP_OK;
}

int ep_linear_backward(const ep_linear_shape *shape, const void *dy, const uint16_t *x, const uint16_t *w,
                       const uint16_t *z, uint16_t *grad_x, void *grad_w, float *grad_bias, void *ws,
                       size_t ws_bytes, void *stream) {
    ep::LinearShape s;
    const int rc = check_linear(shape, &s);
    if (rc != EP_OK) return rc;
    const bool kept = s.act != ep::kActNone || s.gated;
    if (s.M > 0) {
        if (!dy || (kept && !z) || (grad_x && !w) || (grad_w && !x)) return EP_EINVAL;
        if (!ws || ws_bytes < ep::linear_workspace(s)) return EP_EWORKSPACE;
    }
    for (const void *p : {dy, (const void *)x, (const void *)w, (const void *)z, (const void *)grad_x,
                          (const void *)grad_w})
        if (!aligned(p, 16)) return EP_EALIGN;
    if (!aligned(ws, 256)) return EP_EALIGN;
    return hip_status(ep::launch_linear_backward(s, dy, x, w, kept ? z : nullptr, grad_x, grad_w, grad_bias,
                                                 static_cast<uint8_t *>(ws), static_cast<hipStream_t>(stream)));
}

}  // extern "C"
