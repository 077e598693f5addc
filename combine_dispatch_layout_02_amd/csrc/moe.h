// moe.h -- launcher interface between the C ABI (moe_abi.hip) and the kernels
// of the router, the experts' products and the combine's backward pass.  Not
// installed; callers use include/ep.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_internal.h"

namespace ep {

struct Router {
    int64_t T;
    int E, k;
    bool softmax;       // else sigmoid
    int G, Gk, gtop;    // groups, groups kept, scores summed for a group's score
    bool renorm;
    bool bf16;          // logits (and their gradient) are bf16, else fp32
    float scale;
};

hipError_t launch_route(const Router &r, const void *logits, const float *bias, int64_t *topk_idx,
                        float *topk_w, hipStream_t stream);
hipError_t launch_route_backward(const Router &r, const void *logits, const int64_t *topk_idx,
                                 const float *grad_topk_w, void *grad_logits, hipStream_t stream);

hipError_t launch_combine_backward(const Shape &s, const uint16_t *dy, const uint16_t *expert_out,
                                   const int32_t *token_slot, const float *topk_w,
                                   uint16_t *grad_expert_out, float *grad_topk_w, hipStream_t stream);

// The experts' block-scaled products.  Expert e's rows of a (and of the
// output) are [offset[e], offset[e + 1]), or, with M > 0, lie in the block of
// the expert's rank (RANK_MAJOR).
struct ExpertShape {
    int64_t rows;
    int E, K, N;   // gated: N is the width of the result, the weights have 2 N rows
    int R, M;
};

// The grid a product uses, from the shape alone (fits: the launch limits hold).
bool expert_grid_fits(const ExpertShape &s, bool gated);

hipError_t launch_expert_gemm(const ExpertShape &s, const int32_t *offset, const uint8_t *a, const float *as,
                              const uint8_t *w, const float *ws, uint16_t *out, hipStream_t stream);
hipError_t launch_expert_gated(const ExpertShape &s, const int32_t *offset, const uint8_t *a, const float *as,
                               const uint8_t *w, const float *ws, uint8_t *q, float *qs, hipStream_t stream);

}  // namespace ep
