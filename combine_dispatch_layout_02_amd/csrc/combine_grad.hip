// combine_grad.hip -- backward pass of the token-major bf16 combine (gfx950).
//
//   grad_expert_out[slot[t,j], h] = bf16_rne(w[t,j] dy[t,h])
//   grad_topk_w[t,j]              = sum_h dy[t,h] expert_out[slot[t,j], h]
//
// One block per token: it reads dy[t] and the token's k expert rows and writes
// k gradient rows, each once.  bf16 products are exact in binary32; the sums
// are binary32, per lane, then across the wave, then across the waves, in an
// order that the hidden size alone fixes.
#include "ep_device.h"
#include "moe.h"

namespace ep {
namespace {

constexpr int kGradThreads = 256;

__device__ __forceinline__ float wave_sum_f32(float v) {
    for (int m = 1; m < kWave; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

__global__ __launch_bounds__(kGradThreads) void ep_combine_backward_kernel(
    int H, int k, int64_t rows, const uint16_t *dy, const uint16_t *expert_out, const int32_t *token_slot,
    const float *topk_w, uint16_t *grad_out, float *grad_w) {
    __shared__ float part[32][kGradThreads / kWave];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wid = tid / kWave;
    for (int j = 0; j < k; ++j) {
        const int64_t s = token_slot[t * k + j];
        float acc = 0.0f;
        if (s >= 0 && s < rows) {
            const float w = topk_w[t * k + j];
            for (int h = tid * 8; h < H; h += kGradThreads * 8) {
                const vec16 d = ld16(dy + t * H + h), o = ld16(expert_out + s * H + h);
                vec16 g;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    acc = __builtin_fmaf(bf16_lo(d[q]), bf16_lo(o[q]), acc);
                    acc = __builtin_fmaf(bf16_hi(d[q]), bf16_hi(o[q]), acc);
                    g[q] = pack_bf16x2(w * bf16_lo(d[q]), w * bf16_hi(d[q]));
                }
                st16(grad_out + s * H + h, g);
            }
        }
        acc = wave_sum_f32(acc);
        if (lane == 0) part[j][wid] = acc;
    }
    __syncthreads();
    if (tid < k) {
        float sum = 0.0f;
        for (int i = 0; i < kGradThreads / kWave; ++i) sum += part[tid][i];
        grad_w[t * k + tid] = sum;
    }
}

}  // namespace

hipError_t launch_combine_backward(const Shape &s, const uint16_t *dy, const uint16_t *expert_out,
                                   const int32_t *token_slot, const float *topk_w,
                                   uint16_t *grad_expert_out, float *grad_topk_w, hipStream_t stream) {
    hipLaunchKernelGGL(ep_combine_backward_kernel, dim3((unsigned)s.T), dim3(kGradThreads), 0, stream, s.H, s.k,
                       s.rows(), dy, expert_out, token_slot, topk_w, grad_expert_out, grad_topk_w);
    return hipGetLastError();
}

}  // namespace ep
