// combine_grad.hip -- backward pass of the token-major bf16 combine (gfx950).
//
//   grad_expert_out[slot[t,j], h] = bf16_rne(w[t,j] dy[t,h])
//   grad_topk_w[t,j]              = sum_h dy[t,h] expert_out[slot[t,j], h]
//
// One pass: a block takes one token, reads dy[t] and the token's k expert rows
// and writes k gradient rows.  bf16 products are exact in binary32; the sums
// are binary32, per lane, then across the wave, then across the waves, in an
// order that the batch and hidden sizes alone fix.
//
// Bound by memory: 2 (T + 2 V) H bytes for V pairs, as many read as written.
// kBatch slots of kVecs vectors each are loaded together, so that a lane has 8
// loads in flight; dy comes back from the cache for the next slots.  At T =
// 4096, H = 7168, top-8 (998 MB) 192 us, 5.2 TB/s, 0.91 of what a large copy
// reaches on this card (5.7); with 256 threads a token 196 us, with 16 loads in
// flight 195 to 203, plain stores 209, plain loads 211, one slot at a time 217.
#include "ep_device.h"
#include "moe.h"

#include <type_traits>

namespace ep {
namespace {

constexpr int kBatch = 4, kVecs = 2;

// Sum over the wave, in lane 63.
__device__ __forceinline__ float wave_sum_f32(float v) {
    const auto add = [](float x, auto ctrl, auto rows) {
        return x + u2f((uint32_t)__builtin_amdgcn_update_dpp(0, (int)f2u(x), decltype(ctrl)::value,
                                                             decltype(rows)::value, 0xf, false));
    };
    typedef std::integral_constant<int, 0xf> all;
    v = add(v, std::integral_constant<int, 0x111>(), all());
    v = add(v, std::integral_constant<int, 0x112>(), all());
    v = add(v, std::integral_constant<int, 0x114>(), all());
    v = add(v, std::integral_constant<int, 0x118>(), all());
    v = add(v, std::integral_constant<int, 0x142>(), std::integral_constant<int, 0xa>());
    return add(v, std::integral_constant<int, 0x143>(), std::integral_constant<int, 0xc>());
}

template <int kGradThreads>
__global__ __launch_bounds__(kGradThreads) void ep_combine_backward_kernel(
    int64_t T, int H, int k, int64_t rows, const uint16_t *dy, const uint16_t *expert_out, const int32_t *token_slot,
    const float *topk_w, uint16_t *grad_out, float *grad_w) {
    constexpr int kGradWaves = kGradThreads / kWave;
    __shared__ float part[32][kGradWaves];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wid = tid / kWave;
    const int nv = H / 8;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const uint16_t *d = dy + t * H;
        for (int j0 = 0; j0 < k; j0 += kBatch) {
            int64_t s[kBatch];
            float w[kBatch], acc[kBatch] = {};
            bool live[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {   // the same in every lane
                const int64_t at = t * k + min(j0 + j, k - 1);
                s[j] = __builtin_amdgcn_readfirstlane(token_slot[at]);
                w[j] = u2f((uint32_t)__builtin_amdgcn_readfirstlane((int)f2u(topk_w[at])));
                live[j] = j0 + j < k && s[j] >= 0 && s[j] < rows;
                if (!live[j]) s[j] = 0;   // read (there is a row 0), not used
            }
            for (int v0 = tid; v0 < nv; v0 += kGradThreads * kVecs) {
                vec16 x[kVecs], o[kBatch][kVecs];
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    const int v = min(v0 + i * kGradThreads, nv - 1);
                    x[i] = ld16(d + 8 * v);
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) o[j][i] = ld16_nt(expert_out + s[j] * H + 8 * v);
                }
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    if (!live[j]) continue;
#pragma unroll
                    for (int i = 0; i < kVecs; ++i) {
                        const int v = v0 + i * kGradThreads;
                        if (v >= nv) continue;
                        float f[8];
                        uint32_t g[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            acc[j] = __builtin_fmaf(bf16_lo(x[i][q]), bf16_lo(o[j][i][q]), acc[j]);
                            acc[j] = __builtin_fmaf(bf16_hi(x[i][q]), bf16_hi(o[j][i][q]), acc[j]);
                            f[2 * q] = w[j] * bf16_lo(x[i][q]);
                            f[2 * q + 1] = w[j] * bf16_hi(x[i][q]);
                        }
                        pack_bf16(f, g);
                        st16_nt(grad_out + s[j] * H + 8 * v, vec16{g[0], g[1], g[2], g[3]});
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const float sum = wave_sum_f32(acc[j]);
                if (lane == kWave - 1 && j0 + j < k) part[j0 + j][wid] = sum;
            }
        }
        __syncthreads();
        if (tid < k) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kGradWaves; ++i) sum += part[tid][i];
            grad_w[t * k + tid] = sum;
        }
        __syncthreads();
    }
}

}  // namespace

hipError_t launch_combine_backward(const Shape &s, const uint16_t *dy, const uint16_t *expert_out,
                                   const int32_t *token_slot, const float *topk_w,
                                   uint16_t *grad_expert_out, float *grad_topk_w, hipStream_t stream) {
    // one wave a token where that gives waves enough, else four (a row's loads
    // are then fewer trips to memory one after the other)
    const dim3 grid((unsigned)(s.T < (1 << 20) ? s.T : (1 << 20)));
    if (s.T >= 1024)
        hipLaunchKernelGGL(ep_combine_backward_kernel<64>, grid, dim3(64), 0, stream, s.T, s.H, s.k, s.rows(), dy,
                           expert_out, token_slot, topk_w, grad_expert_out, grad_topk_w);
    else
        hipLaunchKernelGGL(ep_combine_backward_kernel<256>, grid, dim3(256), 0, stream, s.T, s.H, s.k, s.rows(), dy,
                           expert_out, token_slot, topk_w, grad_expert_out, grad_topk_w);
    return hipGetLastError();
}

}  // namespace ep
