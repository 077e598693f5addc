// route.hip -- the router: scores, group-limited top-k selection and weights,
// and their gradient, for gfx950.
//
//   p   = sigmoid(z) or softmax(z) over the token's experts
//   key = p + bias; -inf where z is -inf or NaN, or the key is NaN
//   a group's mark = the sum of its group_top largest keys; the topk_groups
//         groups with the largest marks stay, the others' keys become -inf
//   the k largest keys are taken, largest first; ties go to the lowest index
//   w_j = scale p_j, or scale p_j / sum_i p_i over the taken experts
//
// Scores, keys and sums are binary64.  The choice between two experts is a
// comparison of scores that may differ by less than a binary32 rounding, and
// one wrong comparison is a wrong index; at E = 256 the binary64 exponentials
// are a few microseconds of the chip's time at 8192 tokens.
#include "ep_device.h"
#include "moe.h"

#include <type_traits>

namespace ep {
namespace {

constexpr int kRouteWaves = 4;   // tokens per block, one wave each (1 above 1024 experts: the groups' keys in LDS)

__device__ __forceinline__ double shfl_xor_f64(double v, int m) {
    const int2 u = __builtin_bit_cast(int2, v);
    return __builtin_bit_cast(double, int2{__shfl_xor(u.x, m), __shfl_xor(u.y, m)});
}

__device__ __forceinline__ double readlane_f64(double v, int lane) {
    const int2 u = __builtin_bit_cast(int2, v);
    return __builtin_bit_cast(double, int2{__builtin_amdgcn_readlane(u.x, lane), __builtin_amdgcn_readlane(u.y, lane)});
}

__device__ __forceinline__ double wave_sum_f64(double v) {
    for (int m = 1; m < kWave; m <<= 1) v += shfl_xor_f64(v, m);
    return v;
}

__device__ __forceinline__ float wave_max_f32(float v) {
    for (int m = 1; m < kWave; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
    return v;
}

__device__ __forceinline__ float load_logit(const void *z, int64_t i, bool bf16) {
    return bf16 ? u2f((uint32_t) static_cast<const uint16_t *>(z)[i] << 16) : static_cast<const float *>(z)[i];
}

// e^(z - top) with the limit at top = +inf: the experts at +inf share.
__device__ __forceinline__ double exp_below(float z, float top) {
    return z == top ? 1.0 : exp((double)z - (double)top);
}

__device__ __forceinline__ double sigmoid_f64(float z) { return 1.0 / (1.0 + exp(-(double)z)); }

// A binary64 as an unsigned integer of the same order (-0 below +0; the keys
// hold no -0: p >= +0 and p + bias rounds to +0).
__device__ __forceinline__ uint64_t order_bits(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return (u >> 63) ? ~u : (u | (1ull << 63));
}

constexpr uint64_t kNone = 0x000FFFFFFFFFFFFFull;   // order_bits(-inf)

// One wave per token; lane l holds experts l, l + 64, ...: EPL of them.
template <int EPL>
__global__ __launch_bounds__(64 * kRouteWaves) void ep_route_kernel(Router r, const void *logits, const float *bias,
                                                                    int64_t *topk_idx, float *topk_w) {
    extern __shared__ double group_keys[];   // [waves][E] keys, when there are groups
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x / kWave) + threadIdx.x / kWave;
    if (t >= r.T) return;   // wave-uniform; waves share nothing
    const int64_t row = t * r.E;
    const float inf = __builtin_inff();

    float z[EPL];
    float top = -inf;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = i * kWave + lane;
        z[i] = e < r.E ? load_logit(logits, row + e, r.bf16) : -inf;
        if (!(z[i] > -inf)) z[i] = -inf;   // NaN too
        top = fmaxf(top, z[i]);
    }
    double total = 1.0;
    if (r.softmax) {
        top = wave_max_f32(top);
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) s += z[i] == -inf ? 0.0 : exp_below(z[i], top);
        total = wave_sum_f64(s);
    }
    uint64_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = i * kWave + lane;
        key[i] = kNone;
        if (z[i] == -inf) continue;
        double v = r.softmax ? exp_below(z[i], top) / total : sigmoid_f64(z[i]);
        if (bias) v += (double)bias[e];
        if (v == v) key[i] = order_bits(v);
    }

    if (r.G > 1) {
        double *mine = group_keys + (size_t)(threadIdx.x / kWave) * r.E;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = i * kWave + lane;
            const uint64_t u = key[i];
            if (e < r.E) mine[e] = __builtin_bit_cast(double, (u >> 63) ? (u & ~(1ull << 63)) : ~u);
        }
        __builtin_amdgcn_wave_barrier();
        const int per = r.E / r.G;
        double best = -(double)inf, second = -(double)inf;
        if (lane < r.G)
            for (int i = 0; i < per; ++i) {
                const double v = mine[lane * per + i];
                if (v > best) {
                    second = best;
                    best = v;
                } else if (v > second) {
                    second = v;
                }
            }
        double mark = r.gtop == 2 ? best + second : best;
        if (lane >= r.G || !(mark == mark)) mark = -(double)inf;
        int before = 0;   // groups ahead of this lane's: larger, or as large and earlier
        for (int g = 0; g < r.G; ++g) {
            const double other = readlane_f64(mark, g);
            before += (other > mark || (other == mark && g < lane)) ? 1 : 0;
        }
        const uint64_t keep = __ballot(lane < r.G && before < r.Gk);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = i * kWave + lane;
            if (e < r.E && !((keep >> (e / per)) & 1)) key[i] = kNone;
        }
    }

    int taken = -1;   // lane j: the j-th expert
    for (int j = 0; j < r.k; ++j) {
        uint64_t b = kNone;
        int be = r.E;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] > b) {
                b = key[i];
                be = i * kWave + lane;
            }
#pragma unroll
        for (int m = 1; m < kWave; m <<= 1) {
            const uint64_t ob = ((uint64_t)(uint32_t)__shfl_xor((int)(b >> 32), m) << 32) |
                                (uint32_t)__shfl_xor((int)(uint32_t)b, m);
            const int oe = __shfl_xor(be, m);
            if (ob > b || (ob == b && oe < be)) {
                b = ob;
                be = oe;
            }
        }
        if (b <= kNone) break;   // the same in every lane
        if (lane == j) taken = be;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (be == i * kWave + lane) key[i] = kNone;
    }

    // the weights, slot j in lane j
    const float zt = taken >= 0 ? load_logit(logits, row + taken, r.bf16) : -inf;
    const float chosen_top = wave_max_f32(zt);
    double p;
    if (!r.softmax)
        p = taken >= 0 ? sigmoid_f64(zt) : 0.0;
    else if (r.renorm)   // a softmax over the taken experts alone: the common sum cancels
        p = taken >= 0 ? exp_below(zt, chosen_top) : 0.0;
    else
        p = taken >= 0 ? exp_below(zt, top) / total : 0.0;
    if (r.renorm) {
        const double sum = wave_sum_f64(p);
        p = sum > 0.0 ? p / sum : 0.0;
    }
    if (lane < r.k) {
        topk_idx[t * r.k + lane] = taken;
        topk_w[t * r.k + lane] = (float)(p * (double)r.scale);
    }
}

// Gradient of the weights over the logits.  With q_j the share of slot j
// (p_j / sum p) and g_j the weight's gradient times scale:
//   sigmoid           dz_j = g_j p_j (1 - p_j)
//   sigmoid, renorm   dz_j = (g_j - <g, q>) q_j (1 - p_j)
//   softmax           dz_e = p_e (g_e - <g, p>)  for every expert
//   softmax, renorm   dz_j = q_j (g_j - <g, q>), q the softmax over the taken
// Experts that were not taken get 0 but for the plain softmax.  One wave per
// token; the k terms are formed in lanes 0 .. k - 1 and added, slot by slot,
// into the registers of the lane that holds the expert: no atomics, and an
// index that occurs twice counts twice.
template <int EPL>
__global__ __launch_bounds__(64 * kRouteWaves) void ep_route_backward_kernel(Router r, const void *logits,
                                                                             const int64_t *topk_idx,
                                                                             const float *grad_w, void *grad_logits) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x / kWave) + threadIdx.x / kWave;
    if (t >= r.T) return;   // wave-uniform
    const int64_t row = t * r.E;
    const float inf = __builtin_inff();

    int64_t id = lane < r.k ? topk_idx[t * r.k + lane] : -1;
    if (id >= r.E) id = -1;
    const double g = id >= 0 ? (double)grad_w[t * r.k + lane] * (double)r.scale : 0.0;
    float zt = id >= 0 ? load_logit(logits, row + id, r.bf16) : -inf;
    if (!(zt > -inf)) zt = -inf;
    const int taken = (id >= 0 && zt > -inf) ? (int)id : -1;

    float z[EPL];
    float top = -inf;
    double total = 1.0, dz = 0.0, common = 0.0;
    const bool all = r.softmax && !r.renorm;   // every expert gets a gradient
    if (all) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = i * kWave + lane;
            z[i] = e < r.E ? load_logit(logits, row + e, r.bf16) : -inf;
            if (!(z[i] > -inf)) z[i] = -inf;
            top = fmaxf(top, z[i]);
        }
        top = wave_max_f32(top);
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) s += z[i] == -inf ? 0.0 : exp_below(z[i], top);
        total = wave_sum_f64(s);
        const double p = taken >= 0 ? exp_below(zt, top) / total : 0.0;
        dz = g * p;
        common = wave_sum_f64(dz);
    } else if (r.softmax) {
        const float m = wave_max_f32(taken >= 0 ? zt : -inf);
        const double x = taken >= 0 ? exp_below(zt, m) : 0.0;
        const double sum = wave_sum_f64(x);
        const double q = sum > 0.0 ? x / sum : 0.0;
        const double mean = wave_sum_f64(taken >= 0 ? g * q : 0.0);
        dz = taken >= 0 ? q * (g - mean) : 0.0;
    } else {
        // with x = e^-|z|: p = 1 / (1 + x) or x / (1 + x), and 1 - p the other
        const double x = taken >= 0 ? exp(-fabs((double)zt)) : 0.0;
        const double hi = 1.0 / (1.0 + x), lo = x / (1.0 + x);
        const double p = taken >= 0 ? (zt >= 0 ? hi : lo) : 0.0, rest = zt >= 0 ? lo : hi;
        if (r.renorm) {
            const double sum = wave_sum_f64(p);
            const double q = sum > 0.0 ? p / sum : 0.0;
            const double mean = wave_sum_f64(taken >= 0 ? g * q : 0.0);
            dz = taken >= 0 ? (g - mean) * q * rest : 0.0;
        } else {
            dz = taken >= 0 ? g * p * rest : 0.0;
        }
    }

    double out[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) out[i] = (all && z[i] > -inf) ? -common * (exp_below(z[i], top) / total) : 0.0;
    for (int j = 0; j < r.k; ++j) {
        const int e = __builtin_amdgcn_readlane(taken, j);
        if (e < 0) continue;
        const double v = readlane_f64(dz, j);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (e == i * kWave + lane) out[i] += v;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = i * kWave + lane;
        if (e >= r.E) continue;
        if (r.bf16)
            static_cast<uint16_t *>(grad_logits)[row + e] = (uint16_t)f32_to_bf16((float)out[i]);
        else
            static_cast<float *>(grad_logits)[row + e] = (float)out[i];
    }
}

// Calls f with the experts-per-lane constant that holds E experts.
template <typename F>
hipError_t with_epl(int E, F f) {
    if (E <= 64) return f(std::integral_constant<int, 1>());
    if (E <= 128) return f(std::integral_constant<int, 2>());
    if (E <= 256) return f(std::integral_constant<int, 4>());
    if (E <= 512) return f(std::integral_constant<int, 8>());
    if (E <= 1024) return f(std::integral_constant<int, 16>());
    if (E <= 2048) return f(std::integral_constant<int, 32>());
    return f(std::integral_constant<int, 64>());
}

}  // namespace

hipError_t launch_route(const Router &r, const void *logits, const float *bias, int64_t *topk_idx,
                        float *topk_w, hipStream_t stream) {
    const int waves = r.E > 1024 ? 1 : kRouteWaves;
    const size_t lds = r.G > 1 ? sizeof(double) * (size_t)waves * r.E : 0;   // at most 32 KiB
    const dim3 grid((unsigned)((r.T + waves - 1) / waves)), block(kWave * waves);
    return with_epl(r.E, [&](auto epl) {
        hipLaunchKernelGGL(ep_route_kernel<decltype(epl)::value>, grid, block, lds, stream, r, logits, bias, topk_idx,
                           topk_w);
        return hipGetLastError();
    });
}

hipError_t launch_route_backward(const Router &r, const void *logits, const int64_t *topk_idx,
                                 const float *grad_topk_w, void *grad_logits, hipStream_t stream) {
    const dim3 grid((unsigned)((r.T + kRouteWaves - 1) / kRouteWaves)), block(kWave * kRouteWaves);
    return with_epl(r.E, [&](auto epl) {
        hipLaunchKernelGGL(ep_route_backward_kernel<decltype(epl)::value>, grid, block, 0, stream, r, logits, topk_idx,
                           grad_topk_w, grad_logits);
        return hipGetLastError();
    });
}

}  // namespace ep
