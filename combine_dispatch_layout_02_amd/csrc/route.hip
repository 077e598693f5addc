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
// one wrong comparison is a wrong index.
#include "ep_device.h"
#include "moe.h"

#include <type_traits>

namespace ep {
namespace {

constexpr int kRouteWaves = 4;   // tokens per block, one wave each (1 above 1024 experts: the groups' keys in LDS)

__device__ __forceinline__ double readlane_f64(double v, int lane) {
    const int2 u = __builtin_bit_cast(int2, v);
    return __builtin_bit_cast(double, int2{__builtin_amdgcn_readlane(u.x, lane), __builtin_amdgcn_readlane(u.y, lane)});
}

// The value of the lane that a DPP control names, `none` where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp(int none, int v) {
    return __builtin_amdgcn_update_dpp(none, v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_f64(double v) {
    const int2 u = __builtin_bit_cast(int2, v);
    return __builtin_bit_cast(double, int2{dpp<CTRL, ROWS>(0, u.x), dpp<CTRL, ROWS>(0, u.y)});
}

// Reductions over the wave, returned to every lane: inside rows of 16 lanes by
// shifts, then the rows' results carried on, the last lane's value read back.
// Register moves only; a reduction through LDS shuffles takes five times as long.
__device__ __forceinline__ double wave_sum_f64(double v) {
    v += dpp_f64<0x111, 0xf>(v);
    v += dpp_f64<0x112, 0xf>(v);
    v += dpp_f64<0x114, 0xf>(v);
    v += dpp_f64<0x118, 0xf>(v);
    v += dpp_f64<0x142, 0xa>(v);
    v += dpp_f64<0x143, 0xc>(v);
    return readlane_f64(v, kWave - 1);
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = max(v, (uint32_t)dpp<0x111, 0xf>(0, (int)v));
    v = max(v, (uint32_t)dpp<0x112, 0xf>(0, (int)v));
    v = max(v, (uint32_t)dpp<0x114, 0xf>(0, (int)v));
    v = max(v, (uint32_t)dpp<0x118, 0xf>(0, (int)v));
    v = max(v, (uint32_t)dpp<0x142, 0xa>(0, (int)v));
    v = max(v, (uint32_t)dpp<0x143, 0xc>(0, (int)v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1);
}

// Largest of values without NaN, through unsigned integers of the same order.
__device__ __forceinline__ float wave_max_f32(float v) {
    const uint32_t u = f2u(v);
    const uint32_t m = wave_max_u32((u >> 31) ? ~u : (u | 0x80000000u));
    return u2f((m >> 31) ? (m & 0x7FFFFFFFu) : ~m);
}

__device__ __forceinline__ float load_logit(const void *z, int64_t i, bool bf16) {
    return bf16 ? u2f((uint32_t) static_cast<const uint16_t *>(z)[i] << 16) : static_cast<const float *>(z)[i];
}

// binary64 -> bf16 in one rounding: what binary32 cannot hold becomes an odd last
// bit of it (to odd, towards zero), 16 bits below bf16's, so the second rounding
// sees on which side of a middle the value lies.
__device__ __forceinline__ uint32_t f64_to_bf16(double v) {
    const float f = (float)v;
    uint32_t u = f2u(f);
    if ((double)f != v && v == v) u = (u - (fabs((double)f) > fabs(v) ? 1u : 0u)) | 1u;
    return f32_to_bf16(u2f(u));
}

// e^(z - top) with the limit at top = +inf: the experts at +inf share.
__device__ __forceinline__ double exp_below(float z, float top) {
    return z == top ? 1.0 : exp((double)z - (double)top);
}

// e^-z leaves binary64 near z = -710, e^z only near -745; 1 + e^z is 1 there.
__device__ __forceinline__ double sigmoid_f64(float z) {
    const bool low = z < -700.0f;
    const double x = exp((double)(low ? z : -z));
    return low ? x : 1.0 / (1.0 + x);
}

// Below this the taken scores may be subnormal and their shares inexact; a score
// then is e^z times the same factor for all of them (for a sigmoid 1, as 1 + e^z
// is 1), and the shares come from the exponentials over the largest of them.
constexpr double kVanishing = 0x1p-960;

// A binary64 as an unsigned integer of the same order (-0 below +0; the keys
// hold no -0: p >= +0 and p + bias rounds to +0).
__device__ __forceinline__ uint64_t order_bits(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return (u >> 63) ? ~u : (u | (1ull << 63));
}

constexpr uint64_t kNone = 0x000FFFFFFFFFFFFFull;   // order_bits(-inf)

__device__ __forceinline__ double order_value(uint64_t u) {
    return __builtin_bit_cast(double, (u >> 63) ? (u & ~(1ull << 63)) : ~u);
}

// The two largest of two pairs (best >= second each).
__device__ __forceinline__ void merge_two(double &best, double &second, double b, double s) {
    const double low = best < b ? best : b;
    second = second < s ? s : second;
    second = second < low ? low : second;
    best = best < b ? b : best;
}

// Logits of experts lane * EPL ... of a row; -inf past the last and for NaN.
// vec: rows and base are aligned for loads of 4 elements.
template <int EPL>
__device__ __forceinline__ void load_logits(const void *logits, int64_t row, int E, bool bf16, bool vec, int lane,
                                            float (&z)[EPL]) {
    const float inf = __builtin_inff();
    const int e0 = lane * EPL;
    if (EPL >= 4 && vec) {
#pragma unroll
        for (int i = 0; i < EPL; i += 4) {
            const int e = e0 + i;
            float v[4] = {-inf, -inf, -inf, -inf};
            if (e < E) {   // E % 4 == 0: all four or none
                if (bf16) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(logits) + row + e);
                    v[0] = bf16_lo(u.x);
                    v[1] = bf16_hi(u.x);
                    v[2] = bf16_lo(u.y);
                    v[3] = bf16_hi(u.y);
                } else {
                    const vec16 u = ld16(static_cast<const float *>(logits) + row + e);
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = u2f(u[q]);
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (i + q < EPL) z[i + q] = v[q];
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) z[i] = e0 + i < E ? load_logit(logits, row + e0 + i, bf16) : -inf;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (!(z[i] > -inf)) z[i] = -inf;
}

// One wave per token; lane l holds experts l EPL ... l EPL + EPL - 1, so that
// the lowest lane, then the lowest place, is the lowest index.  What bounds a
// small batch is the chain of dependent steps in a wave, so the reductions are
// register moves: the largest upper halves of the keys by a maximum over the
// wave, ties by the lower halves, the first lane of those left by a ballot.
// One token, 256 experts in 8 groups: a call every 5.4 us on the GPU; with the
// reductions through LDS shuffles and the groups scanned from LDS 11.7.  8192
// tokens (8.4 MB of logits): 16 us against 26, where the binary64 exponentials
// and the k rounds of selection, some 8 waves on each SIMD, are what it costs.
template <int EPL>
__global__ __launch_bounds__(64 * kRouteWaves) void ep_route_kernel(Router r, const void *logits, const float *bias,
                                                                    int64_t *topk_idx, float *topk_w, bool vec) {
    constexpr bool KEEP = EPL <= 16;         // scores stay in registers for the weights
    extern __shared__ double group_keys[];   // [waves][E] keys, for groups that lanes do not split evenly
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x / kWave) + threadIdx.x / kWave;
    if (t >= r.T) return;   // wave-uniform; waves share nothing
    const int64_t row = t * r.E;
    const float inf = __builtin_inff();

    float z[EPL];
    load_logits(logits, row, r.E, r.bf16, vec, lane, z);
    float top = -inf;
    double total = 1.0;
    double p[KEEP ? EPL : 1];   // sigmoid, or e^(z - top)
    if (r.softmax) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) top = fmaxf(top, z[i]);
        top = wave_max_f32(top);
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const double v = z[i] == -inf ? 0.0 : exp_below(z[i], top);
            if (KEEP) p[KEEP ? i : 0] = v;
            s += v;
        }
        total = wave_sum_f64(s);
    }
    uint64_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane * EPL + i;
        double v;
        if (r.softmax)
            v = (KEEP ? p[KEEP ? i : 0] : exp_below(z[i], top)) / total;
        else
            v = sigmoid_f64(z[i]);
        if (KEEP && !r.softmax) p[KEEP ? i : 0] = v;
        if (bias && e < r.E) v += (double)bias[e];
        key[i] = (z[i] == -inf || !(v == v)) ? kNone : order_bits(v);
    }

    if (r.G > 1) {
        const int per = r.E / r.G, span = per / EPL;   // experts and lanes of a group
        double best = -(double)inf, second = -(double)inf;
        const bool even = per % EPL == 0 && (span & (span - 1)) == 0 && span <= 16;
        int home;          // a lane that holds group `lane`'s mark
        if (even) {        // groups are runs of 1, 2, 4, 8 or 16 lanes
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const double v = order_value(key[i]);
                second = v > best ? best : (v > second ? v : second);
                best = v > best ? v : best;
            }
            if (span > 1) merge_two(best, second, dpp_f64<0xB1, 0xf>(best), dpp_f64<0xB1, 0xf>(second));    // lane ^ 1
            if (span > 2) merge_two(best, second, dpp_f64<0x4E, 0xf>(best), dpp_f64<0x4E, 0xf>(second));    // lane ^ 2
            if (span > 4) merge_two(best, second, dpp_f64<0x141, 0xf>(best), dpp_f64<0x141, 0xf>(second));  // 8 reversed
            if (span > 8) merge_two(best, second, dpp_f64<0x140, 0xf>(best), dpp_f64<0x140, 0xf>(second));  // 16 reversed
            home = span;
        } else {
            double *mine = group_keys + (size_t)(threadIdx.x / kWave) * r.E;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (lane * EPL + i < r.E) mine[lane * EPL + i] = order_value(key[i]);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the wave's own keys: LDS keeps their order
            __builtin_amdgcn_wave_barrier();
            if (lane < r.G)
                for (int i = 0; i < per; ++i) {
                    const double v = mine[lane * per + i];
                    second = v > best ? best : (v > second ? v : second);
                    best = v > best ? v : best;
                }
            home = 1;
        }
        double mark = r.gtop == 2 ? best + second : best;
        if (!(mark == mark)) mark = -(double)inf;
        // this lane's group, and the groups ahead of it: larger, or as large and earlier
        const int mine = lane / home;
        int before = 0;
        for (int g = 0; g < r.G; ++g) {
            const double other = readlane_f64(mark, g * home);
            before += (other > mark || (other == mark && g < mine)) ? 1 : 0;
        }
        const bool kept = mine < r.G && before < r.Gk;
        if (even) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (!kept) key[i] = kNone;
        } else {
            const uint64_t keep = __ballot(kept);   // bit g: group g
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = lane * EPL + i;
                if (e < r.E && !((keep >> (e / per)) & 1)) key[i] = kNone;
            }
        }
    }

    int taken = -1;           // lane j: the j-th expert
    double score = 0.0;       // and its p
    for (int j = 0; j < r.k; ++j) {
        uint64_t b = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < EPL; ++i)
            if (key[i] > b) {
                b = key[i];
                at = i;
            }
        const uint32_t hi = wave_max_u32((uint32_t)(b >> 32));
        if (hi == (uint32_t)(kNone >> 32)) break;   // nothing is left (no number but -inf has these bits)
        uint64_t first = __ballot((uint32_t)(b >> 32) == hi);
        if (first & (first - 1)) {   // several: the largest lower half, then the first lane
            const uint32_t lo = wave_max_u32((uint32_t)(b >> 32) == hi ? (uint32_t)b : 0u);
            first &= __ballot((uint32_t)b == lo);
        }
        const int winner = __builtin_ctzll(first);
        const int place = __builtin_amdgcn_readlane(at, winner);
        if (KEEP) {
            double mine = p[0];
#pragma unroll
            for (int i = 1; i < EPL; ++i)
                if (at == i) mine = p[KEEP ? i : 0];
            const double v = readlane_f64(mine, winner);
            if (lane == j) score = v;
        }
        if (lane == j) taken = winner * EPL + place;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (lane == winner && i == place) key[i] = kNone;
    }

    // the weights, slot j in lane j
    if (!KEEP && taken >= 0) {
        const float zt = load_logit(logits, row + taken, r.bf16);
        score = r.softmax ? exp_below(zt, top) : sigmoid_f64(zt);
    }
    double weight = r.softmax ? score / total : score;
    if (r.renorm) {   // the softmax's common sum cancels
        double sum = wave_sum_f64(score);
        if (sum < kVanishing && (r.softmax || sum > 0.0)) {   // shares of e^z
            const float zt = taken >= 0 ? load_logit(logits, row + taken, r.bf16) : -inf;
            const float m = wave_max_f32(zt);
            score = taken >= 0 ? exp_below(zt, m) : 0.0;
            sum = wave_sum_f64(score);
        }
        weight = sum > 0.0 ? score / sum : 0.0;
    }
    if (taken < 0) weight = 0.0;
    if (lane < r.k) {
        topk_idx[t * r.k + lane] = taken;
        topk_w[t * r.k + lane] = (float)(weight * (double)r.scale);
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
            double part = p, sum = wave_sum_f64(p);
            if (sum > 0.0 && sum < kVanishing) {   // shares of e^z, as in the forward pass
                const float m = wave_max_f32(taken >= 0 ? zt : -inf);
                part = taken >= 0 ? exp_below(zt, m) : 0.0;
                sum = wave_sum_f64(part);
            }
            const double q = sum > 0.0 ? part / sum : 0.0;
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
            static_cast<uint16_t *>(grad_logits)[row + e] = (uint16_t)f64_to_bf16(out[i]);
        else
            static_cast<float *>(grad_logits)[row + e] = (float)out[i];
    }
}

// Waves of a block, a token each.  A launch holds fewer than 2^32 threads, so
// the last batches below 2^26 tokens do not fill up blocks of 4.
int token_waves(const Router &r, int most) { return r.T > (int64_t(1) << 26) - kRouteWaves ? 1 : most; }

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
    const int waves = token_waves(r, r.E > 1024 ? 1 : kRouteWaves);
    const bool vec = r.E % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15u) == 0;
    const size_t lds = r.G > 1 ? sizeof(double) * (size_t)waves * r.E : 0;   // at most 32 KiB
    const dim3 grid((unsigned)((r.T + waves - 1) / waves)), block(kWave * waves);
    return with_epl(r.E, [&](auto epl) {
        hipLaunchKernelGGL(ep_route_kernel<decltype(epl)::value>, grid, block, lds, stream, r, logits, bias, topk_idx,
                           topk_w, vec);
        return hipGetLastError();
    });
}

hipError_t launch_route_backward(const Router &r, const void *logits, const int64_t *topk_idx,
                                 const float *grad_topk_w, void *grad_logits, hipStream_t stream) {
    const int waves = token_waves(r, kRouteWaves);
    const dim3 grid((unsigned)((r.T + waves - 1) / waves)), block(kWave * waves);
    return with_epl(r.E, [&](auto epl) {
        hipLaunchKernelGGL(ep_route_backward_kernel<decltype(epl)::value>, grid, block, 0, stream, r, logits, topk_idx,
                           grad_topk_w, grad_logits);
        return hipGetLastError();
    });
}

}  // namespace ep
