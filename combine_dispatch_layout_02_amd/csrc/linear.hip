// linear.hip -- the dense bf16 product with bias, activation, gate and residual
// in its epilogue, and its backward pass, for gfx950:
//
//   z = x w^T + bias,  y = act(z) + residual  (gated: act(z[:, :N]) * z[:, N:] + residual)
//   dz = dy act'(z) ...,  dx = dz w,  dw = dz^T x,  db = sum of dz's rows
//
// All three products are one kernel.  With C[r, c] = sum_k R[r, k] Q[c, k], an
// operand lies in memory either with its k contiguous (x and w in the first, dz
// in the second) or with its r or c contiguous (w in the second, dz and x in the
// third).  Both kinds go to LDS by direct loads of 16 bytes a lane; the first is
// read from there in the matrix instruction's layout, the second through the
// transposing LDS read.  Q is the instruction's first operand, R its second, so
// a lane's 4 results lie at consecutive c.
#include "dense.h"
#include "ep_device.h"
#include "stream_device.h"
#include "tile_device.h"
#include "tile_order.h"

namespace ep {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------- activations

// p = 1 / (1 + e^-z) and 1 - p, each without cancellation.
struct Sigmoid {
    float p, q;
    __device__ __forceinline__ explicit Sigmoid(float z) {
        const float x = expf(-__builtin_fabsf(z)), r = 1.0f / (1.0f + x);
        p = z >= 0.0f ? r : x * r;
        q = z >= 0.0f ? x * r : r;
    }
};
constexpr float kTanhArg = 1.5957691216057308f;    // 2 sqrt(2 / pi): (1 + tanh(a)) / 2 is the sigmoid of 2 a
constexpr float kSqrtHalf = 0.70710678118654752f, kPdf = 0.39894228040143268f;   // 1 / sqrt(2 pi)

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == kActRelu) return z <= 0.0f ? 0.0f : z;
    if constexpr (ACT == kActSilu) return z * Sigmoid(z).p;
    if constexpr (ACT == kActGelu) return 0.5f * z * erfcf(-kSqrtHalf * z);
    if constexpr (ACT == kActGeluTanh) return z * Sigmoid(kTanhArg * (z + 0.044715f * z * z * z)).p;
    return z;
}

// The value and the derivative.
template <int ACT>
__device__ __forceinline__ void derive(float z, float *f, float *d) {
    if constexpr (ACT == kActRelu) {
        *f = z <= 0.0f ? 0.0f : z;
        *d = z > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (ACT == kActSilu) {
        const Sigmoid s(z);
        *f = z * s.p;
        *d = s.p * (1.0f + z * s.q);
    } else if constexpr (ACT == kActGelu) {
        const float cdf = 0.5f * erfcf(-kSqrtHalf * z);
        *f = z * cdf;
        *d = cdf + z * (expf(-0.5f * z * z) * kPdf);
    } else if constexpr (ACT == kActGeluTanh) {
        const Sigmoid s(kTanhArg * (z + 0.044715f * z * z * z));
        *f = z * s.p;
        // past 20 the second term is below binary32's range, and z z may be infinite
        const float slope = kTanhArg * (1.0f + 3 * 0.044715f * z * z);
        *d = s.p + (__builtin_fabsf(z) > 20.0f ? 0.0f : z * (s.p * s.q) * slope);
    } else {
        *f = z;
        *d = 1.0f;
    }
}

// f(std::integral_constant) for the activation, the same for every lane.
template <int V>
struct Const {
    static constexpr int value = V;
};
template <typename F>
__device__ __forceinline__ void with_activation(int act, const F &f) {
    switch (act) {
        case kActRelu: return f(Const<kActRelu>());
        case kActSilu: return f(Const<kActSilu>());
        case kActGelu: return f(Const<kActGelu>());
        case kActGeluTanh: return f(Const<kActGeluTanh>());
        default: return f(Const<kActNone>());
    }
}

// ---------------------------------------------------------------- tiles

// One operand of a product: B rows (of R or Q) by 64 of k a step.
struct Operand {
    const uint16_t *p;
    int64_t rows;     // of R or Q
    int64_t ld;       // elements from one line of memory to the next
    int64_t split;    // gated weights: B / 2 rows from the first half, B / 2 from `split` on; else 0
};

struct Product {
    Operand r, q;
    int64_t k;         // length of the sums
    int64_t part;      // elements from dz's first part to its second (parts 2)
    int parts;         // the sums run over k as often, R from its parts in turn
    int rtiles, ctiles;
    // what becomes of the sums
    int64_t out_ld;
    void *out;
    bool out_f32;
    const float *bias;
    const uint16_t *residual;
    uint16_t *z;
    int act;
    bool gated, linear;   // linear: bias, activation, ... follow
};

// The lane's part in bringing B rows of an operand into LDS, NL loads of 1 KiB
// by each of W waves.
//   k contiguous (T false): LDS rows are operand rows of 64 k, 128 bytes; piece
//     c of 16 bytes lies at c ^ (row % 8), so that 8 rows' pieces touch every
//     bank once.
//   rows contiguous (T true): LDS rows are k, 2 B bytes; pairs of pieces are
//     permuted by k % 4: the transposing read takes 32 bytes of 4 consecutive k.
template <bool T, int B, int W>
struct Loader {
    static constexpr int NL = B * 128 / 1024 / W;
    static_assert(NL >= 1 && NL * W * 1024 == B * 128, "whole loads");
    const uint16_t *base;
    int64_t step;         // elements from one step to the next (T: a step's 64 lines)
    int64_t second;       // elements to the second half of a gated tile
    uint32_t off[NL];
    int kfirst[T ? NL : 1];   // T: the line; else the lane's first k in a step
    __device__ __forceinline__ void init(const Operand &o, int64_t first, int lane, int wid) {
        if constexpr (!T) {
            base = o.p + first * o.ld;
            step = 64;
            second = o.split * o.ld;
            const int row = lane >> 3, piece = (lane & 7) ^ row;
            kfirst[0] = piece * 8;
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int at = (wid * NL + i) * 8 + row;   // LDS row; those past the end repeat the last one
                const int r = o.split > 0 && at >= B / 2 ? at - B / 2 : at;
                const int64_t last = (o.split > 0 ? o.split : o.rows) - 1 - first;
                off[i] = (uint32_t)(min((int64_t)r, last) * o.ld * 2) + piece * 16;
            }
        } else {
            base = o.p + first;
            step = 64 * o.ld;
            second = 0;
            const int last = (int)min((o.rows - first) / 8 - 1, (int64_t)(B / 8 - 1));   // pieces of a line
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int at = (wid * NL + i) * 64 + lane, line = at / (B / 8), slot = at % (B / 8);
                const int piece = min(slot ^ ((line & 3) << 1), last);
                kfirst[i] = line;
                off[i] = (uint32_t)(line * o.ld * 2) + piece * 16;
            }
        }
    }
    // from: the step's first element, left: of the sum's length from there on
    __device__ __forceinline__ void load(uint8_t *lds, int i, int wid, const uint16_t *from, int left) const {
        const rsrc_t b = buffer(!T && (wid * NL + i) * 8 >= B / 2 ? from + second : from);
        const uint32_t past = kfirst[T ? i : 0] < left ? 0u : kPast;
        load_to_lds(b, lds + (wid * NL + i) * 1024, off[i] | past, 0);
    }
};

// A fragment of 16 rows by 32 k of an operand in LDS, in the matrix
// instruction's layout: lane (l % 16: row, l / 16: 8 consecutive k).
template <bool T, int B>
__device__ __forceinline__ bf16x8 fragment(const uint8_t *lds, int row, int chunk, int lane) {
    const int r16 = lane & 15, quad = lane >> 4;
    if constexpr (!T) {
        const int r = row + r16;
        return __builtin_bit_cast(bf16x8, ld16(lds + r * 128 + (((chunk * 4 + quad) ^ (r & 7)) << 4)));
    } else {
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const int k = chunk * 32 + quad * 8 + (r16 >> 2);
        // lane i of 16 names line i / 4 and its columns 4 (i % 4) .. + 3, and gets column i of the 4 lines
        const int col = row + (r16 & 3) * 4, piece = (col >> 3) ^ ((r16 >> 2) << 1);
        const uint8_t *p = lds + k * (2 * B) + piece * 16 + (col & 7) * 2;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * 2 * B));
        return __builtin_bit_cast(bf16x8, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    }
}

__device__ __forceinline__ void store4(void *out, bool f32, int64_t at, const f32x4 &v) {
    if (f32)
        *reinterpret_cast<f32x4 *>(static_cast<float *>(out) + at) = v;
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + at) =
            uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// The last steps of 4 results at row r and columns c .. c + 3 (gated: the gate's
// in v, the factor's in u).
__device__ __forceinline__ void finish4(const Product &p, int64_t r, int64_t c, f32x4 v, f32x4 u) {
    const int64_t at = r * p.out_ld + c;
    if (p.linear) {
        if (p.bias) {
            v += *reinterpret_cast<const f32x4 *>(p.bias + c);
            if (p.gated) u += *reinterpret_cast<const f32x4 *>(p.bias + p.out_ld + c);
        }
        if (p.z) {
            store4(p.z, false, p.gated ? r * 2 * p.out_ld + c : at, v);
            if (p.gated) store4(p.z, false, r * 2 * p.out_ld + p.out_ld + c, u);
        }
        with_activation(p.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = activate<decltype(act)::value>(v[i]);
        });
        if (p.gated) v *= u;
        if (p.residual) {
            const uint2 d = *reinterpret_cast<const uint2 *>(p.residual + at);
            v += f32x4{bf16_lo(d.x), bf16_hi(d.x), bf16_lo(d.y), bf16_hi(d.y)};
        }
    }
    store4(p.out, p.out_f32, at, v);
}

// One block: BR rows by BC columns of C, WR by WC waves; a step is 64 of k.
template <bool TR, bool TQ, int BR, int BC, int WR, int WC>
__global__ __launch_bounds__(64 * WR * WC) void ep_linear_tile_kernel(Product p) {
    constexpr int W = WR * WC, NR = BR / WR / 16, NC = BC / WC / 16;
    static_assert(NC % 2 == 0, "a gate's columns and their factors in one wave");
    __shared__ __attribute__((aligned(16))) uint8_t rbuf0[BR * 128];
    __shared__ __attribute__((aligned(16))) uint8_t qbuf0[BC * 128];
    __shared__ __attribute__((aligned(16))) uint8_t rbuf1[BR * 128];
    __shared__ __attribute__((aligned(16))) uint8_t qbuf1[BC * 128];

    int rt, ct;
    if (!TileOrder{p.rtiles, p.ctiles}.tile(blockIdx.x, &rt, &ct)) return;
    const int lane = threadIdx.x & (kWave - 1), wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wr = wid / WC, wc = wid % WC;
    const int64_t r0 = (int64_t)rt * BR, c0 = (int64_t)ct * (p.gated ? BC / 2 : BC);

    Loader<TR, BR, W> lr;
    Loader<TQ, BC, W> lq;
    lr.init(p.r, r0, lane, wid);
    lq.init(p.q, c0, lane, wid);
    const int steps = (int)((p.k + 63) / 64), all = steps * p.parts;
    const auto stage = [&](uint8_t *rb, uint8_t *qb, int s) {
        const int part = s >= steps ? 1 : 0, kb = s - part * steps;
        const int left = s < all ? (int)min(p.k - (int64_t)kb * 64, (int64_t)64) : 0;
        const uint16_t *rp = lr.base + part * p.part + kb * lr.step, *qp = lq.base + kb * lq.step;
#pragma unroll
        for (int i = 0; i < lr.NL; ++i) lr.load(rb, i, wid, rp, left);
#pragma unroll
        for (int i = 0; i < lq.NL; ++i) lq.load(qb, i, wid, qp, left);
    };
    // LDS rows of the wave's groups of 16 columns: half of them from each half of the tile
    const auto qrow = [&](int f) { return (f / (NC / 2)) * (BC / 2) + wc * (BC / 2 / WC) + f % (NC / 2) * 16; };

    f32x4 acc[NC][NR] = {};
    const auto step = [&](const uint8_t *rb, const uint8_t *qb, uint8_t *rnext, uint8_t *qnext, int s) {
        // this wave's part of the step has arrived; then every wave's, and the other buffers are free
        wait_loads<0>();
        barrier_only();
        stage(rnext, qnext, s + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            bf16x8 b[NR];
#pragma unroll
            for (int m = 0; m < NR; ++m) b[m] = fragment<TR, BR>(rb, wr * (BR / WR) + 16 * m, c, lane);
#pragma unroll
            for (int f = 0; f < NC; ++f) {
                const bf16x8 a = fragment<TQ, BC>(qb, qrow(f), c, lane);
#pragma unroll
                for (int m = 0; m < NR; ++m) acc[f][m] = mfma(a, b[m], acc[f][m]);
            }
        }
    };
    stage(rbuf0, qbuf0, 0);
    for (int s = 0; s < all; s += 2) {
        step(rbuf0, qbuf0, rbuf1, qbuf1, s);
        if (s + 1 < all) step(rbuf1, qbuf1, rbuf0, qbuf0, s + 1);
    }
    wait_loads<0>();

    const int r16 = lane & 15, quad = lane >> 4;
#pragma unroll
    for (int m = 0; m < NR; ++m) {
        const int64_t r = r0 + wr * (BR / WR) + 16 * m + r16;
        if (r >= p.r.rows) continue;
#pragma unroll
        for (int f = 0; f < NC / 2; ++f) {
            const int64_t c = c0 + qrow(f) + 4 * quad, c2 = c + BC / 2;
            if (p.gated) {
                if (c < p.out_ld) finish4(p, r, c, acc[f][m], acc[f + NC / 2][m]);
            } else {
                if (c < p.out_ld) finish4(p, r, c, acc[f][m], f32x4{});
                if (c2 < p.out_ld) finish4(p, r, c2, acc[f + NC / 2][m], f32x4{});
            }
        }
    }
}

template <bool TR, bool TQ, int BR, int BC, int WR, int WC>
hipError_t launch_tile(Product p, hipStream_t stream) {
    const int cols = p.gated ? BC / 2 : BC;
    p.rtiles = (int)((p.r.rows + BR - 1) / BR);
    p.ctiles = (int)((p.out_ld + cols - 1) / cols);
    hipLaunchKernelGGL((ep_linear_tile_kernel<TR, TQ, BR, BC, WR, WC>),
                       dim3((unsigned)TileOrder::blocks(p.rtiles, p.ctiles)), dim3(64 * WR * WC), 0, stream, p);
    return hipGetLastError();
}

template <bool TR, bool TQ>
hipError_t launch_product(const Product &p, hipStream_t stream) {
    return launch_tile<TR, TQ, 64, 64, 2, 2>(p, stream);
}

// ---------------------------------------------------------------- the gradient over z

// dz from dy and z in bf16 (in one part, or in two: the rounded value and its
// rounded rest) and the sums of its columns over runs of kDzRows rows, for the
// bias.  A wave's lanes take 8 columns each, its 4 waves rows in turn.
constexpr int kDzThreads = 256;
template <typename Dy>
__global__ __launch_bounds__(kDzThreads) void ep_linear_dz_kernel(LinearShape s, const Dy *__restrict__ dy,
                                                                  const uint16_t *__restrict__ z,
                                                                  uint16_t *__restrict__ dz, int parts,
                                                                  float *__restrict__ sums) {
    constexpr int W = kDzThreads / kWave;
    __shared__ float part[W][2][8][kWave];
    const int lane = threadIdx.x & (kWave - 1), wid = threadIdx.x / kWave;
    const int cols = (s.N + 511) / 512, ct = blockIdx.x % cols;
    const int64_t run = blockIdx.x / cols;
    const int c = (ct * kWave + lane) * 8, wide = s.wide();
    const int64_t plane = s.M * wide;
    float sum[2][8] = {};
    const auto unpack = [](vec16 v, float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(v[i]), f[2 * i + 1] = bf16_hi(v[i]);
    };
    const auto store = [&](int64_t at, const float (&f)[8]) {
        vec16 hi, lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h[2], l[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float v = f[2 * i + j];
                h[j] = f32_to_bf16(v);
                // of two parts the first stays finite where the value is
                if (parts > 1 && (h[j] & 0x7FFF) == 0x7F80 && v - v == 0.0f) h[j] = f2u(v) >> 16;
                const float rest = v - u2f(h[j] << 16);
                l[j] = (h[j] & 0x7F80) == 0x7F80 ? 0u : f32_to_bf16(rest);
            }
            hi[i] = h[0] | h[1] << 16;
            lo[i] = l[0] | l[1] << 16;
        }
        st16(dz + at, hi);
        if (parts > 1) st16(dz + plane + at, lo);
    };
    if (c < s.N)
        for (int i = wid; i < kDzRows; i += W) {
            const int64_t r = run * kDzRows + i;
            if (r >= s.M) break;
            float g[8], a[8], b[8] = {};
            if constexpr (sizeof(Dy) == 4) {
                const f32x4 lo = *reinterpret_cast<const f32x4 *>(dy + r * s.N + c),
                            hi = *reinterpret_cast<const f32x4 *>(dy + r * s.N + c + 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) g[j] = lo[j], g[4 + j] = hi[j];
            } else {
                unpack(ld16(dy + r * s.N + c), g);
            }
            if (s.act != kActNone || s.gated) {
                float v[8], u[8];
                unpack(ld16(z + r * wide + c), v);
                if (s.gated) unpack(ld16(z + r * wide + s.N + c), u);
                with_activation(s.act, [&](auto act) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float f, d;
                        derive<decltype(act)::value>(v[j], &f, &d);
                        a[j] = s.gated ? g[j] * u[j] * d : g[j] * d;
                        b[j] = g[j] * f;
                    }
                });
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) a[j] = g[j];
            }
            if (parts > 0) {
                store(r * wide + c, a);
                if (s.gated) store(r * wide + s.N + c, b);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[0][j] += a[j], sum[1][j] += b[j];
        }
    if (!sums) return;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j) part[wid][h][j][lane] = sum[h][j];
    __syncthreads();
    if (wid > 1 || (wid == 1 && !s.gated) || c >= s.N) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += part[w][wid][j][lane];
        sums[run * wide + wid * s.N + c + j] = v;
    }
}

// The runs' sums, added in order; with none, 0.
__global__ __launch_bounds__(256) void ep_linear_bias_kernel(const float *__restrict__ sums, int64_t runs, int wide,
                                                             float *__restrict__ out) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= wide) return;
    float v = 0.0f;
    for (int64_t i = 0; i < runs; ++i) v += sums[i * wide + c];
    out[c] = v;
}

__global__ __launch_bounds__(256) void ep_linear_zero_kernel(vec16 *out, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) out[i] = vec16{};
}

}  // namespace

hipError_t launch_linear(const LinearShape &s, const uint16_t *x, const uint16_t *w, const float *bias,
                         const uint16_t *residual, void *y, uint16_t *z, hipStream_t stream) {
    Product p = {};
    p.r = {x, s.M, s.K, 0};
    p.q = {w, s.wide(), s.K, s.gated ? s.N : 0};
    p.k = s.K;
    p.parts = 1;
    p.out_ld = s.N;
    p.out = y;
    p.out_f32 = s.f32;
    p.bias = bias;
    p.residual = residual;
    p.z = z;
    p.act = s.act;
    p.gated = s.gated;
    p.linear = true;
    return launch_product<false, false>(p, stream);
}

hipError_t launch_linear_backward(const LinearShape &s, const void *dy, const uint16_t *x, const uint16_t *w,
                                  const uint16_t *z, uint16_t *grad_x, void *grad_w, float *grad_bias, uint8_t *ws,
                                  hipStream_t stream) {
    const int wide = s.wide();
    if (s.M == 0) {
        if (grad_w) {
            const int64_t n = (int64_t)wide * s.K * (s.w32 ? 4 : 2) / 16;
            hipLaunchKernelGGL(ep_linear_zero_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream,
                               static_cast<vec16 *>(grad_w), n);
        }
        if (grad_bias)
            hipLaunchKernelGGL(ep_linear_bias_kernel, dim3((unsigned)((wide + 255) / 256)), dim3(256), 0, stream,
                               nullptr, 0, wide, grad_bias);
        return hipGetLastError();
    }
    // two parts only for the product that takes them
    const int parts = s.plain() ? 0 : (s.w32 && grad_w ? 2 : 1);
    uint16_t *dz = reinterpret_cast<uint16_t *>(ws);
    float *sums = reinterpret_cast<float *>(ws + linear_sums_offset(s));
    const int64_t runs = (s.M + kDzRows - 1) / kDzRows;
    if (grad_bias || (parts > 0 && (grad_x || grad_w))) {
        const dim3 grid((unsigned)(runs * ((s.N + 511) / 512)));
        if (s.f32)
            hipLaunchKernelGGL(ep_linear_dz_kernel<float>, grid, dim3(kDzThreads), 0, stream, s,
                               static_cast<const float *>(dy), z, dz, parts, grad_bias ? sums : nullptr);
        else
            hipLaunchKernelGGL(ep_linear_dz_kernel<uint16_t>, grid, dim3(kDzThreads), 0, stream, s,
                               static_cast<const uint16_t *>(dy), z, dz, parts, grad_bias ? sums : nullptr);
    }
    if (grad_bias)
        hipLaunchKernelGGL(ep_linear_bias_kernel, dim3((unsigned)((wide + 255) / 256)), dim3(256), 0, stream, sums,
                           runs, wide, grad_bias);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const uint16_t *d = parts > 0 ? dz : static_cast<const uint16_t *>(dy);
    if (grad_x) {
        Product p = {};
        p.r = {d, s.M, wide, 0};
        p.q = {w, s.K, s.K, 0};
        p.k = wide;
        p.parts = 1;
        p.out_ld = s.K;
        p.out = grad_x;
        e = launch_product<false, true>(p, stream);
        if (e != hipSuccess) return e;
    }
    if (grad_w) {
        Product p = {};
        p.r = {d, wide, wide, 0};
        p.q = {x, s.K, s.K, 0};
        p.k = s.M;
        p.parts = parts > 1 ? 2 : 1;
        p.part = s.M * wide;
        p.out_ld = s.K;
        p.out = grad_w;
        p.out_f32 = s.w32;
        e = launch_product<true, true>(p, stream);
    }
    return e;
}

}  // namespace ep
