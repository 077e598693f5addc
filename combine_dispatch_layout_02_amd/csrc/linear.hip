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
//
// Measured: 4096 rows 7168 -> 2 x 2048 with a gate 195-205 us, 1.2 PFLOP/s, the
// matrix unit busy for 0.59 of a CU's busy cycles, no bank conflicts; without the loads
// into LDS it would take 154, without the reads from LDS 180: what is left is the
// issue of both beside the products, and the epilogue, during which a CU with one
// block multiplies nothing (2048 -> 7168 with a residual: 124-142 us for half the
// products, 0.48).  The gradients of the first: 203 and 198 us, 1.2 PFLOP/s, 0.7.
#include <type_traits>

#include "dense.h"
#include "ep_device.h"
#include "stream_device.h"
#include "tile_device.h"

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

// The lower tail.  From kTail down e^z, or its like, nears binary32's smallest
// normal numbers and leaves them, but a factor (a gate's, a gradient) can bring the
// product back: silu(-96) is 2e-40, of which 3e-4 was lost, and of silu(-103) a
// quarter, before 1e20 multiplied it.  So there act(z) is f y^2 and act'(z) d y^2, and
// the factor is multiplied in between the two y, which are normal numbers down to z
// = -174, -18.6 and -13.0 (below, act(z) u is under 2^-116 for any u).
template <int ACT>
constexpr float kTail = ACT == kActSilu ? -80.0f : ACT == kActGelu ? -12.0f : ACT == kActGeluTanh ? -9.7f : 0.0f;
template <int ACT>
struct Tail {
    float y, f, d;
    __device__ __forceinline__ explicit Tail(float z) {
        if constexpr (ACT == kActGelu) {
            // erfc by its asymptotic series (Abramowitz and Stegun 7.1.23): the first
            // term left out is 945 / z^10, 1.5e-8
            const float r = __builtin_amdgcn_rcpf(z), w = r * r;
            const float s = kPdf * (1.0f - w * (1.0f - w * (3.0f - w * (15.0f - w * 105.0f))));
            y = expf(-0.25f * z * z);
            f = -s;
            d = kPdf * z - s * r;
        } else if constexpr (ACT == kActGeluTanh) {
            y = expf(0.5f * (kTanhArg * (z + 0.044715f * z * z * z)));
            f = z;
            const float near = fmaxf(z, -20.0f);   // y is 0 from there on
            d = 1.0f + near * (kTanhArg * (1.0f + 3 * 0.044715f * near * near));
        } else {
            y = expf(0.5f * z);
            f = z;
            d = 1.0f + z;
        }
    }
    __device__ __forceinline__ float value(float u) const { return f * y * u * y; }
    // dy u act'(z); dy u may leave binary32 above
    __device__ __forceinline__ float slope(float dy, float u) const {
        const float s = dy * u;
        return __builtin_isfinite(s) ? s * y * d * y : dy * y * (u * y) * d;
    }
};
// Whether a lane of the wave has one of its 8 values there: the others' time is one
// comparison of their least.
template <int ACT>
__device__ __forceinline__ bool any_in_tail(const float (&z)[8]) {
    if constexpr (kTail<ACT> == 0.0f) return false;
    float least = z[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) least = fminf(least, z[i]);
    return __ballot(least < kTail<ACT>) != 0;
}
// z[i] becomes act(z[i]) u[i], or act(z[i]).
template <int ACT, bool GATED>
__device__ __forceinline__ void activate8(float (&z)[8], const float (&u)[8]) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = GATED ? activate<ACT>(z[i]) * u[i] : activate<ACT>(z[i]);
    if (any_in_tail<ACT>(z)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (z[i] < kTail<ACT>) v[i] = Tail<ACT>(z[i]).value(GATED ? u[i] : 1.0f);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = v[i];
}

// f(std::integral_constant) for the activation, the same for every lane.
template <int V>
struct Const {
    static constexpr int value = V;
};
template <typename F>
__host__ __device__ __forceinline__ void with_activation(int act, const F &f) {
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
    int64_t part;      // elements from one part of dz to the next
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

// The lane's part in bringing B rows by KS of k of an operand into LDS, NL loads
// of 1 KiB by each of W waves, and in reading it from there.
//   k contiguous (T false): LDS rows are operand rows, 128 (KS = 64) or 64 bytes.
//     Their 16-byte pieces are permuted by the row (`place`), so that the 16
//     lanes that one cycle of a 16-byte LDS read serves (0-3, 12-15, 20-27, and
//     the others of 32) touch every bank once.
//   rows contiguous (T true): LDS rows are lines of k, 2 B bytes.  The transposing
//     read takes 32 bytes of 4 lines for 16 lanes, and of 8 lines for 32: those go
//     to 8 different loads (`line`), whose places lie 32 bytes off each other.
template <bool T, int B, int W, int KS>
struct Side {
    static constexpr int NL = B * KS * 2 / 1024 / W, BLOCKS = NL * W, PIECES = KS / 8;
    static_assert(NL >= 1 && BLOCKS * 1024 == B * KS * 2, "whole loads");
    static constexpr int LINE = 2 * B, PLACE = T ? 1056 : 1024, BYTES = BLOCKS * PLACE;
    const uint16_t *base;
    int64_t step;         // elements from one step to the next (T: a step's KS lines)
    int64_t second;       // elements to the second half of a gated tile
    uint32_t off[NL];
    int kfirst[T ? NL : 1];   // T: the line; else the lane's first k in a step
    uint32_t from;            // the lane's part of a fragment's place in LDS

    static __device__ __forceinline__ int place(int row) { return KS == 64 ? row & 7 : (4 - (row >> 2)) & 3; }
    // The line in place s (s % BLOCKS: the load, s / BLOCKS: where in it): 0-3, 8-11, 4-7, 12-15, 16-19, ...
    static __device__ __forceinline__ int line(int s) { return (s & 0x33) | (s & 4) << 1 | (s & 8) >> 1; }
    static __host__ __device__ constexpr int line_at(int s) { return s % BLOCKS * PLACE + s / BLOCKS * LINE; }

    // first: the tile's first row, row: the wave's first row in the tile
    __device__ __forceinline__ void init(const Operand &o, int64_t first, int row, int lane, int wid) {
        const int r16 = lane & 15, quad = lane >> 4;
        if constexpr (!T) {
            base = o.p + first * o.ld;
            step = KS;
            second = o.split * o.ld;
            const int lr = lane / PIECES, piece = (lane % PIECES) ^ place(lr);
            kfirst[0] = piece * 8;
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int at = (wid * NL + i) * (64 / PIECES) + lr;   // LDS row; those past the end repeat the last one
                const int r = o.split > 0 && at >= B / 2 ? at - B / 2 : at;
                const int64_t last = (o.split > 0 ? o.split : o.rows) - 1 - first;
                off[i] = (uint32_t)(min((int64_t)r, last) * o.ld * 2) + piece * 16;
            }
            from = (uint32_t)((row + r16) * (KS * 2) + ((quad ^ place(r16)) << 4));
        } else {
            base = o.p + first;
            step = KS * o.ld;
            second = 0;
            const int last = (int)min((o.rows - first) / 8 - 1, (int64_t)(B / 8 - 1));   // pieces of a line
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                kfirst[i] = line(wid * NL + i + lane * 16 / LINE * BLOCKS);
                off[i] = (uint32_t)(kfirst[i] * o.ld * 2) + min(lane * 16 % LINE / 16, last) * 16;
            }
            // lane i of 16 names line i / 4 and its columns 4 (i % 4) .. + 3, and gets column i of the 4 lines
            const int s = (r16 >> 2) + 4 * (quad & 1);
            from = (uint32_t)(line_at(s) + (quad >> 1) * line_at(16) + (row + (r16 & 3) * 4) * 2);
        }
    }
    // from: the step's first element, left: of the sum's length from there on
    __device__ __forceinline__ void load(uint8_t *lds, int i, int wid, const uint16_t *p, int left) const {
        const rsrc_t b = buffer(!T && (wid * NL + i) * (64 / PIECES) >= B / 2 ? p + second : p);
        const uint32_t past = kfirst[T ? i : 0] < left ? 0u : kPast;
        load_to_lds(b, lds + (wid * NL + i) * PLACE, off[i] | past, 0);
    }
    // 16 rows (the wave's first + row) by 32 k in the matrix instruction's layout: lane (l % 16: row, l / 16: 8 of k)
    __device__ __forceinline__ bf16x8 fragment(const uint8_t *lds, int row, int chunk) const {
        if constexpr (!T) {
            // 4 pieces on is a change of one bit of the permuted place
            return __builtin_bit_cast(bf16x8, ld16(lds + (chunk ? from ^ 64 : from) + row * (KS * 2)));
        } else {
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            const uint8_t *p = lds + from + row * 2 + line_at(32 * chunk);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + line_at(8)));
            return __builtin_bit_cast(bf16x8, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
        }
    }
};

// 8 results of a row, as a lane has them for the epilogue.
struct Eight {
    float v[8];
    // The lane's 4 values of one group of 16 columns (at 4 quad) and of the next
    // become 8 neighbours of one of them: lanes of odd quads hand over their a
    // for the b of the quad before.  A store is then 16 bytes a lane, 64 a row.
    __device__ __forceinline__ Eight(const f32x4 &a, const f32x4 &b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const auto s = __builtin_amdgcn_permlane16_swap(f2u(a[i]), f2u(b[i]), false, false);
            v[i] = u2f(s[0]);
            v[4 + i] = u2f(s[1]);
        }
    }
    // The first of those columns, from the first of a's group.
    static __device__ __forceinline__ int column(int quad) { return 16 * (quad & 1) + 8 * (quad >> 1); }
    __device__ __forceinline__ void add(const float *p) {   // 8 fp32 values
        const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += a[i], v[4 + i] += b[i];
    }
    __device__ __forceinline__ void add(vec16 w) {   // 8 bf16 values
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] += bf16_lo(w[i]), v[2 * i + 1] += bf16_hi(w[i]);
    }
    __device__ __forceinline__ void store(float *p) const {
        *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4 *>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
    __device__ __forceinline__ void store(uint16_t *p) const {
        st16(p, vec16{pack_bf16x2_cvt(v[0], v[1]), pack_bf16x2_cvt(v[2], v[3]), pack_bf16x2_cvt(v[4], v[5]),
                      pack_bf16x2_cvt(v[6], v[7])});
    }
    __device__ __forceinline__ void store(void *out, bool f32, int64_t at) const {
        if (f32)
            store(static_cast<float *>(out) + at);
        else
            store(static_cast<uint16_t *>(out) + at);
    }
};

// The last steps of 8 results at row r, columns c .. c + 7 (gated: their factors in u).
template <bool GATED>
__device__ __forceinline__ void finish(const Product &p, int64_t r, int64_t c, Eight v, Eight u, vec16 residual) {
    const int64_t at = r * p.out_ld + c;
    if (p.linear) {
        if (p.bias) {
            v.add(p.bias + c);
            if (GATED) u.add(p.bias + p.out_ld + c);
        }
        if (p.z) {
            v.store(p.z + (GATED ? at + r * p.out_ld : at));
            if (GATED) u.store(p.z + at + (r + 1) * p.out_ld);
        }
        with_activation(p.act, [&](auto act) { activate8<decltype(act)::value, GATED>(v.v, u.v); });
        if (p.residual) v.add(residual);
    }
    v.store(p.out, p.out_f32, at);
}

// Which tile a block takes.  Consecutive blocks go to the 8 XCDs in turn; each
// XCD takes an eighth of the tiles, in groups of 8 rows by 4 columns (fewer rows
// where there are fewer), which share their operands in its L2.
struct Order {
    int rows, cols;
    __host__ __device__ int64_t blocks() const { return ((int64_t)rows * cols + 7) / 8 * 8; }
    __device__ __forceinline__ bool tile(uint32_t block, int *row, int *col) const {
        const uint32_t total = rows * cols, share = (total + 7) / 8, t = block % 8 * share + block / 8;
        if (t >= total) return false;
        const uint32_t band = t / (8 * cols), in = t % (8 * cols), left = rows - 8 * band, high = left < 8 ? left : 8;
        const uint32_t group = in / (4 * high), at = in % (4 * high), wide = cols - 4 * group < 4 ? cols - 4 * group : 4;
        *row = (int)(8 * band + at / wide);
        *col = (int)(4 * group + at % wide);
        return true;
    }
};

// One block: BR rows by BC columns of C, WR by WC waves; a step is KS of k.  NB
// steps' operands have room in LDS: while step s is multiplied, the fragments of
// s + 1 are read and the operands of s + NB are on their way into the place of s,
// which every wave had read before the barrier.  Where tiles are few, SK such
// groups of waves each take a part of the steps, and the first adds up the sums
// in order.  With P parts of R beside each other, every step has those of all, each
// with sums of its own, and Q is brought once for them; with P 1 they follow each
// other (p.parts).
template <bool TR, bool TQ, bool GATED, int BR, int BC, int WR, int WC, int KS, int NB, int SK, int P>
struct Tile {
    static constexpr int W = WR * WC, THREADS = 64 * W * SK, ROWS = BR / WR / 16, NR = P * ROWS, NC = BC / WC / 16,
                         CH = KS / 32;
    static_assert(NC % (GATED ? 4 : 2) == 0, "pairs of groups of columns, of a gate's and of their factors, in one wave");
    static_assert(NB >= 2 && NB <= 4, "as many buffers");
    typedef Side<TR, BR, W, KS> R;
    typedef Side<TQ, BC, W, KS> Q;
    static constexpr int RBYTES = P * R::BYTES, BYTES = RBYTES + Q::BYTES;
    static_assert(SK == 1 || (W * NC * NR * 1024 <= SK * BYTES && SK <= NB + 1), "a buffer takes the sums of a part");
    static constexpr int BUFFERS = NB, LDS = SK * BYTES;   // of each buffer
    // The buffers are the kernel's, one array each, so that the compiler can tell them apart.
    static __device__ __forceinline__ void run(const Product &p, uint32_t block, uint8_t *buf0, uint8_t *buf1,
                                               uint8_t *buf2, uint8_t *buf3);
};

template <bool TR, bool TQ, bool GATED, int BR, int BC, int WR, int WC, int KS, int NB, int SK, int P>
__device__ __forceinline__ void Tile<TR, TQ, GATED, BR, BC, WR, WC, KS, NB, SK, P>::run(
    const Product &p, uint32_t block, uint8_t *buf0, uint8_t *buf1, uint8_t *buf2, uint8_t *buf3) {
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wid = wave % W, sk = wave / W;
    const auto buf = [&](int j) {
        return (j % NB == 0 ? buf0 : (j % NB == 1 ? buf1 : (j % NB == 2 ? buf2 : buf3))) + sk * BYTES;
    };

    int rt, ct;
    if (!Order{p.rtiles, p.ctiles}.tile(block, &rt, &ct)) return;
    const int wr = wid / WC, wc = wid % WC;
    const int64_t r0 = (int64_t)rt * BR, c0 = (int64_t)ct * (GATED ? BC / 2 : BC);

    // the wave's groups of 16 columns; gated: half of them from each half of the tile
    const int cw = wc * (GATED ? BC / 2 / WC : BC / WC);
    const auto qrow = [](int f) { return GATED ? (f / (NC / 2)) * (BC / 2) + f % (NC / 2) * 16 : f * 16; };
    R lr;
    Q lq;
    lr.init(p.r, r0, wr * (BR / WR), lane, wid);
    lq.init(p.q, c0, cw, lane, wid);
    constexpr int LR = P * R::NL, L = LR + Q::NL;
    const int k = (int)p.k, steps = (k + KS - 1) / KS, all = steps * p.parts;
    // this group's steps: as many for each (barriers), the last one's may lie past the sum
    const int share = (all + SK - 1) / SK, s0 = sk * share;
    // The steps are staged in turn: where the next one starts, what is left of k
    // there (0 past the group's last step: nothing is read).
    int part = s0 / steps, at = s0 % steps, todo = min(share, all - s0), left = todo > 0 ? k - at * KS : 0;
    const uint16_t *rp = lr.base + part * p.part + at * lr.step, *qp = lq.base + at * lq.step;
    const auto advance = [&]() {
        rp += lr.step;
        qp += lq.step;
        left -= KS;
        if (++at == steps) {
            at = 0;
            rp = lr.base + ++part * p.part;
            qp = lq.base;
            left = k;
        }
        if (--todo <= 0) left = 0;
    };
    const auto stage = [&](uint8_t *to, int i) {   // load i of the wave
        if (i < LR)
            lr.load(to + i / R::NL * R::BYTES, i % R::NL, wid, rp + i / R::NL * p.part, left);
        else
            lq.load(to + RBYTES, i - LR, wid, qp, left);
        if (i == L - 1) advance();
    };
    struct Fragments {   // of 32 of k
        bf16x8 r[NR], q[NC];
    };
    const auto read = [&](const uint8_t *from, Fragments &f, int c, int i) {   // fragment i of part c of a step
        if (i < NC)
            f.q[i] = lq.fragment(from + RBYTES, qrow(i), c);
        else
            f.r[i - NC] = lr.fragment(from + (i - NC) / ROWS * R::BYTES, 16 * ((i - NC) % ROWS), c);
    };

    f32x4 acc[NC][NR] = {};
    const auto step = [&](Fragments (&f)[2], int first, uint8_t *mine, const uint8_t *after) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const Fragments &now = f[(first + c) % 2];
            Fragments &next = f[(first + c + 1) % 2];
            const bool last = c == CH - 1;
            if (last) {
                // the next step's operands have arrived (behind them NB - 2 steps' are
                // under way), and the last of this step's fragments: every wave's after
                // the barrier, and this step's place is free
                __builtin_amdgcn_s_waitcnt(0x0070 | ((NB - 2) * L & 15) | ((NB - 2) * L >> 4) << 14);   // lgkmcnt(0) too
                barrier_only();
            }
            constexpr int READS = NR + NC;
#pragma unroll
            for (int m = 0; m < NR; ++m) {   // NC matrix instructions, and a share of the rest
                if (last)
#pragma unroll
                    for (int i = m * L / NR; i < (m + 1) * L / NR; ++i) stage(mine, i);
#pragma unroll
                for (int i = m * READS / NR; i < (m + 1) * READS / NR; ++i)
                    read(last ? after : mine, next, last ? 0 : c + 1, i);
#pragma unroll
                for (int n = 0; n < NC; ++n) acc[n][m] = mfma(now.q[n], now.r[m], acc[n][m]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < L; ++i) stage(buf(j), i);
    wait_loads<(NB - 1) * L>();
    barrier_only();
    Fragments f[2];
#pragma unroll
    for (int i = 0; i < NR + NC; ++i) read(buf(0), f[0], 0, i);
    constexpr int TURN = NB % 2 ? 2 * NB : NB;
    // whole turns: steps past the last one multiply zeros
    for (int s = 0; s < share; s += TURN)
#pragma unroll
        for (int j = 0; j < TURN; ++j) step(f, j * CH % 2, buf(j), buf(j + 1));
    wait_loads<0>();

    if constexpr (SK > 1) {
        __syncthreads();
        const auto sums = [&](int q) {   // of part q > 0, this wave's
            return reinterpret_cast<f32x4 *>(q == 1 ? buf0 : (q == 2 ? buf1 : (q == 3 ? buf2 : buf3))) +
                   wid * NC * NR * kWave + lane;
        };
#pragma unroll
        for (int q = 1; q < SK; ++q)
            if (sk == q)
#pragma unroll
                for (int i = 0; i < NC * NR; ++i) sums(q)[i * kWave] = acc[i / NR][i % NR];
        __syncthreads();
        if (sk > 0) return;
#pragma unroll
        for (int q = 1; q < SK; ++q)
#pragma unroll
            for (int i = 0; i < NC * NR; ++i) acc[i / NR][i % NR] += sums(q)[i * kWave];
    }

    if constexpr (P > 1)   // the smallest parts first
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int m = 0; m < ROWS; ++m) {
                f32x4 v = acc[i][(P - 1) * ROWS + m];
#pragma unroll
                for (int q = P - 2; q >= 0; --q) v += acc[i][q * ROWS + m];
                acc[i][m] = v;
            }

    // pairs of groups of columns; the residual's values are all on their way before the first is used
    const int r16 = lane & 15, quad = lane >> 4;
    constexpr int PAIRS = GATED ? NC / 4 : NC / 2, HALF = GATED ? NC / 2 : 0;   // without a gate the factors are not looked at
    const auto row = [&](int m) { return r0 + wr * (BR / WR) + 16 * m + r16; };
    const auto column = [&](int f) { return c0 + cw + 32 * f + Eight::column(quad); };
    const auto inside = [&](int f, int m) { return row(m) < p.r.rows && column(f) < p.out_ld; };
    vec16 residual[PAIRS][ROWS] = {};
    if (p.residual)
#pragma unroll
        for (int f = 0; f < PAIRS; ++f)
#pragma unroll
            for (int m = 0; m < ROWS; ++m)
                if (inside(f, m)) residual[f][m] = ld16(p.residual + row(m) * p.out_ld + column(f));
#pragma unroll
    for (int f = 0; f < PAIRS; ++f) {
#pragma unroll
        for (int m = 0; m < ROWS; ++m) {
            const Eight v(acc[2 * f][m], acc[2 * f + 1][m]), u(acc[2 * f + HALF][m], acc[2 * f + 1 + HALF][m]);
            if (inside(f, m)) finish<GATED>(p, row(m), column(f), v, u, residual[f][m]);
        }
    }
}

template <typename T>
__global__ __launch_bounds__(T::THREADS) void ep_linear_tile_kernel(Product p) {
    __shared__ __attribute__((aligned(16))) uint8_t buf0[T::LDS];
    __shared__ __attribute__((aligned(16))) uint8_t buf1[T::LDS];
    __shared__ __attribute__((aligned(16))) uint8_t buf2[T::BUFFERS > 2 ? T::LDS : 16];
    __shared__ __attribute__((aligned(16))) uint8_t buf3[T::BUFFERS > 3 ? T::LDS : 16];
    T::run(p, blockIdx.x, buf0, buf1, buf2, buf3);
}

template <bool TR, bool TQ, bool GATED, int BR, int BC, int WR, int WC, int KS, int NB, int SK = 1, int P = 1>
hipError_t launch_tile(Product p, hipStream_t stream) {
    typedef Tile<TR, TQ, GATED, BR, BC, WR, WC, KS, NB, SK, P> T;
    if (P > 1) p.parts = 1;
    const int cols = GATED ? BC / 2 : BC;
    p.rtiles = (int)((p.r.rows + BR - 1) / BR);
    p.ctiles = (int)((p.out_ld + cols - 1) / cols);
    hipLaunchKernelGGL(ep_linear_tile_kernel<T>, dim3((unsigned)Order{p.rtiles, p.ctiles}.blocks()), dim3(T::THREADS), 0,
                       stream, p);
    return hipGetLastError();
}

int64_t tile_count(const Product &p, int BR, int BC) {
    const int64_t cols = p.gated ? 2 * p.out_ld : p.out_ld;
    return (p.r.rows + BR - 1) / BR * ((cols + BC - 1) / BC);
}

// The largest tile that still gives 160 blocks (of 256 CUs), as a larger one reads
// less of LDS and memory for a product, by 8 waves as far as pairs of groups of
// columns go; in us:
//   4096 rows 7168 -> 2048 x 2   256 x 256 tiles 195, 128 x 128 236, 256 x 128 242
//   2048 rows 2048 -> 7168       256 x 256 tiles 73, 128 x 128 80
//   1024 rows 7168 -> 2048       64 x 128 (256 tiles) 37.5, 128 x 128 (128) 62, 64 x 64 (512) 46
//   512 rows 4096 -> 4096        64 x 128 (256) 24.0, 128 x 128 (128) 37.6, 64 x 64 (512) 27.5
// The rule leaves the sums' length out; of 4096 rows by 7168 and by 4096 columns (448
// and 256 of the largest tiles), 256 x 256 / 128 x 128: K = 64 31.4 / 37.6 and 20.2 /
// 23.8, 256 38.0 / 36.9 and 23.4 / 22.2, 512 49.3 / 47.5 and 28.8 / 28.5, 1024 70.6 / 75.0
// and 40.2 / 43.9; dx of 4096 x 7168 from K = 128 22.5 / 35.7, 256 28.0 / 35.9, 512 38.6 /
// 46.7.
// The weights' gradient, whose operands both come by lines of k, gains by 256 x 128
// in between (4096 x 2048 from 4096 rows 62, 128 x 128 72; 2560 x 2048 from 16384
// rows 171 / 221), the other products lose (2048 rows 4096 -> 4096 77 / 73).
// 128 x 128 tiles by 8 waves at 64 of k a step against 4 at 32 (two blocks a CU):
// 1024 rows 7168 -> 2048 x 2 59 / 75, 2048 rows 4096 -> 2048 36 / 41; 64 x 128 ones
// by 8 waves against 4: 512 rows 4096 -> 4096 24.5 / 26.8, but with a gate, where
// a wave has a gate's columns and their factors', 45.3 / 44.0.
// Where even those of 64 x 64 are 128 at most, two groups of waves with half the
// steps each, if those are 16 or more:
//   64 rows 7168 -> 2048 x 2 27.9, halved 24.3;  100 rows 4096 -> 4096 18.1, 16.1
//   300 rows 4096 -> 1024    17.8, halved 15.5;  512 rows 7168 -> 256  28.6, 24.9
// Shorter sums lose by it (512 rows by 1024: K = 256 4.7, halved 5.7, 512 5.5 / 5.8, 1024
// 7.3 / 7.1).  Past 128 tiles, with a CU's LDS full of one block, it would still gain where
// sums are long: 768 rows by 1024 (192 tiles) K = 1024 7.4, halved 7.3, 2048 11.1 / 10.0,
// 7168 28.3 / 24.5; 256 tiles 7168 29.0 / 26.5.
template <bool TR, bool TQ, bool GATED>
hipError_t launch_product(const Product &p, hipStream_t stream) {
    const auto tiles = [&](int BR, int BC) { return tile_count(p, BR, BC); };
    // Three parts of dz beside each other where tiles of 64 x 128 are 64 or more, and
    // those of 256 x 256 too few (weights' gradients with dz's kernel, us, beside /
    // after each other: 256 x 7168 from 4096 rows 53 / 83, 512 x 7168 82 / 114; 128 x
    // 2048 from 1024 rows, 32 tiles, 18.4 / 16.8; 4096 x 7168 from 1024 rows, in
    // tiles of 256 x 256 where their sums find no registers, 181 / 164).  Not for
    // short sums, which may come in one launch with the other gradients.
    if constexpr (TR)
        if (p.parts == 3 && 3 * p.k >= 1024 && tiles(256, 256) < 160) {
            if (tiles(128, 128) >= 160) return launch_tile<TR, TQ, GATED, 128, 128, 4, 2, 32, 4, 1, 3>(p, stream);
            if (tiles(64, 128) >= 64) return launch_tile<TR, TQ, GATED, 64, 128, 2, 4, 64, 3, 1, 3>(p, stream);
        }
    if (tiles(256, 256) >= 160) return launch_tile<TR, TQ, GATED, 256, 256, 2, 4, 32, 4>(p, stream);
    if constexpr (TR)
        if (tiles(256, 128) >= 160) return launch_tile<TR, TQ, GATED, 256, 128, 4, 2, 32, 4>(p, stream);
    if (tiles(128, 128) >= 160) return launch_tile<TR, TQ, GATED, 128, 128, GATED ? 4 : 2, GATED ? 2 : 4, 64, 4>(p, stream);
    if (tiles(64, 128) >= 160) return launch_tile<TR, TQ, GATED, 64, 128, 2, GATED ? 2 : 4, 64, 4>(p, stream);
    if (tiles(64, 64) <= 128 && p.k * p.parts >= 1024)
        return launch_tile<TR, TQ, GATED, 64, 64, 4, 1, 64, 4, 2>(p, stream);
    return launch_tile<TR, TQ, GATED, 64, 64, 4, 1, 64, 4>(p, stream);
}

// ---------------------------------------------------------------- few rows

// One block: 16 G weight rows (gated: 8 G of each half) by up to 16 MT rows of
// x, NW waves with a part of K each; the weights' bytes are the time (16 rows 7168
// -> 2 x 2048: 59 MB in 12.2 us, 4.8 TB/s; 7168 -> 7168: 103 MB in 17.5, 5.9).
template <bool GATED, int G, int MT, int NW>
__global__ __launch_bounds__(64 * NW) void ep_linear_stream_kernel(Product p, int ctiles) {
    typedef Step<false, G> S;
    constexpr int KE = S::KE, C = S::CHUNKS;
    __shared__ __attribute__((aligned(16))) uint8_t buf0[NW * G * 2048];
    __shared__ __attribute__((aligned(16))) uint8_t buf1[NW * G * 2048];
    constexpr int NB = 2;
    const auto buf = [&](int j) { return j % NB ? buf1 : buf0; };
    const int c0 = (int)(blockIdx.x % ctiles) * (GATED ? 8 * G : 16 * G);
    const int64_t r0 = (int64_t)(blockIdx.x / ctiles) * 16 * MT;
    const int rows = (int)min(p.r.rows - r0, (int64_t)16 * MT);
    const int lane = threadIdx.x & (kWave - 1), wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane & 15, quad = lane >> 4;
    const uint32_t kbytes = (uint32_t)p.k * 2;
    const int KU = ((int)p.k + KE - 1) / KE;
    const int first = KU * wid / NW, n = KU * (wid + 1) / NW - first;

    // gated: the first half of the LDS rows is the gate's, the second its factor's
    const uint16_t *w0 = p.q.p + (int64_t)c0 * p.q.ld, *w1 = GATED ? w0 + p.q.split * p.q.ld : w0;
    const rsrc_t b0 = buffer(w0), b1 = buffer(w1);
    const int last = (int)p.out_ld - 1 - c0;
    uint32_t woff[2 * G];
    const int srow = lane >> 3;
    const uint32_t piece = (uint32_t)(((lane & 7) ^ srow) << 4);
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) woff[i] = (uint32_t)min(srow + 8 * (GATED ? i % G : i), last) * kbytes + piece;
    const auto stage = [&](uint8_t *to, int i) {
        const uint32_t k = (uint32_t)(first + i) * 128, past = i < n && k + piece < kbytes ? 0u : kPast;
#pragma unroll
        for (int j = 0; j < 2 * G; ++j)
            load_to_lds(GATED && j >= G ? b1 : b0, to + wid * (G * 2048) + j * 1024, woff[j] | past, i < n ? k : 0u);
    };
    const rsrc_t xb = buffer(p.r.p + r0 * p.r.ld);
    uint32_t xoff[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) xoff[m] = 16 * m + r16 < rows ? (uint32_t)(16 * m + r16) * kbytes : kPast;
    struct Values {
        vec16 v[MT][C];
    };
    const auto load_x = [&](int i, Values &to) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const uint32_t at = (uint32_t)(first + i) * 128 + S::at(c, quad);
                to.v[m][c] = load_16(xb, i < n && at < kbytes ? xoff[m] + at : kPast, 0);
            }
    };
    f32x4 acc[G][MT] = {};
    const uint32_t plo = (uint32_t)(r16 * 128 + ((quad ^ (r16 & 7)) << 4));
    const auto step = [&](uint8_t *b, const Values &x, Values &next, int i) {
        wait_step<NB, MT * C, 2 * G>(i);
        const S a(b + wid * (G * 2048), plo);
        __builtin_amdgcn_sched_barrier(0);
        load_x(i + 1, next);
        __builtin_amdgcn_sched_barrier(0);
        stage(b, i + NB);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int g = 0; g < G; ++g)
                    acc[g][m] = mfma(a.a[g][c], __builtin_bit_cast(bf16x8, x.v[m][c]), acc[g][m]);
    };
    Values v[2];
    stage(buf0, 0);
    __builtin_amdgcn_sched_barrier(0);
    load_x(0, v[0]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 1; j < NB; ++j) stage(buf(j), j);
    for (int i = 0; i < n; i += NB) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (j == 0 || i + j < n) step(buf(j), v[j % 2], v[(j + 1) % 2], i + j);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);

    // the parts of K are added in their order: a tile of rows by one wave each
    __syncthreads();
    static_assert(MT <= 2 * NB && MT <= NW, "they fit, and a wave for each");
    const auto part = [&](int m) { return reinterpret_cast<f32x4 *>(buf(m / 2)) + m % 2 * (NW * G * kWave) + lane; };
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int g = 0; g < G; ++g) part(m)[(wid * G + g) * kWave] = acc[g][m];
    __syncthreads();
    if (wid >= MT) return;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (m != wid) continue;
        f32x4 sum[G] = {};
#pragma unroll
        for (int q = 0; q < NW; ++q)
#pragma unroll
            for (int g = 0; g < G; ++g) sum[g] += part(m)[(q * G + g) * kWave];
        const int r = 16 * m + r16;
        vec16 residual = {};
        if constexpr (GATED || G == 1) {
            // the lane's 4 columns and its neighbour's 4 (a quad on)
            const f32x4 &u = sum[G - 1];
            const Eight v(sum[0], sum[0]);
            Eight w(u, u);
            // one group of weight rows: gate in quads 0 and 1, factors in quads 2 and 3
            if constexpr (GATED && G == 1)
#pragma unroll
                for (int i = 0; i < 8; ++i) w.v[i] = __shfl_xor(v.v[i], 32);
            const int c = c0 + 8 * (quad >> 1);
            if (r < rows && quad % 2 == 0 && (!GATED || G > 1 || quad == 0) && c < p.out_ld) {
                if (p.residual) residual = ld16(p.residual + (r0 + r) * p.out_ld + c);
                finish<GATED>(p, r0 + r, c, v, w, residual);
            }
        } else {
            const int c = c0 + Eight::column(quad);
            const Eight v(sum[0], sum[G - 1]);
            if (r < rows && c < p.out_ld) {
                if (p.residual) residual = ld16(p.residual + (r0 + r) * p.out_ld + c);
                finish<GATED>(p, r0 + r, c, v, v, residual);
            }
        }
    }
}

template <bool GATED, int G, int MT, int NW>
hipError_t launch_stream(const Product &p, hipStream_t stream) {
    const int wide = GATED ? 8 * G : 16 * G, ctiles = (int)((p.out_ld + wide - 1) / wide);
    const int64_t blocks = ctiles * ((p.r.rows + 16 * MT - 1) / (16 * MT));
    hipLaunchKernelGGL((ep_linear_stream_kernel<GATED, G, MT, NW>), dim3((unsigned)blocks), dim3(64 * NW), 0, stream,
                       p, ctiles);
    return hipGetLastError();
}

// 16 weight rows a block and 8 waves while every block has a CU of its own, else 32
// and 4 (us for 16 rows of x; 16 x 8 / 32 x 4):
//   7168 -> 1024 10.7 / 11.9    2048 -> 7168       8.2 / 6.3
//   4096 -> 4096  8.0 / 9.2     7168 -> 7168      21.0 / 17.5
//   7168 -> 2048 x 2 12.5 / 14.8    4096 -> 16384 23.9 / 22.4
// Twice the waves or four steps ahead instead of two take a CU's LDS for one block,
// and the next one has to wait for it to end: 15.2 for the 12.5.
template <bool GATED, int MT>
hipError_t launch_stream(const Product &p, hipStream_t stream) {
    if ((GATED ? 2 : 1) * p.out_ld > 16 * 256) return launch_stream<GATED, 2, MT, 4>(p, stream);
    return launch_stream<GATED, 1, MT, 8>(p, stream);
}

// ---------------------------------------------------------------- the gradient over z

// dz from dy and z in bf16 (in one part, or in two or three: the rounded value, its
// rounded rest and the rest of that, together the binary32 value) and the sums of
// its columns over runs of dz_rows rows, for the bias.  One part where dy is bf16
// too, as a gradient between two bf16 operators is; two from an fp32 dy, whose
// precision the caller asks for: they lose 2^-17 of it where one loses 2^-8 (the
// logits' backward pass, 4096 x 7168 -> 256, takes 95 us with dx in two parts,
// 84 in one); three where the weights' gradient stays in fp32.  A thread takes 8 columns
// of a row, CG of them (a power of two, 64 at most) a row of up to 512 columns,
// the block's others further rows, 4 at a time so that their loads are under way
// together.  4096 rows of 2 x 2048 with silu's gate: 84 MB in 27.5 us, 3.1 TB/s, of
// which the vector instructions, 49 for a pair of results, are 11.
constexpr int kDzThreads = 256;
// A kernel for each activation: with all of them in one its code alone took a
// small call 10 us to fetch (100 rows of 512: 18 us).
template <typename Dy, int ACT, bool GATED>
__global__ __launch_bounds__(kDzThreads) void ep_linear_dz_kernel(LinearShape s, const Dy *__restrict__ dy,
                                                                  const uint16_t *__restrict__ z,
                                                                  uint16_t *__restrict__ dz, int parts,
                                                                  float *__restrict__ sums, int shift, int run_rows) {
    constexpr int D = sizeof(Dy) / 2, AT_ONCE = 4;
    __shared__ float part[2][8][kDzThreads];
    const int sub = threadIdx.x >> shift, cg = threadIdx.x & ((1 << shift) - 1), rows = kDzThreads >> shift;
    const int cols = (s.N + 511) / 512, ct = blockIdx.x % cols;
    const int64_t run = blockIdx.x / cols, end = min((run + 1) * run_rows, s.M);
    const int c = ct * 512 + cg * 8, wide = s.wide();
    const int64_t plane = s.M * wide;
    constexpr bool KEPT = ACT != kActNone || GATED;
    float sum[2][8] = {};
    const auto unpack = [](vec16 v, float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(v[i]), f[2 * i + 1] = bf16_hi(v[i]);
    };
    const auto store = [&](int64_t at, float (&f)[8]) {
        if (parts == 1) {
            st16(dz + at, vec16{pack_bf16x2_cvt(f[0], f[1]), pack_bf16x2_cvt(f[2], f[3]), pack_bf16x2_cvt(f[4], f[5]),
                                pack_bf16x2_cvt(f[6], f[7])});
            return;
        }
        for (int n = 0; n < parts; ++n) {
            vec16 out;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t h[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) h[j] = take_part(f[2 * i + j]);
                out[i] = h[0] | h[1] << 16;
            }
            st16(dz + n * plane + at, out);
        }
    };
    for (int64_t r0 = run * run_rows + sub; r0 < end; r0 += rows * AT_ONCE) {
        vec16 gv[AT_ONCE][D] = {}, zv[AT_ONCE] = {}, uv[AT_ONCE] = {};
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const int64_t r = r0 + i * rows;
            if (r >= end || c >= s.N) continue;
#pragma unroll
            for (int j = 0; j < D; ++j) gv[i][j] = ld16(dy + r * s.N + c + 8 / D * j);
            if (KEPT) zv[i] = ld16(z + r * wide + c);
            if (GATED) uv[i] = ld16(z + r * wide + s.N + c);
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const int64_t r = r0 + i * rows;
            if (r >= end || c >= s.N) continue;
            float g[8], a[8], b[8] = {}, v[8], u[8];
            if constexpr (D == 2) {
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = u2f(gv[i][j / 4][j % 4]);
            } else {
                unpack(gv[i][0], g);
            }
            unpack(zv[i], v);
            unpack(uv[i], u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float f, d;
                derive<ACT>(v[j], &f, &d);
                const float gu = GATED ? g[j] * u[j] : g[j];
                a[j] = ACT == kActRelu ? (v[j] <= 0.0f ? 0.0f : gu) : gu * d;   // gu may be infinite beside a closed gate
                if (GATED) b[j] = g[j] * f;
            }
            if (any_in_tail<ACT>(v)) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (v[j] < kTail<ACT>) {
                        const Tail<ACT> t(v[j]);
                        a[j] = t.slope(g[j], GATED ? u[j] : 1.0f);
                        if (GATED) b[j] = t.value(g[j]);
                    }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[0][j] += a[j], sum[1][j] += b[j];
            store(r * wide + c, a);
            if (GATED) store(r * wide + s.N + c, b);
        }
    }
    if (!sums) return;
#pragma unroll
    for (int h = 0; h < (GATED ? 2 : 1); ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j) part[h][j][threadIdx.x] = sum[h][j];
    __syncthreads();
    if (sub > (GATED ? 1 : 0) || c >= s.N) return;   // the rows' threads, in order; rows is 4 or more
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float v = 0.0f;
        for (int i = 0; i < rows; ++i) v += part[sub][j][(i << shift) + cg];
        sums[run * wide + sub * s.N + c + j] = v;
    }
}

// The runs' sums: 16 columns a block and 16 threads to a column, each with a 16th
// of the runs, added in order; with no runs, 0.
__device__ __forceinline__ void add_runs(const float *__restrict__ sums, int64_t runs, int wide, float *__restrict__ out,
                                         uint32_t block, float (*part)[16]) {
    const int lane = threadIdx.x % 16, group = threadIdx.x / 16, c = block * 16 + lane;
    float v = 0.0f;
    if (c < wide)
        for (int64_t i = runs * group / 16; i < runs * (group + 1) / 16; ++i) v += sums[i * wide + c];
    part[group][lane] = v;
    __syncthreads();
    if (group > 0 || c >= wide) return;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += part[i][lane];
    out[c] = v;
}
__global__ __launch_bounds__(256) void ep_linear_bias_kernel(const float *__restrict__ sums, int64_t runs, int wide,
                                                             float *__restrict__ out) {
    __shared__ float part[16][16];
    add_runs(sums, runs, wide, out, blockIdx.x, part);
}

// The three gradients of a small call in one launch: blocks of the one over x,
// then those over w, then the bias'.
struct Gradients {
    Product x, w;
    uint32_t xblocks, wblocks;
    const float *sums;
    int64_t runs;
    int wide;
    float *bias;
};
typedef Tile<false, true, false, 64, 64, 4, 1, 64, 4, 1, 1> SmallX;
typedef Tile<true, true, false, 64, 64, 4, 1, 64, 4, 1, 1> SmallW;
__global__ __launch_bounds__(256) void ep_linear_gradients_kernel(Gradients g) {
    static_assert(SmallX::THREADS == 256 && SmallW::THREADS == 256, "one kind of block");
    static_assert(SmallX::BUFFERS == 4 && SmallW::BUFFERS == 4, "the same buffers for all");
    constexpr int LDS = SmallX::LDS > SmallW::LDS ? SmallX::LDS : SmallW::LDS;
    static_assert(2 * 4 * LDS <= 160 * 1024, "two blocks a CU");
    __shared__ __attribute__((aligned(16))) uint8_t buf0[LDS];
    __shared__ __attribute__((aligned(16))) uint8_t buf1[LDS];
    __shared__ __attribute__((aligned(16))) uint8_t buf2[LDS];
    __shared__ __attribute__((aligned(16))) uint8_t buf3[LDS];
    if (blockIdx.x < g.xblocks)
        SmallX::run(g.x, blockIdx.x, buf0, buf1, buf2, buf3);
    else if (blockIdx.x - g.xblocks < g.wblocks)
        SmallW::run(g.w, blockIdx.x - g.xblocks, buf0, buf1, buf2, buf3);
    else
        add_runs(g.sums, g.runs, g.wide, g.bias, blockIdx.x - g.xblocks - g.wblocks,
                 reinterpret_cast<float (*)[16]>(buf0));
}

// At most kZeroBlocks blocks: a launch has to stay below 2^32 threads, and 16 bytes
// for each end at 64 GiB.
constexpr int64_t kZeroBlocks = 1 << 16;
__global__ __launch_bounds__(256) void ep_linear_zero_kernel(vec16 *out, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) out[i] = vec16{};
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
    // Few rows: the weights' bytes are the time, and the tile form has too few blocks
    // to fetch them.  Stream / tile form, us: 16 rows 7168 -> 2048 x 2 15 / 26; 32 rows
    // 7168 -> 7168 20.5 / 25, 7168 -> 2048 x 2 20.7 / 22.8, 4096 -> 4096 12.9 / 15.7;
    // from 128 tiles of 64 columns on it has enough (4096 -> 8192 16.4 / 15.9,
    // -> 16384 28 / 23).
    if (s.M <= 16) return s.gated ? launch_stream<true, 1>(p, stream) : launch_stream<false, 1>(p, stream);
    if (s.M <= 32 && s.wide() < 128 * 64) return s.gated ? launch_stream<true, 2>(p, stream) : launch_stream<false, 2>(p, stream);
    return s.gated ? launch_product<false, false, true>(p, stream) : launch_product<false, false, false>(p, stream);
}

hipError_t launch_linear_backward(const LinearShape &s, const void *dy, const uint16_t *x, const uint16_t *w,
                                  const uint16_t *z, uint16_t *grad_x, void *grad_w, float *grad_bias, uint8_t *ws,
                                  hipStream_t stream) {
    const int wide = s.wide();
    if (s.M == 0) {
        if (grad_w) {
            const int64_t n = (int64_t)wide * s.K * (s.w32 ? 4 : 2) / 16;
            const int64_t blocks = (n + 255) / 256;
            hipLaunchKernelGGL(ep_linear_zero_kernel, dim3((unsigned)(blocks < kZeroBlocks ? blocks : kZeroBlocks)),
                               dim3(256), 0, stream, static_cast<vec16 *>(grad_w), n);
        }
        if (grad_bias)
            hipLaunchKernelGGL(ep_linear_bias_kernel, dim3((unsigned)((wide + 15) / 16)), dim3(256), 0, stream,
                               nullptr, 0, wide, grad_bias);
        return grad_w || grad_bias ? hipGetLastError() : hipSuccess;
    }
    // three parts only for the product that takes them
    const int two = s.f32 ? 2 : 1, parts = s.plain() ? 0 : (s.w32 && grad_w ? 3 : two);
    uint16_t *dz = reinterpret_cast<uint16_t *>(ws);
    float *sums = reinterpret_cast<float *>(ws + linear_sums_offset(s));
    const int run_rows = dz_rows(s);
    const int64_t runs = (s.M + run_rows - 1) / run_rows;
    if (grad_bias || (parts > 0 && (grad_x || grad_w))) {
        const dim3 grid((unsigned)(runs * ((s.N + 511) / 512)));
        int shift = 0;   // threads to a row
        while (shift < 6 && (8 << shift) < s.N) ++shift;
        const auto launch = [&](const auto *from, auto gated) {
            typedef std::remove_const_t<std::remove_pointer_t<decltype(from)>> Dy;
            with_activation(s.act, [&](auto act) {
                hipLaunchKernelGGL((ep_linear_dz_kernel<Dy, decltype(act)::value, decltype(gated)::value != 0>), grid,
                                   dim3(kDzThreads), 0, stream, s, from, z, dz, parts, grad_bias ? sums : nullptr,
                                   shift, run_rows);
            });
        };
        if (s.f32)
            s.gated ? launch(static_cast<const float *>(dy), Const<1>()) : launch(static_cast<const float *>(dy), Const<0>());
        else
            s.gated ? launch(static_cast<const uint16_t *>(dy), Const<1>())
                    : launch(static_cast<const uint16_t *>(dy), Const<0>());
    }
    const uint16_t *d = parts > 0 ? dz : static_cast<const uint16_t *>(dy);
    Gradients g = {};
    g.sums = sums;
    g.runs = runs;
    g.wide = wide;
    g.bias = grad_bias;
    g.x.r = {d, s.M, wide, 0};
    g.x.q = {w, s.K, s.K, 0};
    g.x.k = wide;
    g.x.parts = two;
    g.x.part = s.M * wide;
    g.x.out_ld = s.K;
    g.x.out = grad_x;
    g.w.r = {d, wide, wide, 0};
    g.w.q = {x, s.K, s.K, 0};
    g.w.k = s.M;
    g.w.parts = parts > 1 ? parts : 1;
    g.w.part = s.M * wide;
    g.w.out_ld = s.K;
    g.w.out = grad_w;
    g.w.out_f32 = s.w32;
    const unsigned columns = grad_bias ? (unsigned)((wide + 15) / 16) : 0;
    // Small calls: what counts is the launches.  One for all three against three of
    // them, with dz's, us: 100 rows 1000 -> 512 (160 tiles) 10.1 / 15.6, 340 rows 1536
    // -> 512 (336) 10.6 / 17.4, 1000 rows 1024 -> 960 (496) 18.2 / 25.2, 1000 rows 1000
    // -> 1000 (512) 23.8 / 29.3.  Up to 512 tiles both products' blocks have room on
    // the chip at once: two a CU, as all kinds of blocks share one set of buffers, 66
    // KiB (with a set for each, 132, those cases took 10.2, 13.3, 23.2 and 27.5).  And
    // sums below 1024 are those that launch_product does not halve: a gradient that
    // is asked for alone has the same bits.
    if (grad_x && grad_w && tile_count(g.x, 64, 64) + tile_count(g.w, 64, 64) <= 512 &&
        wide * g.x.parts < 1024 && s.M * g.w.parts < 1024) {
        const auto tiles = [](Product &p) {
            p.rtiles = (int)((p.r.rows + 63) / 64);
            p.ctiles = (int)((p.out_ld + 63) / 64);
            return (uint32_t)Order{p.rtiles, p.ctiles}.blocks();
        };
        g.xblocks = tiles(g.x);
        g.wblocks = tiles(g.w);
        hipLaunchKernelGGL(ep_linear_gradients_kernel, dim3(g.xblocks + g.wblocks + columns), dim3(256), 0, stream, g);
        return hipGetLastError();
    }
    if (grad_bias)
        hipLaunchKernelGGL(ep_linear_bias_kernel, dim3(columns), dim3(256), 0, stream, sums, runs, wide, grad_bias);
    hipError_t e = grad_x || grad_w || grad_bias ? hipGetLastError() : hipSuccess;
    if (grad_x && e == hipSuccess) e = launch_product<false, true, false>(g.x, stream);
    if (grad_w && e == hipSuccess) e = launch_product<true, true, false>(g.w, stream);
    return e;
}

}  // namespace ep
