// few.hip -- the whole experts' layer for a few tokens, for gfx950, in two
// kernels:
//
//   h[t, j]  = w[t, j] silu(G_e x[t]) * (U_e x[t]),   e = topk_idx[t, j]
//   y[t]     = residual[t] + sum_j D_e h[t, j]
//
// At this size each expert's weights serve a few rows, and their bytes are the
// time: 3 H I of them for every expert that a token has, read once.  Both
// kernels stream them through LDS by direct loads, 64 or 32 rows by 128 bytes a
// wave and step, two or four steps ahead, without a barrier; the products run
// in 16-bit matrix instructions, with e4m3 weights widened to bf16 (exactly)
// on their way.  The weights are the first operand, the tokens' rows the
// second, so a lane's 4 results lie at consecutive columns of one token.
//
// Measured, first + second kernel: one token, 8 experts of 7168 x 2048 in e4m3,
// 45 + 29 us (5.2 and 4.1 TB/s); 32 tokens over 64 such experts, top-8, 306 + 165
// (6.1 and 5.7; a large plain read reaches 6.8); 64 tokens, 96 experts of 2048 x
// 1408, top-6, 117 + 64 (4.7 and 4.3: K or I in waves' parts of few steps).
//
// No expert's rows are gathered first: a block of the first kernel finds its
// expert and that one's tokens in topk_idx by itself, and one extra block writes
// down for the second kernel which expert has which rows.
#include "dense.h"
#include "ep_device.h"
#include "stream_device.h"
#include "tile_device.h"

namespace ep {
namespace {

// ---------------------------------------------------------------- the segments

// Sum up to and with the lane.
__device__ __forceinline__ int scan(int v) {
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const int u = __shfl_up(v, d);
        if (lane >= d) v += u;
    }
    return v;
}

// Which expert has which rows, for the second kernel: one block, experts
// ascending, each one's tokens ascending, 16 a segment.  It also clears that
// kernel's counts of blocks that are done.
constexpr int kPlanThreads = 256;
struct Plan {
    uint32_t used[128];              // a bit for every expert
    uint16_t ids[kFewTokens * 32];   // topk_idx, 0xFFFF where masked
    uint16_t list[kFewTokens * 32];  // the experts that are used
    uint16_t first[kFewTokens * 32]; // segments, then the first of each
    int total;
};
__device__ void make_plan(Plan &p, const FewShape &s, const int64_t *idx, int32_t *count, FewSegment *seg,
                          int32_t *arrived) {
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wid = tid / kWave, pairs = s.T * s.k;
    if (tid < 128) p.used[tid] = 0;
    if (tid < kFewJoins) arrived[tid] = 0;
    __syncthreads();
    for (int i = tid; i < pairs; i += kPlanThreads) {
        const int64_t e = idx[i];
        const bool ok = e >= 0 && e < s.E;
        p.ids[i] = ok ? (uint16_t)e : 0xFFFF;
        if (ok) atomicOr(&p.used[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    if (wid == 0) {
        const uint32_t a = p.used[2 * lane], b = p.used[2 * lane + 1];
        uint64_t bits = (uint64_t)b << 32 | a;
        const int upto = scan(__popcll(bits));
        int at = upto - __popcll(bits);
        for (; bits; bits &= bits - 1) p.list[at++] = (uint16_t)(64 * lane + __builtin_ctzll(bits));
        if (lane == kWave - 1) p.total = upto;
    }
    __syncthreads();
    const int used = p.total;
    const auto find = [&](int e) {   // the lane's token: its first slot with expert e, or -1
        int j = -1;
        if (lane < s.T)
            for (int i = s.k - 1; i >= 0; --i)
                if (p.ids[lane * s.k + i] == e) j = i;
        return j;
    };
    for (int d = wid; d < used; d += kPlanThreads / kWave) {
        const int n = __popcll(__ballot(find(p.list[d]) >= 0));
        if (lane == 0) p.first[d] = (uint16_t)((n + 15) / 16);
    }
    __syncthreads();
    if (wid == 0) {
        int carry = 0;
        for (int d = 0; d < used; d += kWave) {
            const int n = d + lane < used ? p.first[d + lane] : 0, upto = scan(n);
            if (d + lane < used) p.first[d + lane] = (uint16_t)(carry + upto - n);
            carry += __shfl(upto, kWave - 1);
        }
        if (lane == 0) *count = carry;
    }
    __syncthreads();
    for (int d = wid; d < used; d += kPlanThreads / kWave) {
        const int e = p.list[d], j = find(e);
        const uint64_t has = __ballot(j >= 0);
        const int rank = __popcll(has & lanemask_lt()), n = __popcll(has);
        for (int g = 0; g * 16 < n; ++g) {
            FewSegment *o = seg + p.first[d] + g;
            const bool in = j >= 0 && rank / 16 == g;
            const uint64_t tokens = __ballot(in);
            if (in) reinterpret_cast<uint16_t *>(o->pair)[rank % 16] = (uint16_t)(lane * s.k + j);
            if (lane == 0) {
                o->tokens = tokens;
                o->expert = e;
                o->rows = min(16, n - 16 * g);
            }
        }
    }
}

// ---------------------------------------------------------------- gate and up

// The experts that are used and their tokens, 16 MT at a time, are numbered in
// order; this is what a block needs to find its own: pairs of every expert.
struct Census {
    uint16_t ids[kFewTokens * 32];   // topk_idx, 0xFFFF where masked
    uint32_t pairs[4096];
};

// One block: 16 GU columns of h (those gate and up rows of the weights) for up
// to 16 MT tokens of one expert; NW waves, each with a part of K.  There are at
// most T k such groups of tokens, and at most one for every expert and one more
// for every 16 MT pairs: the grid has no more than that.  (A block for every
// pair, all but the expert's first ending at once, kept their places busy for the
// time of a look at topk_idx: the layer for 64 tokens, 96 experts, top-6, took 201
// us instead of 175, for 32 tokens, 64 experts, top-8, 499 instead of 471.)
template <bool F8, int GU, int MT, int NW, int NB>
__global__ __launch_bounds__(64 * NW) void ep_few_up_kernel(
    FewShape s, const uint16_t *__restrict__ x, const int64_t *__restrict__ idx, const float *__restrict__ w,
    const uint8_t *__restrict__ up, const float *__restrict__ ups, int32_t *count, FewSegment *seg, int32_t *arrived,
    uint16_t *__restrict__ h, int cols) {
    typedef Step<F8, 2 * GU> S;
    constexpr int KE = S::KE, C = S::CHUNKS, BYTES = GU * 4096;   // of a wave's step
    __shared__ __attribute__((aligned(16))) uint8_t buf0[NW * BYTES];
    __shared__ __attribute__((aligned(16))) uint8_t buf1[NW * BYTES];
    static_assert(NB == 2, "as many buffers");
    const auto buf = [&](int j) { return j % NB == 0 ? buf0 : buf1; };
    __shared__ int32_t rows_pair[16 * MT];
    __shared__ float rows_w[16 * MT];
    static_assert(sizeof(Plan) <= sizeof(buf0), "the plan uses the buffer");
    static_assert(64 * NW == kPlanThreads, "the plan's block");

    if (blockIdx.x == 0) {
        make_plan(*reinterpret_cast<Plan *>(buf0), s, idx, count, seg, arrived);
        return;
    }
    const int slot = (blockIdx.x - 1) / cols, n0 = (int)((blockIdx.x - 1) % cols) * 16 * GU;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wid = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r16 = lane & 15, quad = lane >> 4;

    static_assert(sizeof(Census) <= sizeof(buf0), "it uses the buffer");
    Census &c = *reinterpret_cast<Census *>(buf0);
    for (int i = tid; i < s.E; i += 64 * NW) c.pairs[i] = 0;
    __syncthreads();
    for (int i = tid; i < s.T * s.k; i += 64 * NW) {
        const int64_t id = idx[i];
        const bool ok = id >= 0 && id < s.E;
        c.ids[i] = ok ? (uint16_t)id : 0xFFFF;
        if (ok) atomicAdd(&c.pairs[(int)id], 1u);
    }
    __syncthreads();
    // every wave by itself: a run of experts for each lane
    const auto groups = [&](int e) { return (int)((c.pairs[e] + 16 * MT - 1) / (16 * MT)); };
    const int run = (s.E + kWave - 1) / kWave, e0 = min(lane * run, s.E), e1 = min(e0 + run, s.E);
    int own = 0;
    for (int i = e0; i < e1; ++i) own += groups(i);
    int at = scan(own) - own, found = -1, group = 0;
    if (slot >= at && slot < at + own)
        for (int i = e0; i < e1; ++i) {
            const int g = groups(i);
            if (slot < at + g) {
                found = i;
                group = slot - at;
                break;
            }
            at += g;
        }
    const uint64_t finder = __ballot(found >= 0);
    if (finder == 0) return;   // no such group; the same for the whole block
    const int e = __builtin_amdgcn_readlane(found, __builtin_ctzll(finder));
    const int r0 = 16 * MT * __builtin_amdgcn_readlane(group, __builtin_ctzll(finder));

    // the expert's tokens, a lane for each
    int j = -1;
    float wt = 0.0f;
    if (lane < s.T)
        for (int i = 0; i < s.k; ++i)
            if (c.ids[lane * s.k + i] == e) {
                wt = j < 0 ? w[lane * s.k + i] : wt + w[lane * s.k + i];
                j = j < 0 ? i : j;
            }
    const uint64_t has = __ballot(j >= 0);
    const int rank = __popcll(has & lanemask_lt());
    const int rows = min(16 * MT, (int)__popcll(has) - r0);   // below 0 where the pairs were more than the tokens
    if (rows <= 0) return;   // the same for the whole block
    if (wid == 0 && j >= 0 && rank >= r0 && rank < r0 + rows) {
        rows_pair[rank - r0] = lane * s.k + j;
        rows_w[rank - r0] = wt;
    }
    __syncthreads();   // nobody reads the census any more

    const uint32_t kbytes = (uint32_t)s.H * (F8 ? 1 : 2);
    const int KU = (s.H + KE - 1) / KE;
    const int first = KU * wid / NW, n = KU * (wid + 1) / NW - first;

    const uint8_t *we = up + (size_t)e * 2 * s.I * kbytes;
    const int last = s.I - 1 - n0;   // columns past the end repeat the last one
    const rsrc_t gb = buffer(we + (size_t)n0 * kbytes), ub = buffer(we + ((size_t)s.I + n0) * kbytes);
    Stage<2 * GU> st;
    const int srow = lane >> 3;
    st.piece = (uint32_t)(((lane & 7) ^ srow) << 4);
#pragma unroll
    for (int i = 0; i < 4 * GU; ++i) st.off[i] = (uint32_t)min(srow + 8 * (i % (2 * GU)), last) * kbytes;
    const auto stage = [&](uint8_t *buf, int i) {
        const uint32_t k = i < n ? (uint32_t)(first + i) * 128 : 0u;
        st.go(gb, ub, buf + wid * BYTES, k, i < n ? kbytes : 0u);
    };
    // the tokens' rows, straight into the operands' layout
    const rsrc_t xb = buffer(x, (int64_t)s.T * s.H * 2);
    uint32_t xoff[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        xoff[m] = 16 * m + r16 < rows ? (uint32_t)(rows_pair[16 * m + r16] / s.k) * (uint32_t)s.H * 2 : kPast;
    struct Values {
        vec16 v[MT][C];
    };
    const auto load_x = [&](int i, Values &to) {
        const uint32_t k = (uint32_t)(first + i) * (KE * 2);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const uint32_t at = k + S::at(c, quad);
                to.v[m][c] = load_16(xb, i < n && at < (uint32_t)s.H * 2 ? xoff[m] + at : kPast, 0);
            }
    };
    const int KB = s.H / 128;   // scales of a row of blocks
    const rsrc_t sb = buffer(F8 ? ups + (size_t)e * (2 * s.I / 128) * KB : nullptr, F8 ? (int64_t)(2 * s.I / 128) * KB * 4 : 0);
    const uint32_t soff[2] = {(uint32_t)(n0 / 128) * KB * 4, (uint32_t)((s.I + n0) / 128) * KB * 4};
    // of 4 steps at a time; the columns of a block lie in one of the scales' blocks
    f32x4 sc[2] = {}, nsc[2] = {};
    const auto scales = [&](int i) {
        if constexpr (F8)
#pragma unroll
            for (int g = 0; g < 2; ++g) nsc[g] = load_4f32(sb, soff[g] + (uint32_t)(first + i) * 4, 0);
    };

    f32x4 acc[2 * GU][MT] = {};
    const uint32_t plo = (uint32_t)(r16 * 128 + ((quad ^ (r16 & 7)) << 4));
    const auto step = [&](uint8_t *buf, const Values &x, Values &next, int i, int j) {
        wait_step<NB, MT * C, 4 * GU>(i);
        const S a(buf + wid * BYTES, plo);   // the operands are in registers: their place takes the step NB on
        __builtin_amdgcn_sched_barrier(0);
        load_x(i + 1, next);
        if (j == 0) {
#pragma unroll
            for (int g = 0; g < 2; ++g) sc[g] = nsc[g];
            scales(i + 4);
        }
        __builtin_amdgcn_sched_barrier(0);
        stage(buf, i + NB);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (m > 0 && rows <= 16 * m) break;   // the same for the whole block
            f32x4 d[2 * GU];
#pragma unroll
            for (int g = 0; g < 2 * GU; ++g) d[g] = F8 ? f32x4{} : acc[g][m];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const bf16x8 b = __builtin_bit_cast(bf16x8, x.v[m][c]);
#pragma unroll
                for (int g = 0; g < 2 * GU; ++g) d[g] = mfma(a.a[g][c], b, d[g]);
            }
#pragma unroll
            for (int g = 0; g < 2 * GU; ++g)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[g][m][q] = F8 ? __builtin_fmaf(d[g][q], sc[g / GU][j], acc[g][m][q]) : d[g][q];
        }
    };
    Values v[2];
    scales(0);
    stage(buf0, 0);
    __builtin_amdgcn_sched_barrier(0);
    load_x(0, v[0]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 1; j < NB; ++j) stage(buf(j), j);
    for (int i = 0; i < n; i += 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j == 0 || i + j < n) step(buf(j), v[j % 2], v[(j + 1) % 2], i + j, j);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);

    // the parts of K are added in their order
    __syncthreads();
    static_assert(MT <= 2, "they fit");
    constexpr int N = 2 * GU * MT;
    f32x4 *part = reinterpret_cast<f32x4 *>(buf0);
    if (wid > 0)
#pragma unroll
        for (int i = 0; i < N; ++i) part[((wid - 1) * N + i) * kWave + lane] = acc[i / MT][i % MT];
    __syncthreads();
    if (wid > 0) return;
#pragma unroll
    for (int q = 0; q < NW - 1; ++q)
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i / MT][i % MT] += part[(q * N + i) * kWave + lane];
#pragma unroll
    for (int f = 0; f < GU * MT; ++f) {
        const int g = f / MT, m = f % MT;
        const f32x4 v = gates(acc[g][m], acc[GU + g][m]);
        const int r = 16 * m + r16, col = n0 + 16 * g + 4 * quad;
        if (r >= rows || col >= s.I) continue;   // I % 8 == 0: all 4 in or all out
        // h leaves as two bf16 parts, rounded to nearest: 2^-17 of it is lost, at 4
        // bytes a value that the caches hold
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float f = v[q] * rows_w[r];
            hi[q] = take_part(f);
            lo[q] = f32_to_bf16(f);
        }
        uint16_t *o = h + (size_t)rows_pair[r] * 2 * s.I + col;
        *reinterpret_cast<uint2 *>(o) = uint2{hi[0] | hi[1] << 16, hi[2] | hi[3] << 16};
        *reinterpret_cast<uint2 *>(o + s.I) = uint2{lo[0] | lo[1] << 16, lo[2] | lo[3] << 16};
    }
}

// ---------------------------------------------------------------- down

// One block: 16 G columns of y for all tokens.  The steps of all segments (an
// expert's rows of the weights by K = I, for up to 8 RT of its tokens) form one
// list, and each of the NW waves takes an equal run of it, so that every block
// and wave reads the same amount whatever the routing.  A token's two parts of h
// are two columns of the matrix instruction's second operand: 8 tokens an
// instruction.  When a segment ends, its sums go to the lanes that hold the
// tokens' results; the waves' results are added in order at the end.
template <bool F8, int RT, int TT, int G, int NW, int NB>
__global__ __launch_bounds__(64 * NW) void ep_few_down_kernel(
    FewShape s, const int32_t *__restrict__ count, const FewSegment *__restrict__ seg,
    const uint16_t *__restrict__ h, const uint8_t *__restrict__ down, const float *__restrict__ downs,
    const uint16_t *residual, uint16_t *y, int cols, int parts, float *__restrict__ partial,
    int32_t *__restrict__ arrived) {
    typedef Step<F8, G> S;
    constexpr int KE = S::KE, C = S::CHUNKS;
    __shared__ __attribute__((aligned(16))) uint8_t buf0[NW * G * 2048];
    __shared__ __attribute__((aligned(16))) uint8_t buf1[NW * G * 2048];
    __shared__ __attribute__((aligned(16))) uint8_t buf2[NB > 2 ? NW * G * 2048 : 16];
    __shared__ __attribute__((aligned(16))) uint8_t buf3[NB > 3 ? NW * G * 2048 : 16];
    static_assert(NB >= 2 && NB <= 4, "as many buffers");
    const auto buf = [&](int j) {
        return j % NB == 0 ? buf0 : (j % NB == 1 ? buf1 : (j % NB == 2 ? buf2 : buf3));
    };

    const int ct = blockIdx.x % cols, bp = blockIdx.x / cols, n0 = ct * 16 * G;
    __shared__ int last_block;
    const int lane = threadIdx.x & (kWave - 1), wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane & 15, quad = lane >> 4, c8 = r16 & 7, half = r16 >> 3;
    const uint32_t kbytes = (uint32_t)s.I * (F8 ? 1 : 2);
    const int KU = (s.I + KE - 1) / KE;
    const int total = *count * KU;
    const int at = bp * NW + wid, of = parts * NW;
    const int lo = (int)((int64_t)total * at / of), hi = (int)((int64_t)total * (at + 1) / of);

    Stage<G> st;
    const int srow = lane >> 3, last = s.H - 1 - n0;
    st.piece = (uint32_t)(((lane & 7) ^ srow) << 4);
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) st.off[i] = (uint32_t)min(srow + 8 * i, last) * kbytes;
    f32x4 acc[TT][G] = {};
    if (lo < hi) {
        // the weights' place in the list, two steps ahead
        int wg = lo / KU, wu = lo % KU;
        const auto weights = [&](int g) {
            return buffer(down + ((size_t)seg[g].expert * s.H + n0) * kbytes);
        };
        rsrc_t wb = weights(wg);
        const auto stage = [&](uint8_t *buf, int i) {   // steps lo, lo + 1, ... in turn
            st.go(wb, wb, buf + wid * (G * 2048), (uint32_t)wu * 128, i < hi ? kbytes : 0u);
            if (++wu == KU && i + 1 < hi) {
                wu = 0;
                wb = weights(++wg);
            }
        };
        // the tokens' values and the scales, one step ahead
        const rsrc_t hb = buffer(h, (int64_t)s.T * s.k * s.I * 4);
        const int KB = s.I / 128, HB = (s.H + 127) / 128;
        rsrc_t sb;
        int hg = wg, hu = wu, hrows = 0;
        uint32_t hoff[RT];
        const auto segment = [&](int g) {
            hrows = seg[g].rows;
#pragma unroll
            for (int a = 0; a < RT; ++a) {
                uint32_t q[4];   // one load for the wave, then the lane's choice
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = __builtin_amdgcn_readfirstlane(seg[g].pair[4 * a + i]);
                const uint32_t p01 = c8 & 2 ? q[1] : q[0], p23 = c8 & 2 ? q[3] : q[2];
                const uint32_t two = c8 & 4 ? p23 : p01, pair = c8 & 1 ? two >> 16 : two & 0xFFFFu;
                hoff[a] = 8 * a + c8 < hrows ? (pair * 2 + half) * (uint32_t)s.I * 2 : kPast;
            }
            if constexpr (F8) sb = buffer(downs + ((size_t)seg[g].expert * HB + n0 / 128) * KB, KB * 4);
        };
        segment(hg);
        struct Values {
            vec16 v[RT][C];
            float scale;
        };
        const auto load_h = [&](int i, Values &to) {
#pragma unroll
            for (int a = 0; a < RT; ++a) {
                if (a > 0 && hrows <= 8 * a) break;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const uint32_t at = (uint32_t)hu * (KE * 2) + S::at(c, quad);
                    to.v[a][c] = load_16(hb, i < hi && at < (uint32_t)s.I * 2 ? hoff[a] + at : kPast, 0);
                }
            }
            if constexpr (F8) to.scale = load_f32(sb, 0, (uint32_t)min(hu, KB - 1) * 4);
        };

        f32x4 sum[RT][G] = {};
        int g = wg, u = wu, rows = hrows;
        const uint32_t plo = (uint32_t)(r16 * 128 + ((quad ^ (r16 & 7)) << 4));
        const auto finish = [&]() {   // the segment's sums to the tokens' lanes
            const uint64_t tokens = seg[g].tokens;
#pragma unroll
            for (int a = 0; a < RT; ++a)
#pragma unroll
                for (int i = 0; i < G; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) sum[a][i][q] += __shfl_xor(sum[a][i][q], 8);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                if (((tokens >> (8 * t)) & 0xFF) == 0) continue;
                const uint64_t bit = 1ull << (8 * t + c8);
                const int r = __popcll(tokens & (bit - 1));
                const bool in = (tokens & bit) != 0;
#pragma unroll
                for (int i = 0; i < G; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float v = __shfl(sum[0][i][q], quad * 16 + (r & 7));
                        if constexpr (RT > 1) {
                            const float v1 = __shfl(sum[1][i][q], quad * 16 + (r & 7));
                            v = r < 8 ? v : v1;
                        }
                        acc[t][i][q] += in ? v : 0.0f;
                    }
            }
#pragma unroll
            for (int a = 0; a < RT; ++a)
#pragma unroll
                for (int i = 0; i < G; ++i) sum[a][i] = f32x4{};
        };
        const auto step = [&](uint8_t *buf, const Values &x, Values &next, int i) {
            wait_step<NB, C + (F8 ? 1 : 0), 2 * G>(i - lo);
            const uint8_t *p = buf + wid * (G * 2048);
            const S wv(p, plo);
            __builtin_amdgcn_sched_barrier(0);
            if (++hu == KU && i + 1 < hi) {
                hu = 0;
                segment(++hg);
            }
            load_h(i + 1, next);
            __builtin_amdgcn_sched_barrier(0);
            stage(buf, i + NB);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int a = 0; a < RT; ++a) {
                if (a > 0 && rows <= 8 * a) break;
                f32x4 d[G];
#pragma unroll
                for (int f = 0; f < G; ++f) d[f] = F8 ? f32x4{} : sum[a][f];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const bf16x8 b = __builtin_bit_cast(bf16x8, x.v[a][c]);
#pragma unroll
                    for (int f = 0; f < G; ++f) d[f] = mfma(wv.a[f][c], b, d[f]);
                }
#pragma unroll
                for (int f = 0; f < G; ++f)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        sum[a][f][q] = F8 ? __builtin_fmaf(d[f][q], x.scale, sum[a][f][q]) : d[f][q];
            }
            if (++u == KU || i + 1 == hi) {
                finish();
                u = 0;
                ++g;
                rows = hrows;   // the next step's segment
            }
        };
        Values v[2];
        stage(buf0, lo);
        __builtin_amdgcn_sched_barrier(0);
        load_h(lo, v[0]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 1; j < NB; ++j) stage(buf(j), lo + j);
        constexpr int TURN = NB % 2 ? 2 * NB : NB;
        for (int i = lo; i < hi; i += TURN) {
#pragma unroll
            for (int j = 0; j < TURN; ++j)
                if (j == 0 || i + j < hi) step(buf(j), v[j % 2], v[(j + 1) % 2], i + j);
        }
        __builtin_amdgcn_s_waitcnt(0x0F70);
    }

    // add up the waves, in order
    __syncthreads();
    constexpr int TILE = NW * G * 32;   // f32x4 of 8 tokens: [wave][group of columns][quad][token]
    static_assert((TT + 1) / 2 * TILE * 16 <= NW * G * 2048, "they fit in the first two buffers");
    if (half == 0)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int f = 0; f < G; ++f)
                reinterpret_cast<f32x4 *>(t & 1 ? buf1 : buf0)[(t >> 1) * TILE + (wid * G + f) * 32 + quad * 8 + c8] =
                    acc[t][f];
    __syncthreads();
    const auto each = [&](const auto &f) {   // 4 columns of a token: f(their place in the sums, token, column)
        for (int i = threadIdx.x; i < TT * G * 32; i += 64 * NW) {
            const int at = i % (G * 32), t = i / (G * 32), token = 8 * t + at % 8, col = n0 + at / 8 * 4;
            if (token < s.T && col < s.H) f(t, at, (size_t)token * s.H + col);   // H % 8 == 0
        }
    };
    const auto sum_up = [&](int t, int at) {
        const f32x4 *sums = reinterpret_cast<const f32x4 *>(t & 1 ? buf1 : buf0) + (t >> 1) * TILE + at;
        f32x4 v = {};
#pragma unroll
        for (int q = 0; q < NW; ++q) v += sums[q * G * 32];
        return v;
    };
    const auto finish = [&](f32x4 v, size_t o) {
        if (residual) {
            const uint2 r = *reinterpret_cast<const uint2 *>(residual + o);
            v += f32x4{bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y)};
        }
        *reinterpret_cast<uint2 *>(y + o) = uint2{pack_bf16x2_cvt(v[0], v[1]), pack_bf16x2_cvt(v[2], v[3])};
    };
    if (parts == 1) {
        each([&](int t, int at, size_t o) { finish(sum_up(t, at), o); });
        return;
    }
    // The block that is done last adds up the parts, in their order.  The parts
    // go past the XCDs' own L2s by stores and loads of the whole chip's scope:
    // fences would write back and drop those L2s (2 parts of a token's layer: 171
    // us instead of 71).
    const size_t plane = (size_t)s.T * s.H;
    each([&](int t, int at, size_t o) {
        const f32x4 v = sum_up(t, at);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            __hip_atomic_store(partial + bp * plane + o + i, v[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    });
    __builtin_amdgcn_s_waitcnt(0);   // they have arrived where every XCD sees them
    __syncthreads();
    if (threadIdx.x == 0)
        last_block = __hip_atomic_fetch_add(&arrived[ct], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
    __syncthreads();
    if (!last_block) return;
    each([&](int, int, size_t o) {
        f32x4 v = {};
#pragma unroll 4
        for (int q = 0; q < parts; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] += __hip_atomic_load(partial + q * plane + o + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        finish(v, o);
    });
}

struct Work {   // the workspace's parts
    int32_t *count, *arrived;
    FewSegment *seg;
    uint16_t *h;
    float *partial;
    Work(const FewShape &s, uint8_t *ws)
        : count(reinterpret_cast<int32_t *>(ws)), arrived(count + 64), seg(reinterpret_cast<FewSegment *>(ws + kFewHead)),
          h(reinterpret_cast<uint16_t *>(ws + few_h_offset(s))),
          partial(reinterpret_cast<float *>(ws + few_partial_offset(s))) {}
};

template <bool F8, int RT, int TT>
hipError_t launch_down(const FewShape &s, const Work &k, const uint8_t *down, const float *downs,
                       const uint16_t *residual, uint16_t *y, hipStream_t stream) {
    // Half the LDS (two steps ahead, or 4 waves) and twice the blocks: 1 to 9 % faster
    // for large experts of many tokens, 5 to 11 % slower for few tokens or small ones.
    constexpr int G = kFewColumns / 16, NW = 8, NB = 4;
    const int cols = few_columns(s), parts = few_parts(s);
    hipLaunchKernelGGL((ep_few_down_kernel<F8, RT, TT, G, NW, NB>), dim3((unsigned)(cols * parts)), dim3(64 * NW), 0,
                       stream, s, k.count, k.seg, k.h, down, downs, residual, y, cols, parts, k.partial, k.arrived);
    return hipGetLastError();
}

template <bool F8, int GU, int MT, int NW>
hipError_t launch_up(const FewShape &s, const Work &k, const uint16_t *x, const int64_t *idx, const float *w,
                     const uint8_t *up, const float *ups, hipStream_t stream) {
    const int cols = (s.I + 16 * GU - 1) / (16 * GU), pairs = s.T * s.k;
    const int used = pairs < s.E ? pairs : s.E, most = used + pairs / (16 * MT), groups = most < pairs ? most : pairs;
    hipLaunchKernelGGL((ep_few_up_kernel<F8, GU, MT, NW, 2>), dim3((unsigned)(1 + (int64_t)groups * cols)),
                       dim3(64 * NW), 0, stream, s, x, idx, w, up, ups, k.count, k.seg, k.arrived, k.h, cols);
    return hipGetLastError();
}

template <bool F8>
hipError_t launch(const FewShape &s, const uint16_t *x, const int64_t *idx, const float *w, const uint8_t *up,
                  const float *ups, const uint8_t *down, const float *downs, const uint16_t *residual, uint16_t *y,
                  uint8_t *ws, hipStream_t stream) {
    const Work k(s, ws);
    // 32 tokens of an expert at a time where they have more than 8 on average, else 16
    // (the layer, us, 16 / 32 at a time): 64 tokens top-8 of 48 experts 4096 x 1408
    // 197 / 201, of 32 of 4096 x 2048 237 / 224; 48 tokens top-8 of 16, bf16, 236 / 218;
    // 64 tokens top-6 of 96 176 / 183.
    const hipError_t e = s.T * s.k > 8 * s.E ? launch_up<F8, 2, 2, 4>(s, k, x, idx, w, up, ups, stream)
                                             : launch_up<F8, 2, 1, 4>(s, k, x, idx, w, up, ups, stream);
    if (e != hipSuccess) return e;
    if (s.T <= 8) return launch_down<F8, 1, 1>(s, k, down, downs, residual, y, stream);
    if (s.T <= 16) return launch_down<F8, 2, 2>(s, k, down, downs, residual, y, stream);
    if (s.T <= 32) return launch_down<F8, 2, 4>(s, k, down, downs, residual, y, stream);
    return launch_down<F8, 2, 8>(s, k, down, downs, residual, y, stream);
}

}  // namespace

hipError_t launch_few(const FewShape &s, const uint16_t *x, const int64_t *idx, const float *w, const void *up,
                      const float *ups, const void *down, const float *downs, const uint16_t *residual, uint16_t *y,
                      uint8_t *ws, hipStream_t stream) {
    const uint8_t *u = static_cast<const uint8_t *>(up), *d = static_cast<const uint8_t *>(down);
    return s.f8 ? launch<true>(s, x, idx, w, u, ups, d, downs, residual, y, ws, stream)
                : launch<false>(s, x, idx, w, u, ups, d, downs, residual, y, ws, stream);
}

}  // namespace ep
