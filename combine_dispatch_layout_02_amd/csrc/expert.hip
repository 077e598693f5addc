// expert.hip -- the experts' products over fp8 rows, for gfx950: e4m3 rows
// with one fp32 scale per 128 elements times e4m3 weights with one fp32 scale
// per 128 x 128 block, grouped by the experts' row segments.
//
//   y[s, n] = sum_b as[s, b] ws[e, n / 128, b] sum_{i < 128} a[s, 128 b + i] w[e, n, 128 b + i]
//
// The inner sum of one block is one v_mfma_f32_16x16x128_f8f6f4 (products of
// two e4m3 values are exact in binary32); its 4 values per lane are then
// multiplied by the two scales and added to the binary32 accumulator.  The
// weights are the matrix instruction's first operand, the rows its second: a
// lane's 4 values then share one row (lane % 16) and lie at consecutive n, so
// the row's scale is one register per lane and the result one wide store.
#include "ep_device.h"
#include "moe.h"

namespace ep {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// D = A B over 128 e4m3 values per row and column.  Lane l holds 32 bytes of
// row (or column) l % 16; the two operands name their 128 values in the same
// order, whichever it is.  D: row 4 (l / 16) + i, column l % 16.
__device__ __forceinline__ f32x4 mfma_128(i32x8 a, i32x8 b) {
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

// The 8-bit matrix instruction adds 8 products at a time and drops what lies
// below 2^-13 of their largest (measured): over random blocks of 128 the sum is
// off by 1.5e-5 of itself.  That vanishes in a bf16 result (half a step is
// 2^-9 to 2^-8), so ep_expert_gemm takes it.  The gated product hands on its
// groups' scales in binary32; it widens its operands to f16, exactly, and takes
// the 16-bit instruction (8e-9 on the same blocks, measured) at half the rate.
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
struct Wide {
    f16x8 v[4];
};

__device__ __forceinline__ Wide widen(i32x8 b) {
    Wide w;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b[i], 1.0f, false);
        const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b[i], 1.0f, true);
        w.v[i / 2][4 * (i % 2) + 0] = lo[0];
        w.v[i / 2][4 * (i % 2) + 1] = lo[1];
        w.v[i / 2][4 * (i % 2) + 2] = hi[0];
        w.v[i / 2][4 * (i % 2) + 3] = hi[1];
    }
    return w;
}

__device__ __forceinline__ f32x4 mfma_32(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// The operand of a kernel, and MT products of one with MT others, side by side
// so that no instruction waits for the one before it.
template <bool WIDE>
struct Operand;
template <>
struct Operand<false> {
    typedef i32x8 type;
    static __device__ __forceinline__ type make(i32x8 b) { return b; }
    template <int MT>
    static __device__ __forceinline__ void multiply(const type &a, const type (&b)[MT], f32x4 (&d)[MT]) {
#pragma unroll
        for (int m = 0; m < MT; ++m) d[m] = mfma_128(a, b[m]);
    }
};
template <>
struct Operand<true> {
    typedef Wide type;
    static __device__ __forceinline__ type make(i32x8 b) { return widen(b); }
    template <int MT>
    static __device__ __forceinline__ void multiply(const type &a, const type (&b)[MT], f32x4 (&d)[MT]) {
        const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int m = 0; m < MT; ++m) d[m] = mfma_32(a.v[k], b[m].v[k], k ? d[m] : zero);
    }
};

// A lane's 32 bytes of a 128-byte block: 16 at 16 (l / 16), 16 more 64 on, so
// that one load instruction covers whole 64-byte pieces of 16 rows.
__device__ __forceinline__ i32x8 ld_operand(const uint8_t *p) {
    const vec16 lo = ld16(p), hi = ld16(p + 64);
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// The rows of expert e in a and the output, clamped into [0, rows].
__device__ __forceinline__ void expert_rows(const int32_t *off, const ExpertShape &s, int e, int *lo, int *hi) {
    const int rows = (int)s.rows;
    int b = off[e], t = off[e + 1];
    if (s.M > 0) {
        const int r = e / (s.E / s.R), first = off[r * (s.E / s.R)];
        const int end = (r + 1) * s.M;
        b = min(b - first + r * s.M, end);
        t = min(t - first + r * s.M, end);
    }
    b = min(max(b, 0), rows);
    *lo = b;
    *hi = min(max(t, b), rows);
}

// Row tiles of BM rows are numbered without a pass over the experts first:
// expert e's tiles are off[e] / BM + e and on.  As floor((o + n) / BM) + 1 >=
// floor(o / BM) + ceil(n / BM), no two experts share a number, and rows / BM +
// E numbers suffice; those without a tile end at once.  Every thread looks at
// its share of the experts; the one that finds the tile names the expert.
__device__ __forceinline__ bool find_tile(const int32_t *off, const ExpertShape &s, int slot, int BM, int *found,
                                          int *expert, int *row, int *end) {
    if (threadIdx.x == 0) *found = -1;
    __syncthreads();
    for (int e = threadIdx.x; e < s.E; e += blockDim.x) {
        int lo, hi;
        expert_rows(off, s, e, &lo, &hi);
        const int first = max(off[e], 0) / BM + e;
        if (slot >= first && slot - first < (hi - lo + BM - 1) / BM) *found = e;
    }
    __syncthreads();
    const int e = *found;
    if (e < 0) return false;
    int lo, hi;
    expert_rows(off, s, e, &lo, &hi);
    const int r0 = lo + (slot - (max(off[e], 0) / BM + e)) * BM;
    *expert = e;
    *row = r0;
    *end = hi;
    return r0 >= lo && r0 < hi;   // offsets that do not ascend: no tile
}

// h = g / (1 + e^-g) u
__device__ __forceinline__ float gate(float g, float u) { return g / (1.0f + expf(-g)) * u; }

constexpr int kColWaves = 8;   // waves side by side: 16 weight rows twice each

// BM = 16 MT rows by 256 weight rows (gated: 128 columns of gate and the same
// 128 of up, one scale group of the result), K split over KS waves whose
// parts are added in LDS in wave order.  Operands go straight from memory to
// registers.
template <int MT, int KS, bool GATED>
__global__ __launch_bounds__(64 * kColWaves * KS) void ep_expert_stream_kernel(
    ExpertShape s, const int32_t *off, const uint8_t *a, const float *as, const uint8_t *w, const float *ws,
    uint16_t *out, uint8_t *oq, float *oqs) {
    __shared__ int found;
    __shared__ f32x4 part[KS > 1 ? KS - 1 : 1][KS > 1 ? kColWaves : 1][KS > 1 ? 2 * MT : 1][kWave];
    __shared__ float amax[GATED ? kColWaves : 1][GATED ? 16 * MT : 1];
    typedef Operand<GATED> Op;
    int e, row, end;
    if (!find_tile(off, s, blockIdx.x, 16 * MT, &found, &e, &row, &end)) return;

    const int lane = threadIdx.x & (kWave - 1), wid = threadIdx.x / kWave;
    const int col = wid % kColWaves, ks = wid / kColWaves;
    const int r16 = lane & 15, quad = lane >> 4;
    const int KB = s.K / 128;
    const int wrows = GATED ? 2 * s.N : s.N;
    // the two groups of 16 weight rows of this wave
    const int n0 = GATED ? (int)blockIdx.y * 128 + col * 16 : (int)blockIdx.y * 256 + col * 32;
    const int n1 = GATED ? n0 + s.N : n0 + 16;
    const uint8_t *we = w + (size_t)e * wrows * s.K;
    const float *wse = ws + (size_t)e * ((wrows + 127) / 128) * KB;
    const uint8_t *w0 = we + (size_t)min(n0 + r16, wrows - 1) * s.K + quad * 16;
    const uint8_t *w1 = we + (size_t)min(n1 + r16, wrows - 1) * s.K + quad * 16;
    const float *ws0 = wse + (size_t)(min(n0, wrows - 1) / 128) * KB;
    const float *ws1 = wse + (size_t)(min(n1, wrows - 1) / 128) * KB;
    const uint8_t *ap[MT];
    const float *asp[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int r = min(row + 16 * m + r16, end - 1);   // rows past the segment repeat its last one
        ap[m] = a + (size_t)r * s.K + quad * 16;
        asp[m] = as + (size_t)r * KB;
    }

    f32x4 acc[2][MT] = {};
    const int kb0 = KB * ks / KS, kb1 = KB * (ks + 1) / KS;
    for (int kb = kb0; kb < kb1; ++kb) {
        const auto f0 = Op::make(ld_operand(w0 + (size_t)kb * 128)), f1 = Op::make(ld_operand(w1 + (size_t)kb * 128));
        const float c0 = ws0[kb], c1 = ws1[kb];
        typename Op::type x[MT];
        float sc[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            x[m] = Op::make(ld_operand(ap[m] + (size_t)kb * 128));
            sc[m] = asp[m][kb];
        }
        f32x4 d0[MT], d1[MT];
        Op::multiply(f0, x, d0);
        Op::multiply(f1, x, d1);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const float s0 = sc[m] * c0, s1 = sc[m] * c1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[0][m][i] = __builtin_fmaf(d0[m][i], s0, acc[0][m][i]);
                acc[1][m][i] = __builtin_fmaf(d1[m][i], s1, acc[1][m][i]);
            }
        }
    }
    if constexpr (KS > 1) {
        if (ks > 0)
#pragma unroll
            for (int m = 0; m < 2 * MT; ++m) part[ks - 1][col][m][lane] = acc[m & 1][m >> 1];
        __syncthreads();
        if (ks == 0)
#pragma unroll
            for (int p = 0; p < KS - 1; ++p)
#pragma unroll
                for (int m = 0; m < 2 * MT; ++m) acc[m & 1][m >> 1] += part[p][col][m][lane];
    }

    if constexpr (!GATED) {
        if (ks > 0) return;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = row + 16 * m + r16;
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const int n = n0 + 16 * f + 4 * quad;   // N % 8 == 0: all 4 in or all out
                if (r >= end || n >= s.N) continue;
                uint2 v;
                v.x = pack_bf16x2(acc[f][m][0], acc[f][m][1]);
                v.y = pack_bf16x2(acc[f][m][2], acc[f][m][3]);
                *reinterpret_cast<uint2 *>(out + (size_t)r * s.N + n) = v;
            }
        }
    } else {
        f32x4 h[MT];
        if (ks == 0) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[m][i] = gate(acc[0][m][i], acc[1][m][i]);
                    top = fmaxf(top, fabsf(h[m][i]));
                }
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                if (quad == 0) amax[col][16 * m + r16] = top;
            }
        }
        __syncthreads();
        if (ks > 0) return;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = row + 16 * m + r16;
            float top = 0.0f;
#pragma unroll
            for (int c = 0; c < kColWaves; ++c) top = fmaxf(top, amax[c][16 * m + r16]);
            const float scale = (top == 0.0f) ? 1.0f : top / 448.0f;
            uint32_t q = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) q |= f32_to_e4m3(h[m][i] / scale) << (8 * i);
            if (r >= end) continue;
            *reinterpret_cast<uint32_t *>(oq + (size_t)r * s.N + n0 + 4 * quad) = q;
            if (col == 0 && quad == 0) oqs[(size_t)r * (s.N / 128) + blockIdx.y] = scale;
        }
    }
}

// ---------------------------------------------------------------- many rows

constexpr int kTileThreads = 512, kTileN = 256;   // 8 waves; weight rows of a tile

typedef __amdgpu_buffer_rsrc_t rsrc_t;

// Buffers of at most 2^31 bytes from a wave-uniform base: a load is then one
// 32-bit register of offset per lane and a scalar one per block of K.
__device__ __forceinline__ rsrc_t buffer(const void *p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, 0x7FFFFFFF, 0x00020000);
}

// 16 bytes per lane from memory into LDS at base + 16 lane, without a register.
__device__ __forceinline__ void load_to_lds(rsrc_t b, uint8_t *lds, uint32_t off, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void *)lds, 16, (int)off, (int)soff,
                                             0, 0);
}

__device__ __forceinline__ float load_f32(rsrc_t b, uint32_t off, uint32_t soff) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(b, (int)off, (int)soff, 0));
}

// A lane's 32 bytes of a row of a tile in LDS, given where its two pieces lie.
// Rows are 128 bytes, and their 16-byte pieces are permuted by the row (piece c
// lies at c ^ (r % 8)), so that the 8 lanes of one LDS cycle touch every bank
// once; rows 16 apart have the same permutation.
__device__ __forceinline__ i32x8 lds_operand(const uint8_t *lo16, const uint8_t *hi16) {
    const vec16 lo = ld16(lo16), hi = ld16(hi16);
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// One block: BM rows by 256 weight rows (gated: 128 gate rows and the matching
// 128 up rows), 8 waves, WN of them side by side.  Both operands of a block of
// K = 128 are staged in LDS, two buffers in turn: the next block's loads are
// in flight while this one is multiplied.
template <int BM, int WN, bool GATED>
__global__ __launch_bounds__(kTileThreads) void ep_expert_tile_kernel(
    ExpertShape s, const int32_t *off, const uint8_t *a, const float *as, const uint8_t *w, const float *ws,
    uint16_t *out, uint8_t *oq, float *oqs, int slots, int cols) {
    constexpr int WM = 8 / WN, NF = kTileN / WN / 16, MF = BM / WM / 16;
    constexpr int HALF = GATED ? 2 : 1;            // gate and up, or one product
    constexpr int WCOLS = kTileN / HALF / WN;      // columns of the result per wave
    typedef Operand<GATED> Op;
    __shared__ __attribute__((aligned(16))) uint8_t buf0[(kTileN + BM) * 128];
    __shared__ __attribute__((aligned(16))) uint8_t buf1[(kTileN + BM) * 128];
    __shared__ int found;
    __shared__ float amax[GATED ? WN : 1][GATED ? BM : 1];

    // consecutive blocks go to the 8 XCDs in turn; each XCD takes a contiguous
    // eighth of the tiles, 8 row tiles by all columns at a time, so that the
    // 32 blocks it runs together share their operands in its L2
    const int tile = (int)blockIdx.x;
    const int per = 8 * cols, sb = tile / per, in = tile % per;
    const int slot = sb * 8 + in % 8, ct = in / 8;
    if (slot >= slots) return;
    int e, row, end;
    if (!find_tile(off, s, slot, BM, &found, &e, &row, &end)) return;

    const int lane = threadIdx.x & (kWave - 1), wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wn = wid % WN, wm = wid / WN;
    const int r16 = lane & 15, quad = lane >> 4;
    const int KB = s.K / 128;
    const int wrows = HALF * s.N;
    const int n0 = ct * (kTileN / HALF);           // first column of the result
    const uint8_t *we = w + (size_t)e * wrows * s.K;
    const float *wse = ws + (size_t)e * ((wrows + 127) / 128) * KB;

    // staging: pass p of the block covers 64 rows, a wave 8 of them
    const int srow = wid * 8 + (lane >> 3);                    // + 64 p
    const uint32_t piece = (uint32_t)(((lane & 7) ^ (srow & 7)) << 4);
    // gated: all 128 rows of gate and of up are there, 64 rows on is a scalar
    // offset; else the last tile's rows past the end repeat the last one
    uint32_t woff[GATED ? 1 : kTileN / 64], xoff[BM / 64];
#pragma unroll
    for (int p = 0; p < (GATED ? 1 : kTileN / 64); ++p)
        woff[p] = (uint32_t)(GATED ? srow : min(srow + 64 * p, wrows - 1 - n0)) * (uint32_t)s.K + piece;
#pragma unroll
    for (int p = 0; p < BM / 64; ++p)
        xoff[p] = (uint32_t)min(srow + 64 * p, end - 1 - row) * (uint32_t)s.K + piece;
    const uint8_t *w0 = we + (size_t)n0 * s.K;
    const rsrc_t wb0 = buffer(w0), wb1 = buffer(GATED ? w0 + (size_t)s.N * s.K : w0);
    const rsrc_t xb = buffer(a + (size_t)row * s.K);

    constexpr int PIECES = (kTileN + BM) / 64;
    const auto stage = [&](uint8_t *buf, int kb, int p) {   // piece p of a block of K
        if (GATED && p < kTileN / 64)
            load_to_lds(p < 2 ? wb0 : wb1, buf + p * 8192 + wid * 1024, woff[0], (p & 1) * 64 * s.K + kb * 128);
        else if (p < kTileN / 64)
            load_to_lds(wb0, buf + p * 8192 + wid * 1024, woff[p], kb * 128);
        else
            load_to_lds(xb, buf + p * 8192 + wid * 1024, xoff[p - kTileN / 64], kb * 128);
    };

    // scales: one register per lane and group of 16 rows, one (or gate's and
    // up's) per wave, loaded a block ahead
    const rsrc_t asb = buffer(as + (size_t)row * KB), wsb = buffer(wse);
    uint32_t asoff[MF], wsoff[HALF];
#pragma unroll
    for (int m = 0; m < MF; ++m)
        asoff[m] = (uint32_t)min(wm * 16 * MF + 16 * m + r16, end - 1 - row) * (uint32_t)KB * 4;
#pragma unroll
    for (int h = 0; h < HALF; ++h)
        wsoff[h] = (uint32_t)(min(n0 + h * s.N + wn * WCOLS, wrows - 1) / 128) * (uint32_t)KB * 4;

    f32x4 acc[NF][MF] = {};
    float sx[MF], sw[HALF];
    const auto scales = [&](int kb) {
#pragma unroll
        for (int m = 0; m < MF; ++m) sx[m] = load_f32(asb, asoff[m], kb * 4);
#pragma unroll
        for (int h = 0; h < HALF; ++h) sw[h] = load_f32(wsb, wsoff[h], kb * 4);
    };
    const uint32_t plo = (uint32_t)((quad ^ (r16 & 7)) << 4), phi = plo ^ 64;
    const uint32_t wlo = (uint32_t)(wn * WCOLS + r16) * 128 + plo, whi = (uint32_t)(wn * WCOLS + r16) * 128 + phi;
    const uint32_t xrow = (uint32_t)(kTileN + wm * 16 * MF + r16) * 128;
    const uint32_t xlo = xrow + plo, xhi = xrow + phi;
    const auto multiply = [&](const uint8_t *buf, const float (&x)[MF], const float (&c)[HALF], const auto &between) {
        typename Op::type xf[MF];
#pragma unroll
        for (int m = 0; m < MF; ++m) xf[m] = Op::make(lds_operand(buf + xlo + 2048 * m, buf + xhi + 2048 * m));
        const auto weights = [&](int n) {
            const int at = GATED ? n / (NF / 2) * 128 * 128 + 2048 * (n % (NF / 2)) : 2048 * n;
            return lds_operand(buf + wlo + at, buf + whi + at);
        };
        const auto add = [&](int n, const f32x4 (&d)[MF]) {
#pragma unroll
            for (int m = 0; m < MF; ++m) {
                const float sc = x[m] * c[GATED ? n / (NF / 2) : 0];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][m][i] = __builtin_fmaf(d[m][i], sc, acc[n][m][i]);
                asm volatile("" : "+v"(acc[n][m]));   // added here, not sunk into the next block of K
            }
        };
        i32x8 wf = weights(0);
        f32x4 last[MF];
#pragma unroll
        for (int n = 0; n < NF; ++n) {
            // the next weights are on their way and the last products are being
            // scaled while these are multiplied; the fence keeps the scheduler
            // from fetching all of them at once
            const i32x8 wnext = weights(n + 1 < NF ? n + 1 : n);
            f32x4 d[MF];
            Op::multiply(Op::make(wf), xf, d);
            between(n);
            if constexpr (GATED) {   // no registers to spare for a second set of products
                add(n, d);
            } else {
                if (n > 0) add(n - 1, last);
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);   // 2 reads of LDS, then in turn
#pragma unroll
                for (int m = 0; m < MF; ++m) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // a matrix instruction
                    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);   // and 4 vector ones
                }
#pragma unroll
                for (int m = 0; m < MF; ++m) last[m] = d[m];
            }
            __builtin_amdgcn_sched_barrier(0);
            wf = wnext;
        }
        if constexpr (!GATED) add(NF - 1, last);
    };
    // The next block's loads are issued a few at a time between the matrix
    // instructions: all at once they fill the memory pipe's queue and every
    // wave waits at the start of the block.  The last block loads itself again
    // (a branch here would cost registers).
    const auto step = [&](const uint8_t *cur, uint8_t *next, int kb) {
        float x[MF], c[HALF];
#pragma unroll
        for (int m = 0; m < MF; ++m) x[m] = sx[m];
#pragma unroll
        for (int h = 0; h < HALF; ++h) c[h] = sw[h];
        __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): this wave's part of the block has arrived
        __syncthreads();                      // every wave's part; and the other buffer is free
        const int after = min(kb + 1, KB - 1);
        scales(after);
        multiply(cur, x, c, [&](int n) {
#pragma unroll
            for (int p = n * PIECES / NF; p < (n + 1) * PIECES / NF; ++p) stage(next, after, p);
        });
    };
#pragma unroll
    for (int p = 0; p < PIECES; ++p) stage(buf0, 0, p);
    scales(0);
    for (int kb = 0; kb < KB; kb += 2) {
        step(buf0, buf1, kb);
        if (kb + 1 < KB) step(buf1, buf0, kb + 1);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);

    if constexpr (!GATED) {
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            const int r = row + wm * 16 * MF + 16 * m + r16;
#pragma unroll
            for (int n = 0; n < NF; ++n) {
                const int c = n0 + wn * WCOLS + 16 * n + 4 * quad;   // N % 8 == 0: all 4 in or all out
                if (r >= end || c >= s.N) continue;
                uint2 v;
                v.x = pack_bf16x2(acc[n][m][0], acc[n][m][1]);
                v.y = pack_bf16x2(acc[n][m][2], acc[n][m][3]);
                *reinterpret_cast<uint2 *>(out + (size_t)r * s.N + c) = v;
            }
        }
    } else {
        // h takes the place of the gate's accumulators
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            float top = 0.0f;
#pragma unroll
            for (int n = 0; n < NF / 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[n][m][i] = gate(acc[n][m][i], acc[n + NF / 2][m][i]);
                    top = fmaxf(top, fabsf(acc[n][m][i]));
                }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            if (quad == 0) amax[wn][wm * 16 * MF + 16 * m + r16] = top;
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            const int i = wm * 16 * MF + 16 * m + r16, r = row + i;
            float top = 0.0f;
#pragma unroll
            for (int c = 0; c < WN; ++c) top = fmaxf(top, amax[c][i]);
            const float scale = (top == 0.0f) ? 1.0f : top / 448.0f;
            if (r >= end) continue;
#pragma unroll
            for (int n = 0; n < NF / 2; ++n) {
                uint32_t q = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) q |= f32_to_e4m3(acc[n][m][j] / scale) << (8 * j);
                *reinterpret_cast<uint32_t *>(oq + (size_t)r * s.N + n0 + wn * WCOLS + 16 * n + 4 * quad) = q;
            }
            if (wn == 0 && quad == 0) oqs[(size_t)r * (s.N / 128) + ct] = scale;
        }
    }
}

constexpr int kStreamMT = 4, kStreamKS = 1;

int64_t tile_slots(const ExpertShape &s, int BM) { return s.rows / BM + s.E; }

}  // namespace

bool expert_grid_fits(const ExpertShape &s, bool gated) {
    const int64_t cols = gated ? s.N / 128 : (s.N + 255) / 256;
    return cols <= 65535 && tile_slots(s, 16) * 1024 < (int64_t(1) << 32);
}

namespace {

template <int BM, int WN, bool GATED>
hipError_t launch_tile(const ExpertShape &s, const int32_t *offset, const uint8_t *a, const float *as,
                       const uint8_t *w, const float *ws, uint16_t *out, uint8_t *q, float *qs, hipStream_t stream) {
    const int slots = (int)tile_slots(s, BM), cols = GATED ? s.N / 128 : (s.N + kTileN - 1) / kTileN;
    const int64_t blocks = (int64_t)((slots + 7) / 8) * 8 * cols;
    hipLaunchKernelGGL((ep_expert_tile_kernel<BM, WN, GATED>), dim3((unsigned)blocks), dim3(kTileThreads), 0, stream,
                       s, offset, a, as, w, ws, out, q, qs, slots, cols);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_gemm(const ExpertShape &s, const int32_t *offset, const uint8_t *a, const float *as,
                              const uint8_t *w, const float *ws, uint16_t *out, hipStream_t stream) {
    if (s.rows / s.E >= 64) return launch_tile<256, 2, false>(s, offset, a, as, w, ws, out, nullptr, nullptr, stream);
    const dim3 grid((unsigned)tile_slots(s, 16 * kStreamMT), (unsigned)((s.N + 255) / 256));
    hipLaunchKernelGGL((ep_expert_stream_kernel<kStreamMT, kStreamKS, false>), grid,
                       dim3(kWave * kColWaves * kStreamKS), 0, stream, s, offset, a, as, w, ws, out, nullptr, nullptr);
    return hipGetLastError();
}

hipError_t launch_expert_gated(const ExpertShape &s, const int32_t *offset, const uint8_t *a, const float *as,
                               const uint8_t *w, const float *ws, uint8_t *q, float *qs, hipStream_t stream) {
    if (s.rows / s.E >= 64) return launch_tile<256, 2, true>(s, offset, a, as, w, ws, nullptr, q, qs, stream);
    const dim3 grid((unsigned)tile_slots(s, 16 * kStreamMT), (unsigned)(s.N / 128));
    hipLaunchKernelGGL((ep_expert_stream_kernel<kStreamMT, kStreamKS, true>), grid,
                       dim3(kWave * kColWaves * kStreamKS), 0, stream, s, offset, a, as, w, ws, nullptr, q, qs);
    return hipGetLastError();
}

}  // namespace ep
