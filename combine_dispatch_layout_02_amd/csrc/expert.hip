// expert.hip -- the experts' products over fp8 rows, for gfx950: e4m3 rows
// with one fp32 scale per 128 elements times e4m3 weights with one fp32 scale
// per 128 x 128 block, grouped by the experts' row segments.
//
//   y[s, n] = sum_b as[s, b] ws[e, n / 128, b] sum_{i < 128} a[s, 128 b + i] w[e, n, 128 b + i]
//
// The inner sum of one block is one v_mfma_f32_16x16x128_f8f6f4, or 16-bit
// matrix instructions on operands widened exactly (see below); its 4 values per
// lane are then multiplied by the two scales and added to the binary32
// accumulator.  The
// weights are the matrix instruction's first operand, the rows its second: a
// lane's 4 values then share one row (lane % 16) and lie at consecutive n, so
// the row's scale is one register per lane and the result one wide store.
#include "ep_device.h"
#include "moe.h"
#include "tile_order.h"

namespace ep {
namespace {

constexpr int kTileThreads = 512, kTileN = 256;   // of the tiled forms: 8 waves; weight rows of a tile

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
    static __device__ __forceinline__ void multiply(const type (&a)[2], const type &b, f32x4 (&d)[2]) {
        d[0] = mfma_128(a[0], b);
        d[1] = mfma_128(a[1], b);
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
    static __device__ __forceinline__ void multiply(const type (&a)[2], const type &b, f32x4 (&d)[2]) {
        const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int f = 0; f < 2; ++f) d[f] = mfma_32(a[f].v[k], b.v[k], k ? d[f] : zero);
    }
};

typedef __amdgpu_buffer_rsrc_t rsrc_t;

// A barrier that waits for the waves alone: __syncthreads also waits for every
// load on its way to LDS.  What a wave needs of those it waits for itself.
__device__ __forceinline__ void barrier_only() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// A buffer of `bytes` bytes (2^31 - 1 at most) from a wave-uniform base: a load
// is then one 32-bit register of offset per lane and a scalar one per block of
// K, and reads 0 past the end.
__device__ __forceinline__ rsrc_t buffer(const void *p, int64_t bytes = 0x7FFFFFFF) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0,
                                             (int)(bytes < 0x7FFFFFFF ? bytes : 0x7FFFFFFF), 0x00020000);
}

// 16 bytes per lane from memory into LDS at base + 16 lane, without a register.
__device__ __forceinline__ void load_to_lds(rsrc_t b, uint8_t *lds, uint32_t off, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void *)lds, 16, (int)off, (int)soff,
                                             0, 0);
}

__device__ __forceinline__ float load_f32(rsrc_t b, uint32_t off, uint32_t soff) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(b, (int)off, (int)soff, 0));
}

__device__ __forceinline__ f32x4 load_4f32(rsrc_t b, uint32_t off, uint32_t soff) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, (int)soff, 0));
}

// A lane's 32 bytes of a row of a tile in LDS, given where its two pieces lie.
// Rows are 128 bytes, and their 16-byte pieces are permuted by the row (piece c
// lies at c ^ (r % 8)), so that the 8 lanes of one LDS cycle touch every bank
// once; rows 16 apart have the same permutation.
__device__ __forceinline__ i32x8 lds_operand(const uint8_t *lo16, const uint8_t *hi16) {
    const vec16 lo = ld16(lo16), hi = ld16(hi16);
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// A lane's 4 bf16 at columns 4 quad of one group of 16 columns (a) and of the
// next (b), quad = lane / 16, become 8 of one of them: lanes of odd quads hand
// over their a for the b of the quad before.  A store is then 16 bytes a lane
// and 64 a row (with 8 and 32, 32768 rows of 7168 took 40 us more).
__device__ __forceinline__ vec16 eight(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1) {
    const auto s0 = __builtin_amdgcn_permlane16_swap(a0, b0, false, false);
    const auto s1 = __builtin_amdgcn_permlane16_swap(a1, b1, false, false);
    return vec16{s0[0], s1[0], s0[1], s1[1]};
}
// The first of those columns, from the first of a's group.
__device__ __forceinline__ int column8(int quad) { return 16 * (quad & 1) + 8 * (quad >> 1); }

// The rows of expert e in a and the output, clamped into [0, rows].
__device__ __forceinline__ void expert_rows(const int32_t *off, const ExpertShape &s, int e, int *lo, int *hi) {
    const int rows = (int)s.rows;
    int64_t b = off[e], t = off[e + 1];
    if (s.M > 0) {
        const int r = e / (s.E / s.R), first = off[r * (s.E / s.R)];
        const int64_t shift = (int64_t)r * s.M - first, end = (int64_t)(r + 1) * s.M;
        b = min(b + shift, end);
        t = min(t + shift, end);
    }
    *lo = (int)min(max(b, (int64_t)0), (int64_t)rows);
    *hi = (int)min(max(t, (int64_t)*lo), (int64_t)rows);
}

// Row tiles of BM rows are numbered without a pass over the experts first:
// expert e's tiles are lo / BM + e and on, lo its first row.  As floor((o + n) /
// BM) + 1 >= floor(o / BM) + ceil(n / BM), no two experts share a number, and
// rows / BM + E numbers suffice; those without a tile end at once.  Every thread looks at
// its share of the experts; the one that finds the tile names the expert.
__device__ __forceinline__ bool find_tile(const int32_t *off, const ExpertShape &s, int slot, int BM, int *found,
                                          int *expert, int *row, int *end) {
    if (threadIdx.x == 0) *found = -1;
    __syncthreads();
    for (int e = threadIdx.x; e < s.E; e += blockDim.x) {
        int lo, hi;
        expert_rows(off, s, e, &lo, &hi);
        const int first = lo / BM + e;
        if (slot >= first && slot - first < (hi - lo + BM - 1) / BM) *found = e;
    }
    __syncthreads();
    const int e = *found;
    if (e < 0) return false;
    int lo, hi;
    expert_rows(off, s, e, &lo, &hi);
    const int r0 = lo + (slot - (lo / BM + e)) * BM;
    *expert = e;
    *row = r0;
    *end = hi;
    return r0 >= lo && r0 < hi;   // offsets that do not ascend: no tile
}

// The tile of this block among those that have rows, in TileOrder's order: the
// experts' tiles are counted and added up over the block, a run of experts per
// thread, and the thread whose run holds the tile names it.  Offsets that do not
// ascend: the counts saturate, and every row stays one of the buffer's.
struct TileSearch {
    int expert, row, end;
    int sums[kTileThreads / kWave];   // of the waves
};
__device__ __forceinline__ bool order_tile(const int32_t *off, const ExpertShape &s, int BM, int cols,
                                           TileSearch *found, int *expert, int *row, int *end, int *col) {
    const auto add = [](int a, int b) { return min(a + b, 1 << 30); };
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wid = tid / kWave;
    const int run = (s.E + kTileThreads - 1) / kTileThreads, e0 = tid * run, e1 = min(e0 + run, s.E);
    int mine = 0, lo = 0, hi = 0;
    for (int e = e0; e < e1; ++e) {
        expert_rows(off, s, e, &lo, &hi);
        mine = add(mine, (hi - lo + BM - 1) / BM);
    }
    // up to and with this thread: inside rows of 16 lanes, across them, across the waves
    int upto = mine;
    upto = add(upto, __builtin_amdgcn_update_dpp(0, upto, 0x111, 0xf, 0xf, false));
    upto = add(upto, __builtin_amdgcn_update_dpp(0, upto, 0x112, 0xf, 0xf, false));
    upto = add(upto, __builtin_amdgcn_update_dpp(0, upto, 0x114, 0xf, 0xf, false));
    upto = add(upto, __builtin_amdgcn_update_dpp(0, upto, 0x118, 0xf, 0xf, false));
    upto = add(upto, __builtin_amdgcn_update_dpp(0, upto, 0x142, 0xa, 0xf, false));
    upto = add(upto, __builtin_amdgcn_update_dpp(0, upto, 0x143, 0xc, 0xf, false));
    if (tid == 0) found->expert = -1;
    if (lane == kWave - 1) found->sums[wid] = upto;
    __syncthreads();
    int total = 0, before = 0;
#pragma unroll
    for (int i = 0; i < kTileThreads / kWave; ++i) {
        if (i == wid) before = total;
        total = add(total, found->sums[i]);
    }
    upto = add(upto, before);
    total = __builtin_amdgcn_readfirstlane(total);
    int slot;
    if (!TileOrder{total, cols}.tile(blockIdx.x, &slot, col)) return false;   // the same for the whole block
    int at = upto - mine;
    if (slot >= at && slot < upto) {
        int e = e0;
        if (run > 1)   // else lo and hi are the expert's
            for (; e < e1; ++e) {
                expert_rows(off, s, e, &lo, &hi);
                const int n = (hi - lo + BM - 1) / BM;
                if (slot - at < n) break;
                at += n;
            }
        found->expert = min(e, s.E - 1);
        found->row = lo + (slot - at) * BM;
        found->end = hi;
    }
    __syncthreads();
    *expert = __builtin_amdgcn_readfirstlane(found->expert);
    *row = __builtin_amdgcn_readfirstlane(found->row);
    *end = __builtin_amdgcn_readfirstlane(found->end);
    return *expert >= 0 && *row >= 0 && *row < *end;
}

// h = g / (1 + e^-g) u, for negative g as g e^g / (1 + e^g) u: what is divided
// by lies in [1, 2].  Below -80, where e^g nears binary32's smallest values, it
// is taken as the square of y = e^(g/2), with u multiplied in between: h keeps
// its precision however small e^g is (1 + e^g is 1 there; y itself leaves the
// normal range at g = -174, where |h| < 2^-116 for any u).  The hardware's
// reciprocal is within one step, so h is off by 5 steps at most: 1 of expf (2 of
// its square), 1 of the reciprocal, half of the sum and of the three products
// each; and by half the smallest subnormal where h is subnormal itself.
template <bool DEEP>
__device__ __forceinline__ float gate(float g, float u) {
    const bool deep = DEEP && g < -80.0f;
    const float x = expf(deep ? 0.5f * g : -__builtin_fabsf(g)), r = __builtin_amdgcn_rcpf(1.0f + x);
    return deep ? g * x * u * x : g * (g >= 0.0f ? r : x * r) * u;
}
// A lane's values; a wave without such gates does not pay for the choice (32
// values a lane, 5 % of a tile's time at K = 1024).
template <typename V>
__device__ __forceinline__ V gates(V g, V u) {
    constexpr int n = sizeof(V) / sizeof(float);
    float least = g[0];
#pragma unroll
    for (int i = 1; i < n; ++i) least = fminf(least, g[i]);
    V h;
    if (__ballot(least < -80.0f) == 0) {
#pragma unroll
        for (int i = 0; i < n; ++i) h[i] = gate<false>(g[i], u[i]);
    } else {
#pragma unroll
        for (int i = 0; i < n; ++i) h[i] = gate<true>(g[i], u[i]);
    }
    return h;
}

// A group's scale: its largest magnitude / 448, 1 for zeros.  Where the quotient
// would round to 0 it is the smallest subnormal, so that the bytes still hold h
// to e4m3's precision and nothing is divided by 0.
__device__ __forceinline__ float group_scale(float top) { return top == 0.0f ? 1.0f : fmaxf(top / 448.0f, 0x1p-149f); }

// Four values over their group's scale, as e4m3 bytes.  The quotients are those
// of the IEEE division: a correctly rounded reciprocal and one correction of the
// quotient by its remainder, a third of its instructions, and at the ends of the
// range the division itself.  The conversion makes NaN of what would round past
// 448.  A normal scale is within half a step of the largest magnitude / 448, so
// quotients stay below 464 and round to 448 at most; a subnormal one may have
// lost a third of its value, so there they are clamped (a NaN stays).
struct Divisor {
    float scale, inv;
    bool plain;
    __device__ __forceinline__ explicit Divisor(float s) : scale(s), inv(1.0f / s), plain(s > 0x1p-100f && s < 0x1p100f) {}
    __device__ __forceinline__ float corrected(float h) const {
        const float q = h * inv;
        return __builtin_fmaf(__builtin_fmaf(-q, scale, h), inv, q);
    }
    __device__ __forceinline__ float clamped(float h) const {
        const float q = h / scale;
        return q > 448.0f ? 448.0f : (q < -448.0f ? -448.0f : q);
    }
    __device__ __forceinline__ uint32_t quantise(float a, float b, float c, float d) const {
        if (plain) {
            a = corrected(a), b = corrected(b), c = corrected(c), d = corrected(d);
        } else {
            a = clamped(a), b = clamped(b), c = clamped(c), d = clamped(d);
        }
        const int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
    }
};

// ---------------------------------------------------------------- few rows

// BM = 16 MT rows by 32 CW weight rows (gated: CW = 8, 128 columns of gate and
// the same 128 of up, one scale group of the result), CW waves side by side
// with 16 weight rows twice each, K split over KS groups of them whose parts
// are added in LDS in their order.  Here the weights are what
// counts: each is read once.  Loading them straight into the operands' layout
// costs the address unit a cycle per lane pair, as neighbouring lanes hold
// different rows, and bounds the kernel at a third of the memory rate; so each
// wave copies its 32 weight rows' next block of K (4 KiB, whole 128-byte
// lines) into its own part of LDS and reads the operands from there, with two
// blocks in flight and no barrier.  The rows of a are shared by the waves: XB
// blocks of K at a time, two buffers, a barrier per change.
// Bound by the weights' bytes: gated, 1024 rows over 256 experts, K = 7168,
// 4096 weight rows (7.4 GB) 1200 us, 6.2 TB/s of the 6.8 a stream of reads
// reaches; 8 rows of 8 experts (235 MB) 55 us, 4.3 TB/s, of which about 10 us
// are the launch, the first loads and the sum of the parts of K.
template <int MT, int CW, int KS, bool GATED>
__global__ __attribute__((amdgpu_waves_per_eu(4, 4)))
__launch_bounds__(64 * CW * KS) void ep_expert_stream_kernel(
    ExpertShape s, const int32_t *off, const uint8_t *a, const float *as, const uint8_t *w, const float *ws,
    uint16_t *out, uint8_t *oq, float *oqs, int cols) {
    constexpr int XB = KS > 2 ? 1 : 2;           // blocks of K of a's rows per change
    constexpr int XBYTES = 16 * MT * 128 * XB;   // 2, 4 or 8 KiB
    static_assert(!GATED || CW == 8, "a scale group of the result per block");
    static_assert(XBYTES <= 1024 * CW, "one piece of a's rows per wave");
    __shared__ __attribute__((aligned(16))) uint8_t wbuf0[CW * KS * 4096];
    __shared__ __attribute__((aligned(16))) uint8_t wbuf1[CW * KS * 4096];
    __shared__ __attribute__((aligned(16))) uint8_t xbuf0[KS * XBYTES];
    __shared__ __attribute__((aligned(16))) uint8_t xbuf1[KS * XBYTES];
    // two blocks share a CU's 160 KiB to the byte: the tile's expert and the
    // groups' maxima use the buffers before and after
    int *found = reinterpret_cast<int *>(xbuf0);
    float (*amax)[16 * MT] = reinterpret_cast<float (*)[16 * MT]>(wbuf1);
    typedef Operand<GATED> Op;
    int e, row, end;
    // columns first: an expert's blocks spread over the XCDs, also where only a
    // few experts have rows
    const int ct = blockIdx.x % cols;
    if (!find_tile(off, s, blockIdx.x / cols, 16 * MT, found, &e, &row, &end)) return;
    __syncthreads();   // everyone has read it

    const int lane = threadIdx.x & (kWave - 1), wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int col = wid % CW, ks = wid / CW;
    const int r16 = lane & 15, quad = lane >> 4;
    const int KB = s.K / 128;
    const int wrows = GATED ? 2 * s.N : s.N;
    // the two groups of 16 weight rows of this wave
    const int n0 = GATED ? ct * 128 + col * 16 : (ct * CW + col) * 32;
    const int n1 = GATED ? n0 + s.N : n0 + 16;
    const uint8_t *we = w + (size_t)e * wrows * s.K;
    const float *wse = ws + (size_t)e * ((wrows + 127) / 128) * KB;
    // this wave's blocks of K; every group walks `steps` of them (barriers)
    const int first = KB * ks / KS, n = KB * (ks + 1) / KS - first, steps = (KB + KS - 1) / KS;

    // staging: instruction i of a wave covers 8 rows, 8 lanes each
    const int srow = lane >> 3;
    const uint32_t piece = (uint32_t)(((lane & 7) ^ srow) << 4);
    const int m0 = min(n0, wrows - 1), m1 = min(n1, wrows - 1);   // rows past the end repeat the last one
    const rsrc_t wb0 = buffer(we + (size_t)m0 * s.K), wb1 = buffer(we + (size_t)m1 * s.K);
    uint32_t woff[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        woff[i] = (uint32_t)min(srow + 8 * (i & 1), wrows - 1 - (i < 2 ? m0 : m1)) * (uint32_t)s.K + piece;
    // a block past the last is read from past the buffer's end: zeros, no memory
    // traffic, and the same count of loads under way in every step
    const auto past = [&](int i) { return i < n ? 0u : 0x80000000u; };
    const auto stage_w = [&](uint8_t *buf, int i) {
        const uint32_t k = (uint32_t)(first + i) * 128;
#pragma unroll
        for (int p = 0; p < 4; ++p)
            load_to_lds(p < 2 ? wb0 : wb1, buf + wid * 4096 + p * 1024, woff[p] | past(i), k);
    };
    // a's rows: [block of K][row][128 bytes], 8 lines per wave (where there are
    // fewer pieces than waves, two waves bring the same one)
    const rsrc_t xb = buffer(a + (size_t)row * s.K);
    constexpr int PIECES = XBYTES / 1024;
    const int xline = col % PIECES * 8 + srow, xr = xline % (16 * MT), xblock = xline / (16 * MT);
    const uint32_t xoff = (uint32_t)min(xr, end - 1 - row) * (uint32_t)s.K + (uint32_t)xblock * 128 +
                          (uint32_t)(((lane & 7) ^ (xr & 7)) << 4);
    const auto stage_x = [&](uint8_t *buf, int i) {   // blocks i .. i + XB - 1 of K
        load_to_lds(xb, buf + ks * XBYTES + col % PIECES * 1024, xoff | past(i + xblock), (uint32_t)(first + i) * 128);
    };
    // scales, four blocks of K at a time
    const rsrc_t asb = buffer(as + (size_t)row * KB, (s.rows - row) * KB * 4);
    const rsrc_t wsb = buffer(wse, (int64_t)((wrows + 127) / 128) * KB * 4);
    uint32_t asoff[MT], wsoff[2];
#pragma unroll
    for (int m = 0; m < MT; ++m) asoff[m] = (uint32_t)min(16 * m + r16, end - 1 - row) * (uint32_t)KB * 4;
    wsoff[0] = (uint32_t)(m0 / 128) * (uint32_t)KB * 4;
    wsoff[1] = (uint32_t)(m1 / 128) * (uint32_t)KB * 4;

    const uint32_t plo = (uint32_t)(r16 * 128 + ((quad ^ (r16 & 7)) << 4)), phi = plo ^ 64;
    f32x4 acc[2][MT] = {};
    f32x4 cx[MT], cw[2], nx[MT], nw[2];
    const auto scales = [&](int i) {
        const uint32_t k = (uint32_t)(first + i) * 4;
#pragma unroll
        for (int m = 0; m < MT; ++m) nx[m] = load_4f32(asb, asoff[m] | past(i), k);
        nw[0] = load_4f32(wsb, wsoff[0] | past(i), k);
        nw[1] = load_4f32(wsb, wsoff[1] | past(i), k);
    };
    const auto step = [&](uint8_t *wbuf, const uint8_t *xbuf, int i, int part, int j) {
        // this block of weights has arrived: the wait before the change of a's
        // rows covers it, or 5 later loads to LDS may be under way, the next
        // block's and one piece of a's rows (other loads only add to those)
        if (part > 0) {
            __builtin_amdgcn_s_waitcnt(0x0F75);   // vmcnt(5)
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        }
        const uint8_t *wp = wbuf + wid * 4096;
        const i32x8 f0 = lds_operand(wp + plo, wp + phi), f1 = lds_operand(wp + 2048 + plo, wp + 2048 + phi);
        const typename Op::type wf[2] = {Op::make(f0), Op::make(f1)};
        // the operands are in registers: their place takes the block after next
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        __builtin_amdgcn_sched_barrier(0);
        stage_w(wbuf, i + 2);
        __builtin_amdgcn_sched_barrier(0);
        const uint8_t *xp = xbuf + ks * XBYTES + part * (16 * MT * 128);
        i32x8 xr = lds_operand(xp + plo, xp + phi);
#pragma unroll
        for (int m = 0; m < MT; ++m) {   // one group of rows at a time: few registers, two blocks to a CU
            const auto x = Op::make(xr);
            if (m + 1 < MT) xr = lds_operand(xp + 2048 * (m + 1) + plo, xp + 2048 * (m + 1) + phi);
            f32x4 d[2];
            Op::multiply(wf, x, d);
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const float sc = cx[m][j] * cw[f][j];
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[f][m][q] = __builtin_fmaf(d[f][q], sc, acc[f][m][q]);
                asm volatile("" : "+v"(acc[f][m]));   // added here, not after the next loads
            }
        }
    };
    const auto group = [&](int i, bool whole) {   // four blocks of K
#pragma unroll
        for (int m = 0; m < MT; ++m) cx[m] = nx[m];
        cw[0] = nw[0];
        cw[1] = nw[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (!whole && i + j >= steps) break;
            if (j % XB == 0) {
                // a's rows for this change have arrived in every wave (behind
                // them only the next block of weights may be under way: 4
                // loads); the other buffer is free
                __builtin_amdgcn_s_waitcnt(0x0F74);   // vmcnt(4)
                barrier_only();
                stage_x((j / XB) % 2 ? xbuf0 : xbuf1, i + j + XB);
            }
            if (whole || i + j < n)   // wave-uniform
                step(j % 2 ? wbuf1 : wbuf0, (j / XB) % 2 ? xbuf1 : xbuf0, i + j, j % XB, j);
            else
                __builtin_amdgcn_s_waitcnt(0x0F70);
            if (j == 0) scales(i + 4);
        }
    };
    stage_w(wbuf0, 0);
    stage_x(xbuf0, 0);
    scales(0);
    stage_w(wbuf1, 1);
    int i = 0;
    for (; i + 4 <= KB / KS; i += 4) group(i, true);
    if (i < steps) group(i, false);
    __builtin_amdgcn_s_waitcnt(0x0F70);

    if constexpr (KS > 1) {
        // the parts of K, in the place of the weights
        static_assert((KS - 1) * 2 * MT * 1024 <= KS * 4096, "they fit");
        __syncthreads();
        f32x4 *part = reinterpret_cast<f32x4 *>(wbuf0);
        if (ks > 0)
#pragma unroll
            for (int m = 0; m < 2 * MT; ++m)
                part[(((ks - 1) * CW + col) * 2 * MT + m) * kWave + lane] = acc[m & 1][m >> 1];
        __syncthreads();
        if (ks == 0)
#pragma unroll
            for (int p = 0; p < KS - 1; ++p)
#pragma unroll
                for (int m = 0; m < 2 * MT; ++m)
                    acc[m & 1][m >> 1] += part[((p * CW + col) * 2 * MT + m) * kWave + lane];
    }

    if constexpr (!GATED) {
        if (ks > 0) return;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = row + 16 * m + r16;
            float v[8];
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = acc[i / 4][m][i % 4];
            pack_bf16(v, o);
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const int n = n0 + 16 * f + 4 * quad;   // N % 8 == 0: all 4 in or all out
                if (r >= end || n >= s.N) continue;
                *reinterpret_cast<uint2 *>(out + (size_t)r * s.N + n) = uint2{o[2 * f], o[2 * f + 1]};
            }
        }
    } else {
        f32x4 h[MT];
        float tops[MT];
        if (ks == 0) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float top = 0.0f;
                h[m] = gates(acc[0][m], acc[1][m]);
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(h[m][i]));
                top = fmaxf(top, __shfl_xor(top, 16));
                tops[m] = fmaxf(top, __shfl_xor(top, 32));
            }
        }
        __syncthreads();   // nobody reads the buffers any more
        if (ks == 0 && quad == 0)
#pragma unroll
            for (int m = 0; m < MT; ++m) amax[col][16 * m + r16] = tops[m];
        __syncthreads();
        if (ks > 0) return;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = row + 16 * m + r16;
            float top = 0.0f;
#pragma unroll
            for (int c = 0; c < CW; ++c) top = fmaxf(top, amax[c][16 * m + r16]);
            const float scale = group_scale(top);
            if (r >= end) continue;
            *reinterpret_cast<uint32_t *>(oq + (size_t)r * s.N + n0 + 4 * quad) =
                Divisor(scale).quantise(h[m][0], h[m][1], h[m][2], h[m][3]);
            if (col == 0 && quad == 0) oqs[(size_t)r * (s.N / 128) + ct] = scale;
        }
    }
}

// ---------------------------------------------------------------- many rows

// One block: BM rows by 256 weight rows, 8 waves, 2 by 4.  Blocks of K = 128 of
// both operands are staged in LDS: the weights in three buffers, two blocks on,
// a's rows in three or, at 256 rows, two, which fills the LDS.
// Bound by the latency of those loads: 32768 rows, 32 experts, K = 2048, 7168
// weight rows 625 to 644 us on two cards, 1.5 PFLOP/s (weights one block on only
// 680).  Timed apart, on the form before with 680 us: without the products 626,
// without the loads 487, without the result's stores 571.
template <int BM>
__global__ __launch_bounds__(kTileThreads) void ep_expert_tile_kernel(
    ExpertShape s, const int32_t *off, const uint8_t *a, const float *as, const uint8_t *w, const float *ws,
    uint16_t *out, int slots, int cols) {
    constexpr int WN = 2, WM = 4, NF = kTileN / WN / 16, MF = BM / WM / 16;
    constexpr int XS = BM <= 128 ? 3 : 2;          // buffers of a's rows: what 160 KiB of LDS hold
    __shared__ __attribute__((aligned(16))) uint8_t wbuf0[kTileN * 128];
    __shared__ __attribute__((aligned(16))) uint8_t wbuf1[kTileN * 128];
    __shared__ __attribute__((aligned(16))) uint8_t wbuf2[kTileN * 128];
    __shared__ __attribute__((aligned(16))) uint8_t xbuf0[BM * 128];
    __shared__ __attribute__((aligned(16))) uint8_t xbuf1[BM * 128];
    int *found = reinterpret_cast<int *>(xbuf0);   // before the buffers, which may fill the LDS to the byte

    // 8 row tiles by all columns at a time, a row tile's columns on one XCD
    // (an eighth of the tiles to each XCD, as the gated tiles have it, is slower: 760 us
    // against 689; so are 8 row tiles by an eighth of the columns, 712 against 682)
    const int per = 8 * cols, sb = blockIdx.x / per, in = blockIdx.x % per;
    const int slot = sb * 8 + in % 8, ct = in / 8;
    if (slot >= slots) return;
    int e, row, end;
    if (!find_tile(off, s, slot, BM, found, &e, &row, &end)) return;
    __syncthreads();   // everyone has read it

    const int lane = threadIdx.x & (kWave - 1), wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wn = wid % WN, wm = wid / WN;
    const int r16 = lane & 15, quad = lane >> 4;
    const int KB = s.K / 128;
    const int n0 = ct * kTileN;                    // first column of the result
    const uint8_t *w0 = w + ((size_t)e * s.N + n0) * s.K;
    const float *wse = ws + (size_t)e * ((s.N + 127) / 128) * KB;

    // staging: pass p of the block covers 64 rows, a wave 8 of them
    const int srow = wid * 8 + (lane >> 3);                    // + 64 p
    const uint32_t piece = (uint32_t)(((lane & 7) ^ (srow & 7)) << 4);
    // rows past the last repeat it
    uint32_t woff[kTileN / 64], xoff[BM / 64];
#pragma unroll
    for (int p = 0; p < kTileN / 64; ++p)
        woff[p] = (uint32_t)min(srow + 64 * p, s.N - 1 - n0) * (uint32_t)s.K + piece;
#pragma unroll
    for (int p = 0; p < BM / 64; ++p)
        xoff[p] = (uint32_t)min(srow + 64 * p, end - 1 - row) * (uint32_t)s.K + piece;
    const rsrc_t wb = buffer(w0), xb = buffer(a + (size_t)row * s.K);

    constexpr int WP = kTileN / 64, XP = BM / 64, PIECES = WP + XP;
    const auto stage_w = [&](uint8_t *buf, int kb, int p) {   // piece p of a block of K of the weights
        load_to_lds(wb, buf + p * 8192 + wid * 1024, woff[p] | (kb < KB ? 0u : 0x80000000u), kb * 128);
    };
    const auto stage_x = [&](uint8_t *buf, int kb, int p) {   // and of a's rows
        load_to_lds(xb, buf + p * 8192 + wid * 1024, xoff[p] | (kb < KB ? 0u : 0x80000000u), kb * 128);
    };

    // scales: one register per lane and group of 16 rows, one per wave (its 128
    // weight rows are one block of theirs), loaded a block ahead
    const rsrc_t asb = buffer(as + (size_t)row * KB), wsb = buffer(wse);
    uint32_t asoff[MF];
#pragma unroll
    for (int m = 0; m < MF; ++m)
        asoff[m] = (uint32_t)min(wm * 16 * MF + 16 * m + r16, end - 1 - row) * (uint32_t)KB * 4;
    const uint32_t wsoff = (uint32_t)(min(n0 + wn * 128, s.N - 1) / 128) * (uint32_t)KB * 4;

    f32x4 acc[NF][MF] = {};
    float sx[MF], sw;
    const auto scales = [&](int kb) {
#pragma unroll
        for (int m = 0; m < MF; ++m) sx[m] = load_f32(asb, asoff[m], kb * 4);
        sw = load_f32(wsb, wsoff, kb * 4);
    };
    const uint32_t plo = (uint32_t)((quad ^ (r16 & 7)) << 4), phi = plo ^ 64;
    const uint32_t wlo = (uint32_t)(wn * 128 + r16) * 128 + plo, whi = wlo ^ 64;
    const uint32_t xrow = (uint32_t)(wm * 16 * MF + r16) * 128;
    const uint32_t xlo = xrow + plo, xhi = xrow + phi;
    const auto multiply = [&](const uint8_t *wbuf, const uint8_t *xbuf, const float (&x)[MF], float c, const auto &between) {
        i32x8 xf[MF];
#pragma unroll
        for (int m = 0; m < MF; ++m) xf[m] = lds_operand(xbuf + xlo + 2048 * m, xbuf + xhi + 2048 * m);
        const auto weights = [&](int n) { return lds_operand(wbuf + wlo + 2048 * n, wbuf + whi + 2048 * n); };
        const auto add = [&](int n, const f32x4 (&d)[MF]) {
#pragma unroll
            for (int m = 0; m < MF; ++m) {
                const float sc = x[m] * c;
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][m][i] = __builtin_fmaf(d[m][i], sc, acc[n][m][i]);
                asm volatile("" : "+v"(acc[n][m]));   // added here, not sunk into the next block of K
            }
        };
        // While the products with weights n run, those after next are on their
        // way and the last products are scaled.  The fences keep the scheduler
        // from fetching everything at once.
        i32x8 wf[2] = {weights(0), weights(1)};
        f32x4 last[MF];
#pragma unroll
        for (int n = 0; n < NF; ++n) {
            const i32x8 wnext = weights(n + 2 < NF ? n + 2 : NF - 1);
            f32x4 d[MF];
            Operand<false>::multiply(wf[0], xf, d);
            if (n > 0) add(n - 1, last);
            between(n);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);   // 2 reads of LDS, then in turn
#pragma unroll
            for (int m = 0; m < MF; ++m) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // a matrix instruction
                __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);   // and 4 vector ones
            }
            __builtin_amdgcn_sched_barrier(0);
            wf[0] = wf[1];
            wf[1] = wnext;
#pragma unroll
            for (int m = 0; m < MF; ++m) last[m] = d[m];
        }
        add(NF - 1, last);
    };
    // The loads of later blocks are issued a few at a time between the matrix
    // instructions: all at once they fill the memory pipe's queue and every wave
    // waits.  Past the last block they read past the buffer's end (zeros, no
    // memory traffic), which keeps the counts of the waits.
    const auto step = [&](const uint8_t *wcur, const uint8_t *xcur, uint8_t *wnext, uint8_t *xnext, int kb) {
        // this wave's part of the block has arrived, of what came later at most
        // the weights two blocks on (with three buffers of a's rows, and those)
        // are under way; then every wave's part, and the buffers of the block
        // before are free
        __builtin_amdgcn_s_waitcnt(0x0F70 | (XS == 3 ? PIECES : WP));
        barrier_only();
        float x[MF];
        const float c = sw;
#pragma unroll
        for (int m = 0; m < MF; ++m) x[m] = sx[m];
        scales(min(kb + 1, KB - 1));
        __builtin_amdgcn_sched_barrier(0);
        multiply(wcur, xcur, x, c, [&](int n) {
#pragma unroll
            for (int p = n * PIECES / NF; p < (n + 1) * PIECES / NF; ++p)
                if (p < XP)
                    stage_x(xnext, kb + XS - 1, p);
                else
                    stage_w(wnext, kb + 2, p - XP);
        });
    };
    scales(0);
#pragma unroll
    for (int p = 0; p < WP; ++p) stage_w(wbuf0, 0, p);
#pragma unroll
    for (int p = 0; p < XP; ++p) stage_x(xbuf0, 0, p);
    if (XS == 3)
#pragma unroll
        for (int p = 0; p < XP; ++p) stage_x(xbuf1, 1, p);
#pragma unroll
    for (int p = 0; p < WP; ++p) stage_w(wbuf1, 1, p);
    if constexpr (XS == 3) {
        __shared__ __attribute__((aligned(16))) uint8_t xbuf2[BM * 128];
        for (int kb = 0; kb < KB; kb += 3) {
            step(wbuf0, xbuf0, wbuf2, xbuf2, kb);
            if (kb + 1 < KB) step(wbuf1, xbuf1, wbuf0, xbuf0, kb + 1);
            if (kb + 2 < KB) step(wbuf2, xbuf2, wbuf1, xbuf1, kb + 2);
        }
    } else {
        for (int kb = 0; kb < KB; kb += 6) {
            step(wbuf0, xbuf0, wbuf2, xbuf1, kb);
            if (kb + 1 < KB) step(wbuf1, xbuf1, wbuf0, xbuf0, kb + 1);
            if (kb + 2 < KB) step(wbuf2, xbuf0, wbuf1, xbuf1, kb + 2);
            if (kb + 3 < KB) step(wbuf0, xbuf1, wbuf2, xbuf0, kb + 3);
            if (kb + 4 < KB) step(wbuf1, xbuf0, wbuf0, xbuf1, kb + 4);
            if (kb + 5 < KB) step(wbuf2, xbuf1, wbuf1, xbuf0, kb + 5);
        }
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);

#pragma unroll
    for (int m = 0; m < MF; ++m) {
        const int r = row + wm * 16 * MF + 16 * m + r16;
        float v[4 * NF];
        uint32_t o[2 * NF];
#pragma unroll
        for (int i = 0; i < 4 * NF; ++i) v[i] = acc[i / 4][m][i % 4];
        pack_bf16(v, o);
#pragma unroll
        for (int n = 0; n < NF; n += 2) {
            const vec16 v = eight(o[2 * n], o[2 * n + 1], o[2 * n + 2], o[2 * n + 3]);
            const int c = n0 + wn * 128 + 16 * n + column8(quad);   // N % 8 == 0: all 8 in or all out
            if (r < end && c < s.N) st16(out + (size_t)r * s.N + c, v);
        }
    }
}

// ---------------------------------------------------------------- many rows, 16-bit products

typedef float f32x16 __attribute__((ext_vector_type(16)));

// 16 bytes of e4m3 as two operands of the 32 x 32 x 16 instruction.
struct Pair {
    f16x8 v[2];
};
__device__ __forceinline__ Pair widen16(vec16 b) {
    Pair w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)b[i], 1.0f, false);
        const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)b[i], 1.0f, true);
        w.v[i / 2][4 * (i % 2) + 0] = lo[0];
        w.v[i / 2][4 * (i % 2) + 1] = lo[1];
        w.v[i / 2][4 * (i % 2) + 2] = hi[0];
        w.v[i / 2][4 * (i % 2) + 3] = hi[1];
    }
    return w;
}

// The permutation of a row's pieces where 32 lanes read 32 rows: a 16-byte read
// takes lanes 0-3, 12-15, 20-27 in one cycle and the others of 32 in the next,
// and bits 1, 3 and 4 of the row tell the 8 rows of one parity in each apart
// (with the rows' last three bits, at 32768 rows, 126 million conflicts of
// banks and 1948 us; so none and 1930 us).
__device__ __forceinline__ int place32(int r) { return ((r >> 1) & 1) | ((r >> 2) & 6); }

// The gated product in tiles of 128 rows by 128 gate and the matching 128 up
// rows: 8 waves, 4 by 2, each 32 gate and 32 up rows by 64 rows of a.  The
// widening and the scaling take 3 vector instructions for every 16 cycles of
// matrix instructions; beside 16 x 16 x 32 ones two of those are free, beside
// 32 x 32 x 16 ones, half as many to issue, three (measured: 19.5 against 24
// cycles).  Three buffers of LDS: two blocks of K are under way.
// Bound by the 16-bit matrix instructions (busy for 0.59 of the time) with the
// vector ones beside them: 32768 rows, 32 experts, K = 7168, 4096 weight rows
// 1890 to 1960 us on two cards, 1.0 PFLOP/s; with 16 x 16 x 32 instructions 2040.
__global__ __launch_bounds__(kTileThreads) void ep_expert_gated_tile_kernel(
    ExpertShape s, const int32_t *off, const uint8_t *a, const float *as, const uint8_t *w, const float *ws,
    uint8_t *oq, float *oqs, int cols) {
    constexpr int BM = 128, WN = 4, PIECES = (kTileN + BM) / 64, BYTES = (kTileN + BM) * 128;
    __shared__ __attribute__((aligned(16))) uint8_t buf0[BYTES];
    __shared__ __attribute__((aligned(16))) uint8_t buf1[BYTES];
    __shared__ __attribute__((aligned(16))) uint8_t buf2[BYTES];
    __shared__ TileSearch found;
    __shared__ float amax[WN][BM];

    int row, ct, e, end;
    if (!order_tile(off, s, BM, cols, &found, &e, &row, &end, &ct)) return;

    const int lane = threadIdx.x & (kWave - 1), wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wn = wid % WN, wm = wid / WN;
    const int r32 = lane & 31, half = lane >> 5;
    const int KB = s.K / 128;
    const uint8_t *we = w + ((size_t)e * 2 * s.N + (size_t)ct * 128) * s.K;   // N % 128 == 0: all 128 rows are there
    const float *wse = ws + (size_t)e * (2 * s.N / 128) * KB;

    const int srow = wid * 8 + (lane >> 3);                    // + 64 p
    const uint32_t piece = (uint32_t)(((lane & 7) ^ place32(srow)) << 4);
    const uint32_t woff = (uint32_t)srow * (uint32_t)s.K + piece;
    uint32_t xoff[BM / 64];
#pragma unroll
    for (int p = 0; p < BM / 64; ++p)
        xoff[p] = (uint32_t)min(srow + 64 * p, end - 1 - row) * (uint32_t)s.K + piece;
    const rsrc_t wb0 = buffer(we), wb1 = buffer(we + (size_t)s.N * s.K), xb = buffer(a + (size_t)row * s.K);
    const auto stage = [&](uint8_t *buf, int kb, int p) {   // piece p of a block of K
        const uint32_t past = kb < KB ? 0u : 0x80000000u;
        if (p < kTileN / 64)
            load_to_lds(p < 2 ? wb0 : wb1, buf + p * 8192 + wid * 1024, woff | past, (p & 1) * 64 * s.K + kb * 128);
        else
            load_to_lds(xb, buf + p * 8192 + wid * 1024, xoff[p - kTileN / 64] | past, kb * 128);
    };

    const rsrc_t asb = buffer(as + (size_t)row * KB), wsb = buffer(wse);
    uint32_t asoff[2], wsoff[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) asoff[m] = (uint32_t)min(wm * 64 + 32 * m + r32, end - 1 - row) * (uint32_t)KB * 4;
#pragma unroll
    for (int f = 0; f < 2; ++f) wsoff[f] = (uint32_t)(ct + f * (s.N / 128)) * (uint32_t)KB * 4;
    float sx[2], sw[2];
    const auto scales = [&](int kb) {
#pragma unroll
        for (int m = 0; m < 2; ++m) sx[m] = load_f32(asb, asoff[m], kb * 4);
#pragma unroll
        for (int f = 0; f < 2; ++f) sw[f] = load_f32(wsb, wsoff[f], kb * 4);
    };

    // a lane's 16 bytes of quarter q of a row: piece 2 q + half, permuted by the row
    const uint32_t wrow = (uint32_t)(wn * 32 + r32) * 128, xrow = (uint32_t)(kTileN + wm * 64 + r32) * 128;
    const uint32_t p0 = (uint32_t)((half ^ place32(r32)) << 4);
    vec16 raw[4];      // gate, up, two groups of rows of a: the quarter after the next
    Pair o[4];         // the next quarter, widened
    const auto read = [&](const uint8_t *buf, int q) {
        const uint32_t p = p0 ^ (uint32_t)(q << 5);
        raw[0] = ld16(buf + wrow + p);
        raw[1] = ld16(buf + wrow + p + 128 * 128);
        raw[2] = ld16(buf + xrow + p);
        raw[3] = ld16(buf + xrow + p + 32 * 128);
    };
    f32x16 acc[2][2] = {}, d[2][2] = {};
    float x[2] = {}, c[2] = {};
    const auto add = [&](int t) {   // the sums of the last block, scaled
        const float sc = x[t >> 1] * c[t & 1];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            acc[t & 1][t >> 1][i] = __builtin_fmaf(d[t & 1][t >> 1][i], sc, acc[t & 1][t >> 1][i]);
        asm volatile("" : "+v"(acc[t & 1][t >> 1]));   // added here, not later
    };
    // The quarters of all blocks form one chain: while one is multiplied, the
    // next is widened and the one after that read from LDS, across the change
    // of the block too, so that nothing waits for LDS behind a barrier.
    const auto step = [&](const uint8_t *cur, const uint8_t *after, uint8_t *next, int kb) {
        float nx[2], nc[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) nx[m] = sx[m], nc[m] = sw[m];
        scales(min(kb + 1, KB - 1));
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q == 2) {
                // from here on the next block is read: it has arrived in every
                // wave (of later loads, the 4 pieces staged above may be under
                // way), and every wave has read the last of this one, whose
                // buffer is filled again from the next step on
                __builtin_amdgcn_s_waitcnt(0x0074);   // lgkmcnt(0), vmcnt(4)
                barrier_only();
            }
            Pair n[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) n[i] = widen16(raw[i]);
            read(q < 2 ? cur : after, (q + 2) % 4);
            if (q < 3)
#pragma unroll
                for (int p = q * 2; p < q * 2 + 2; ++p) stage(next, kb + 2, p);
            const f32x16 zero = {};
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if (q + k == 0) add(t);
                    d[t & 1][t >> 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(o[t & 1].v[k], o[2 + (t >> 1)].v[k],
                                                                              q + k ? d[t & 1][t >> 1] : zero, 0, 0, 0);
                }
            if (q > 0) {
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // a matrix instruction
                    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);   // and 4 vector ones
                }
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = n[i];
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) x[m] = nx[m], c[m] = nc[m];
    };
    static_assert(PIECES == 6, "two pieces in each of the first three quarters");
#pragma unroll
    for (int p = 0; p < PIECES; ++p) stage(buf0, 0, p);
    scales(0);
#pragma unroll
    for (int p = 0; p < PIECES; ++p) stage(buf1, 1, p);
    __builtin_amdgcn_s_waitcnt(0x0F70 | PIECES);
    barrier_only();
    read(buf0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = widen16(raw[i]);
    read(buf0, 1);
    for (int kb = 0; kb < KB; kb += 3) {
        step(buf0, buf1, buf2, kb);
        if (kb + 1 < KB) step(buf1, buf2, buf0, kb + 1);
        if (kb + 2 < KB) step(buf2, buf0, buf1, kb + 2);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);
#pragma unroll
    for (int t = 0; t < 4; ++t) add(t);

    // value i of a lane: column 8 (i / 4) + 4 half + i % 4, row r32 of each group
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        float top = 0.0f;
        acc[0][m] = gates(acc[0][m], acc[1][m]);
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(acc[0][m][i]));
        top = fmaxf(top, __shfl_xor(top, 32));
        if (half == 0) amax[wn][wm * 64 + 32 * m + r32] = top;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int i = wm * 64 + 32 * m + r32, r = row + i;
        const float top = fmaxf(fmaxf(amax[0][i], amax[1][i]), fmaxf(amax[2][i], amax[3][i]));
        const float scale = group_scale(top);
        if (r >= end) continue;
        uint8_t *o = oq + (size_t)r * s.N + ct * 128 + wn * 32 + 4 * half;
        const Divisor by(scale);
#pragma unroll
        for (int g = 0; g < 4; ++g)
            *reinterpret_cast<uint32_t *>(o + 8 * g) = by.quantise(acc[0][m][4 * g], acc[0][m][4 * g + 1],
                                                                   acc[0][m][4 * g + 2], acc[0][m][4 * g + 3]);
        if (wn == 0 && half == 0) oqs[(size_t)r * (s.N / 128) + ct] = scale;
    }
}

int64_t tile_slots(const ExpertShape &s, int BM) { return s.rows / BM + s.E; }

}  // namespace

// The widest grid is that of the 32-row form (the ones with narrower blocks are
// taken for a few hundred of them only).
bool expert_grid_fits(const ExpertShape &s, bool gated) {
    const int64_t cols = gated ? s.N / 128 : (s.N + 255) / 256;
    return (tile_slots(s, 32) + 8) * cols * kTileThreads < (int64_t(1) << 32);
}

namespace {

template <int BM>
hipError_t launch_tile(const ExpertShape &s, const int32_t *offset, const uint8_t *a, const float *as,
                       const uint8_t *w, const float *ws, uint16_t *out, hipStream_t stream) {
    const int slots = (int)tile_slots(s, BM), cols = (s.N + kTileN - 1) / kTileN;
    const int64_t blocks = (int64_t)((slots + 7) / 8) * 8 * cols;
    hipLaunchKernelGGL(ep_expert_tile_kernel<BM>, dim3((unsigned)blocks), dim3(kTileThreads), 0, stream, s, offset, a,
                       as, w, ws, out, slots, cols);
    return hipGetLastError();
}

hipError_t launch_gated_tile(const ExpertShape &s, const int32_t *offset, const uint8_t *a, const float *as,
                             const uint8_t *w, const float *ws, uint8_t *q, float *qs, hipStream_t stream) {
    const int slots = (int)tile_slots(s, 128), cols = s.N / 128;
    hipLaunchKernelGGL(ep_expert_gated_tile_kernel, dim3((unsigned)TileOrder::blocks(slots, cols)),
                       dim3(kTileThreads), 0, stream, s, offset, a, as, w, ws, q, qs, cols);
    return hipGetLastError();
}

template <int MT, int CW, int KS, bool GATED>
hipError_t launch_stream(const ExpertShape &s, const int32_t *offset, const uint8_t *a, const float *as,
                         const uint8_t *w, const float *ws, uint16_t *out, uint8_t *q, float *qs, hipStream_t stream) {
    const int cols = GATED ? s.N / 128 : (s.N + 32 * CW - 1) / (32 * CW);
    hipLaunchKernelGGL((ep_expert_stream_kernel<MT, CW, KS, GATED>), dim3((unsigned)(tile_slots(s, 16 * MT) * cols)),
                       dim3(kWave * CW * KS), 0, stream, s, offset, a, as, w, ws, out, q, qs, cols);
    return hipGetLastError();
}

// Which form: by the rows of an expert on average, as if they filled the buffer
// (the host knows no counts), and by how many blocks come of it (16 rows against
// 256 weight rows each where rows are few; partial tiles counted as half of the
// experts that can have rows).  Measured, uniform routing, us; L: 32 experts, K =
// 7168 and 4096 (gated) or 2048 weight rows; S: 96 experts, K = 1024, 768 weight
// rows; 1: one expert as L, its mean rows in brackets.
//   mean rows               L 1/4   L 8  L 128  L 256  L 1024   S 85  S 171   1 (8)  1 (64)  1 (512)
//   gated   16 rows, 2 of K    55   191    678   1241    4002     89    147      31      31       64
//           32 rows            90   170    405    691    2343     44     75      39      39       44
//           128-row tile       89   232    358    576    1908     41     63      78      79       83
//   product 16 rows, 8 of K    26    90    443    807    2996    148    272      12      13       44
//           16 rows, 2 of K    47   114    349    629    2014     85    133      29      29       32
//           32 rows            47   108    197    318     997     43     73      29      31       31
//           128-row tile       64   120    176    249     709     30     47      49      50       60
//           256-row tile       90   122    130    258     629     38     45      77      78       94
// Gated tiles start at 64 rows: 32 rows against tiles at 48, 64 and 96 rows, L 221
// and 236, 261 and 238, 341 and 249; 64 experts, K = 2048, 2816 weight rows at 64
// and 96 rows 146 and 112, 199 and 117; 256 experts as L at 32, 64 and 128 rows
// 1555 and 1821, 1988 and 1920, 3070 and 2809.
// With 96 blocks and more the split of K in 8 loses where K is short (K = 2048,
// 7168 weight rows, 8 rows of 8 experts: 37, 32 rows 31, 16 rows with K in 2 parts
// 27).  Where K is long it still gains at some 400 blocks (product L 8), and at L
// 256 tiles of 128 rows by 4 %: the rule takes neither.
template <bool GATED>
hipError_t launch_product(const ExpertShape &s, const int32_t *offset, const uint8_t *a, const float *as,
                          const uint8_t *w, const float *ws, uint16_t *out, uint8_t *q, float *qs, hipStream_t stream) {
    const int64_t mean = s.rows / s.E, cols = GATED ? s.N / 128 : (s.N + 255) / 256;
    const int64_t used = s.rows < s.E ? s.rows : s.E;
    const auto tiles = [&](int BM) { return (2 * (s.rows / BM) + used) * cols / 2; };
    const int64_t blocks = (s.rows / 16 + used) * cols;
    if constexpr (GATED) {
        if (mean >= 64 && tiles(128) >= 160) return launch_gated_tile(s, offset, a, as, w, ws, q, qs, stream);
        if (blocks < 256) return launch_stream<1, 8, 2, true>(s, offset, a, as, w, ws, out, q, qs, stream);
    } else {
        if (mean >= 96 && tiles(256) >= 192) return launch_tile<256>(s, offset, a, as, w, ws, out, stream);
        if (mean >= 40 && tiles(128) >= 128) return launch_tile<128>(s, offset, a, as, w, ws, out, stream);
        if (blocks < 96) return launch_stream<1, 2, 8, false>(s, offset, a, as, w, ws, out, q, qs, stream);
        if (blocks < 256 && mean < 16)
            return launch_stream<1, 8, 2, false>(s, offset, a, as, w, ws, out, q, qs, stream);
    }
    return launch_stream<2, 8, 1, GATED>(s, offset, a, as, w, ws, out, q, qs, stream);
}

}  // namespace

hipError_t launch_expert_gemm(const ExpertShape &s, const int32_t *offset, const uint8_t *a, const float *as,
                              const uint8_t *w, const float *ws, uint16_t *out, hipStream_t stream) {
    return launch_product<false>(s, offset, a, as, w, ws, out, nullptr, nullptr, stream);
}

hipError_t launch_expert_gated(const ExpertShape &s, const int32_t *offset, const uint8_t *a, const float *as,
                               const uint8_t *w, const float *ws, uint8_t *q, float *qs, hipStream_t stream) {
    return launch_product<true>(s, offset, a, as, w, ws, nullptr, q, qs, stream);
}

}  // namespace ep
