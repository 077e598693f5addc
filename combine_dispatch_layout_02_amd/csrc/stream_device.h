// stream_device.h -- weights streamed through LDS for a few rows: what the
// kernels that are bound by their weights' bytes share on the device.
#pragma once

#include "tile_device.h"

namespace ep {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kPast = 0x80000000u;   // past any buffer's end: reads 0, no memory traffic

__device__ __forceinline__ vec16 load_16(rsrc_t b, uint32_t off, uint32_t soff) {
    return __builtin_bit_cast(vec16, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, (int)soff, 0));
}

// 8 e4m3 values as bf16, exactly.
__device__ __forceinline__ bf16x8 widen8(uint32_t a, uint32_t b) {
    bf16x8 o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t v = i ? b : a;
        const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false);
        const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true);
        o[4 * i + 0] = lo[0];
        o[4 * i + 1] = lo[1];
        o[4 * i + 2] = hi[0];
        o[4 * i + 3] = hi[1];
    }
    return o;
}

// v rounded to bf16, which leaves v with the rest, exactly: the value's next part.
// Of a value in [1, 2) 2^-8 is left at most after one part, 2^-17 after two, nothing
// after three.  A finite value's part is finite: cut where it would round up to
// infinity.
__device__ __forceinline__ uint32_t take_part(float &v) {
    uint32_t h = f32_to_bf16(v);
    if ((h & 0x7FFF) == 0x7F80 && v - v == 0.0f) h = f2u(v) >> 16;
    v = (h & 0x7F80) == 0x7F80 ? 0.0f : v - u2f(h << 16);
    return h;
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// A step of one wave: 128 bytes of K of G groups of 16 weight rows, in LDS as
// 128-byte rows whose 16-byte pieces are permuted by the row (piece c lies at c
// ^ (r % 8)), so that the lanes of one LDS cycle touch every bank once.  A lane
// takes pieces `quad` and `quad + 4` of row lane % 16; the second operand's
// lane names the same values of K.
template <bool F8, int G>
struct Step {
    static constexpr int KE = F8 ? 128 : 64;     // values of K
    static constexpr int CHUNKS = F8 ? 4 : 2;    // matrix instructions of 32 values
    bf16x8 a[G][CHUNKS];
    // The reads and their wait are one block of assembly: for a read that the
    // compiler sees, it waits until no load into LDS that it cannot tell apart
    // is under way, which the steps' own counts make unnecessary.
    __device__ __forceinline__ Step(const uint8_t *lds, uint32_t plo) {
        const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t *)lds + plo;
        vec16 v[G][2];
        if constexpr (G == 4)
            asm volatile(
                "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\t"
                "ds_read_b128 %2, %8 offset:2048\n\tds_read_b128 %3, %9 offset:2048\n\t"
                "ds_read_b128 %4, %8 offset:4096\n\tds_read_b128 %5, %9 offset:4096\n\t"
                "ds_read_b128 %6, %8 offset:6144\n\tds_read_b128 %7, %9 offset:6144\n\ts_waitcnt lgkmcnt(0)"
                : "=&v"(v[0][0]), "=&v"(v[0][1]), "=&v"(v[1][0]), "=&v"(v[1][1]), "=&v"(v[2][0]), "=&v"(v[2][1]),
                  "=&v"(v[3][0]), "=&v"(v[3][1])
                : "v"(at), "v"(at ^ 64)
                : "memory");
        else if constexpr (G == 2)
            asm volatile(
                "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\t"
                "ds_read_b128 %2, %4 offset:2048\n\tds_read_b128 %3, %5 offset:2048\n\ts_waitcnt lgkmcnt(0)"
                : "=&v"(v[0][0]), "=&v"(v[0][1]), "=&v"(v[1][0]), "=&v"(v[1][1])
                : "v"(at), "v"(at ^ 64)
                : "memory");
        else
            asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                         : "=&v"(v[0][0]), "=&v"(v[0][1])
                         : "v"(at), "v"(at ^ 64)
                         : "memory");
#pragma unroll
        for (int g = 0; g < G; ++g)
            if constexpr (F8) {
                a[g][0] = widen8(v[g][0][0], v[g][0][1]);
                a[g][1] = widen8(v[g][0][2], v[g][0][3]);
                a[g][2] = widen8(v[g][1][0], v[g][1][1]);
                a[g][3] = widen8(v[g][1][2], v[g][1][3]);
            } else {
                a[g][0] = __builtin_bit_cast(bf16x8, v[g][0]);
                a[g][1] = __builtin_bit_cast(bf16x8, v[g][1]);
            }
    }
    // Where chunk c of the second operand starts, as bytes of bf16 values from the step's first.
    static __device__ __forceinline__ uint32_t at(int c, int quad) {
        return F8 ? (uint32_t)((c >> 1) * 128 + quad * 32 + (c & 1) * 16) : (uint32_t)(c * 64 + quad * 16);
    }
};

// The weights' way into LDS: 2 G loads of 8 rows each.  Rows are given by their
// byte offsets from the buffer's base; a step past the end reads nothing.
template <int G>
struct Stage {
    uint32_t off[2 * G];   // of the lane's row in each load, without K
    uint32_t piece;        // byte of K in the step
    __device__ __forceinline__ void go(rsrc_t b0, rsrc_t b1, uint8_t *lds, uint32_t k, uint32_t bytes) const {
        const uint32_t past = k + piece < bytes ? 0u : kPast;   // the end of K
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) load_to_lds(i < G ? b0 : b1, lds + i * 1024, (off[i] + piece) | past, k);
    }
};

// Waits until at most N of the wave's later loads are under way.
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "the counter's width");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
// A step's weights have arrived.  Step s issues the values of the second operand
// for s + 1 (X loads at least) and the weights for s + NB (W loads): behind the
// weights of a step are those of the NB - 1 steps before it, or, for the first
// ones, what was issued ahead of all steps.
template <int NB, int X, int W>
__device__ __forceinline__ void wait_step(int i) {
    if (i >= NB - 1)
        wait_loads<(NB - 1) * (X + W)>();
    else
        wait_loads<X + (NB - 1) * W>();
}

}  // namespace ep
