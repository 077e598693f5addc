// tile_device.h -- what the kernels of products share on the device: loads of
// tiles into LDS, waits, and the gate.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_device.h"

namespace ep {

typedef float f32x4 __attribute__((ext_vector_type(4)));

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

}  // namespace ep
