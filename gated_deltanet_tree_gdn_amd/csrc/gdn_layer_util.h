// gdn_layer_util.h -- loads, stores, sums over lanes and gate functions shared
// by the kernels of gdn_layer.h.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gdn_layer.h"

namespace gdn {

__host__ __device__ constexpr int dtype_size(int dtype) { return dtype == GDN_BF16 ? 2 : 4; }

// A grid of n workgroups or more, in rows of 2^20: one dimension may not have
// 2^32 threads.  Kernels number workgroups by block_id() and drop those from n on.
inline dim3 grid_of(int64_t n) {
    const int64_t row = n < (1 << 20) ? n : 1 << 20;
    return dim3(static_cast<unsigned>(row), static_cast<unsigned>((n + row - 1) / row));
}
__device__ __forceinline__ int64_t block_id() { return int64_t(blockIdx.y) * gridDim.x + blockIdx.x; }

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __builtin_bit_cast(float, u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __builtin_bit_cast(float, u & 0xffff0000u); }

// Two fp32 values as packed bf16, rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    bf16x2 v;
    v[0] = static_cast<__bf16>(a);
    v[1] = static_cast<__bf16>(b);
    return __builtin_bit_cast(uint32_t, v);
}

// Element i of an array whose dtype is known at run time (uniform over the
// wavefront, so the branch costs a scalar compare).
__device__ __forceinline__ float load1(const void* p, int dtype, int64_t i) {
    if (dtype == GDN_BF16)
        return __builtin_bit_cast(float, static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
    return static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void store1(void* p, int dtype, int64_t i, float x) {
    if (dtype == GDN_BF16)
        static_cast<__bf16*>(p)[i] = static_cast<__bf16>(x);
    else
        static_cast<float*>(p)[i] = x;
}

// Elements i .. i + 7, with the alignment of an element: 16-byte accesses may
// start anywhere.
__device__ __forceinline__ void load8(const void* p, int dtype, int64_t i, float (&x)[8]) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
    typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));
    if (dtype == GDN_BF16) {
        const u32x4 u = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = bf16_lo(u[j]);
            x[2 * j + 1] = bf16_hi(u[j]);
        }
    } else {
        const f32x4* f = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
        const f32x4 a = f[0], b = f[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = a[j];
            x[4 + j] = b[j];
        }
    }
}

__device__ __forceinline__ void store8(void* p, int dtype, int64_t i, const float (&x)[8]) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
    typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));
    if (dtype == GDN_BF16) {
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) =
            u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
    } else {
        f32x4* f = reinterpret_cast<f32x4*>(static_cast<float*>(p) + i);
        f[0] = f32x4{x[0], x[1], x[2], x[3]};
        f[1] = f32x4{x[4], x[5], x[6], x[7]};
    }
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// Sum over aligned groups of W lanes, the result in every lane: exchanges
// with lanes xor 1 and xor 2 (quad permutes), then mirrored halves and rows
// of 16, then across rows.
template <int W>
__device__ __forceinline__ float lane_sum(float x) {
    if constexpr (W >= 2) x += dpp<0xB1>(x);
    if constexpr (W >= 4) x += dpp<0x4E>(x);
    if constexpr (W >= 8) x += dpp<0x141>(x);
    if constexpr (W >= 16) x += dpp<0x140>(x);
    if constexpr (W >= 32) x += __shfl_xor(x, 16);
    if constexpr (W >= 64) x += __shfl_xor(x, 32);
    return x;
}

// 1 / (1 + e^-a) with the hardware's exponential and reciprocal (1 ulp each).
__device__ __forceinline__ float sigmoidf(float a) { return __builtin_amdgcn_rcpf(1.0f + __expf(-a)); }

__device__ __forceinline__ float activate(int act, float a) {
    switch (act) {
        case GDN_ACT_SILU: return a * sigmoidf(a);
        case GDN_ACT_GELU: return 0.5f * a * (1.0f + erff(a * 0.70710678118654752f));
        case GDN_ACT_SIGMOID: return sigmoidf(a);
        default: return a;
    }
}

// Waits until at most N of the wavefront's loads and stores are outstanding
// (any number: kAnyLoads) and, if READS, until its LDS accesses are done.  For
// kernels with loads straight to LDS: a fence would wait for every one of them
// (they count as LDS writes); what has to have arrived is exactly what the
// count says.
constexpr int kAnyLoads = 63;
template <int N, bool READS = true>
__device__ __forceinline__ void wait_count() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | (READS ? 0 : 15) << 8 | (N >> 4) << 14);
    asm volatile("" ::: "memory");
}

// The same, then meets the workgroup.
template <int N, bool READS = true>
__device__ __forceinline__ void loads_barrier() {
    wait_count<N, READS>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

}  // namespace gdn
