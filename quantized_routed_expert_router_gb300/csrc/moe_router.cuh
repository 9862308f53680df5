// moe_router.cuh - what the calls on router logits share (moe_router_stats.cu,
// moe_topk.cu): a warp holds a row, J vectors of VEC values a lane, and value i of
// vector j is expert 32*VEC*j + VEC*lane + i.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace moe {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}
// maxima to which a NaN is the largest: a row with one is not taken for a row of nothing but -inf
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
__device__ __forceinline__ float warp_max(float v) {
    float m;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// e^x for x <= 0 by the machine's exp: off by (4 + 1.3 |x|) 2^-24 of itself, 0 below 2^-126
__device__ __forceinline__ float exp_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}
// VEC consecutive values of a row as they lie in memory (VEC 1: any alignment), and their values
template <typename T, int VEC>
struct Raw {
    uint32_t w[VEC == 1 ? 1 : VEC * sizeof(T) / 4];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (VEC == 1 && sizeof(T) == 2) w[0] = *reinterpret_cast<const uint16_t *>(p);
        else if constexpr (VEC == 1) w[0] = *reinterpret_cast<const uint32_t *>(p);
        else if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4 *>(w) = *reinterpret_cast<const uint4 *>(p);
        else *reinterpret_cast<uint2 *>(w) = *reinterpret_cast<const uint2 *>(p);
    }
    __device__ __forceinline__ float value(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
};
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float v[VEC]) {
    if constexpr (VEC == 1) {
        p[0] = (T)v[0];
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2 *>(p) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
}

}  // namespace
}  // namespace moe
