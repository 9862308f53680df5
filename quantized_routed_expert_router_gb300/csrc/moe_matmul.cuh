// moe_matmul.cuh - arguments and epilogue of moe_matmul.
#pragma once

#include <cuda_bf16.h>
#include <stddef.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

struct MatmulArgs {
    const __nv_bfloat16 *x, *w;
    const float *bias;
    const int32_t *rows, *offsets;
    const void *residual;
    void *z, *y;
    unsigned *status;
    int X, M, G, N, K;
    int act, transposed, ybf16;
};

__device__ __forceinline__ float load_y(const void *p, size_t i, int bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void store_y(void *p, size_t i, float v, int bf16) {
    if (bf16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<float *>(p)[i] = v;
}
__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + expf(-v)); }
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
__device__ __forceinline__ float silu_slope(float v) {
    const float s = sigmoid(v);
    return s * (1.f + v * (1.f - s));
}
__device__ __forceinline__ float gelu(float v) { return 0.5f * v * (1.f + erff(v * 0.70710678118654752f)); }
__device__ __forceinline__ float gelu_slope(float v) {
    return 0.5f * (1.f + erff(v * 0.70710678118654752f)) + v * 0.39894228040143268f * expf(-0.5f * v * v);
}

// one value of the product (gate and up: two) to z and y
__device__ __forceinline__ void finish(const MatmulArgs &a, int place, int g, int n, float v, float up) {
    const size_t i = (size_t)place * a.N + n, wide = (size_t)place * 2 * a.N + n;
    if (a.act == MOE_ACT_SWIGLU_GRAD) {
        const float gate = load_y(a.z, wide, a.ybf16), u = load_y(a.z, wide + a.N, a.ybf16);
        store_y(a.y, wide, v * u * silu_slope(gate), a.ybf16);
        store_y(a.y, wide + a.N, v * silu(gate), a.ybf16);
        return;
    }
    if (a.act == MOE_ACT_SILU_GRAD || a.act == MOE_ACT_GELU_GRAD) {
        const float z = load_y(a.z, i, a.ybf16);
        store_y(a.y, i, v * (a.act == MOE_ACT_SILU_GRAD ? silu_slope(z) : gelu_slope(z)), a.ybf16);
        return;
    }
    if (a.act == MOE_ACT_SWIGLU) {
        if (a.bias) {
            v += a.bias[(size_t)g * 2 * a.N + n];
            up += a.bias[(size_t)g * 2 * a.N + a.N + n];
        }
        if (a.z) {
            store_y(a.z, wide, v, a.ybf16);
            store_y(a.z, wide + a.N, up, a.ybf16);
        }
        v = silu(v) * up;
    } else {
        if (a.bias) v += a.bias[(size_t)g * a.N + n];
        if (a.z) store_y(a.z, i, v, a.ybf16);
        if (a.act == MOE_ACT_SILU) v = silu(v);
        else if (a.act == MOE_ACT_GELU) v = gelu(v);
    }
    if (a.residual) v += load_y(a.residual, i, a.ybf16);
    store_y(a.y, i, v, a.ybf16);
}

}  // namespace moe
