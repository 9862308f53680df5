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
    int wdims;       // dimensions of w's tensor map: 5 gate and up rows in turns, 4 transposed in 64s of columns, 3
    int KB;          // blocks of depth
    int ntn, whole;  // column tiles, and those that the matrix's end does not cut off
    // test hook: bound on waits in units of 2^16 cycles; arrivals that never come at a stage's copies, at its products
    uint32_t wait;
    int hold_copies, hold_products;
};

// 1 / (1 + exp(-v)) by the machine's exp and reciprocal: off by (5 + 1.3 |v|) 2^-24 of itself, 0 below 2^-126
__device__ __forceinline__ float sigmoid(float v) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
__device__ __forceinline__ float silu_slope(float v) {
    const float s = sigmoid(v);
    return s * (1.f + v * (1.f - s));
}
__device__ __forceinline__ float gelu(float v) { return 0.5f * v * (1.f + erff(v * 0.70710678118654752f)); }
__device__ __forceinline__ float gelu_slope(float v) {
    return 0.5f * (1.f + erff(v * 0.70710678118654752f)) + v * 0.39894228040143268f * expf(-0.5f * v * v);
}

// (what passes by once leaves L2 first: the rows and matrices that other tiles take again are to stay)
__device__ __forceinline__ float get(const float *p) { return __ldcs(p); }
__device__ __forceinline__ float get(const __nv_bfloat16 *p) { return __bfloat162float(__ldcs(p)); }
__device__ __forceinline__ void put(float *p, float v) { __stcs(p, v); }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { __stcs(p, __float2bfloat16_rn(v)); }

// one value of the product (with the gated activation: a gate and an up value) to z and y
template <typename TY>
__device__ __forceinline__ void finish(const MatmulArgs &a, int g, int place, int n, float v, float up) {
    const size_t N = (size_t)a.N, at = place * N + n, at2 = place * 2 * N + n;
    TY *y = static_cast<TY *>(a.y), *z = static_cast<TY *>(a.z);
    if (a.act == MOE_ACT_SWIGLU_GRAD) {
        const float gate = get(z + at2), u = get(z + at2 + N);
        put(y + at2, v * u * silu_slope(gate));
        put(y + at2 + N, v * silu(gate));
        return;
    }
    if (a.act == MOE_ACT_SILU_GRAD || a.act == MOE_ACT_GELU_GRAD) {
        const float f = get(z + at);
        put(y + at, v * (a.act == MOE_ACT_SILU_GRAD ? silu_slope(f) : gelu_slope(f)));
        return;
    }
    if (a.act == MOE_ACT_SWIGLU) {
        if (a.bias) {
            v += a.bias[g * 2 * N + n];
            up += a.bias[g * 2 * N + N + n];
        }
        if (z) {
            put(z + at2, v);
            put(z + at2 + N, up);
        }
        v = silu(v) * up;
    } else {
        if (a.bias) v += a.bias[g * N + n];
        if (z) put(z + at, v);
        if (a.act == MOE_ACT_SILU) v = silu(v);
        else if (a.act == MOE_ACT_GELU) v = gelu(v);
    }
    if (a.residual) v += get(static_cast<const TY *>(a.residual) + at);
    put(y + at, v);
}

// C places of a column, FULL: all of them are there, otherwise the first cnt; rows are `step` values apart
template <bool FULL, typename TY, int C>
__device__ __forceinline__ void fetch(const TY *p, size_t step, int cnt, float (&v)[C]) {
#pragma unroll
    for (int j = 0; j < C; ++j, p += step) v[j] = FULL || j < cnt ? get(p) : 0.f;
}
template <bool FULL, typename TY, int C>
__device__ __forceinline__ void spread(TY *p, size_t step, int cnt, const float (&v)[C]) {
#pragma unroll
    for (int j = 0; j < C; ++j, p += step)
        if (FULL || j < cnt) put(p, v[j]);
}

// the residual of C places (0 without one), or z where the gradient takes it
template <bool FULL, typename TY, int C>
__device__ __forceinline__ void fetch_extra(const MatmulArgs &a, int place, int cnt, int n, float (&x)[C]) {
    const TY *p = static_cast<const TY *>(a.act >= MOE_ACT_SILU_GRAD ? a.z : a.residual);
    if (p) {
        fetch<FULL>(p + (size_t)place * a.N + n, (size_t)a.N, cnt, x);
    } else {
#pragma unroll
        for (int j = 0; j < C; ++j) x[j] = 0.f;
    }
}

// Products of C places with one column of the tile (lane by lane) to y and z.
//   v : the products; of `cnt` places, the first of which is `place`
//   n : this lane's column of y, which is there
//   b : its bias
// What a place takes here counts beside the products (a tile of 128 x 256 has 16384 cycles of them at K = 2048): bounds and
// what is absent are tested once for all places, not at each (30 instructions a value, then 17000 cycles a tile).
//   x : where PRE, what fetch_extra has brought for the activations that are not gated
template <int ACT, bool FULL, bool PRE, typename TY, int C>
__device__ __forceinline__ void emit(const MatmulArgs &a, float (&v)[C], const float (&x)[C], int cnt, int place, int n,
                                     float b, int lane) {
    const size_t N = (size_t)a.N;
    TY *y = static_cast<TY *>(a.y), *z = static_cast<TY *>(a.z);
    const TY *r = static_cast<const TY *>(a.residual);
    if constexpr (ACT == MOE_ACT_SWIGLU) {
        // Lanes 0 to 15 hold gate columns, lanes 16 to 31 the up columns that belong to them.  Two places at a time, either
        // lane of a pair takes one of them: it gives away its product of the other and gets what it lacks.
        const int half = lane >> 4;
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] += b;
        if (z) spread<FULL>(z + (size_t)place * 2 * N + half * N + n, 2 * N, cnt, v);
        float h[C / 2], add[C / 2];
        const int mine = (cnt + 1 - half) >> 1;   // places that this lane takes
        if (r) {
            fetch<FULL>(r + (size_t)(place + half) * N + n, 2 * N, mine, add);
        } else {
#pragma unroll
            for (int j = 0; j < C / 2; ++j) add[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < C / 2; ++j) {
            const float keep = half ? v[2 * j + 1] : v[2 * j];
            const float got = __shfl_xor_sync(0xFFFFFFFFu, half ? v[2 * j] : v[2 * j + 1], 16);
            h[j] = silu(half ? got : keep) * (half ? keep : got) + add[j];
        }
        spread<FULL>(y + (size_t)(place + half) * N + n, 2 * N, mine, h);
    } else if constexpr (ACT == MOE_ACT_SWIGLU_GRAD) {
        const size_t at = (size_t)place * 2 * N + n;
        float g[C], u[C];
        fetch<FULL>(z + at, 2 * N, cnt, g);
        fetch<FULL>(z + at + N, 2 * N, cnt, u);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const float s = sigmoid(g[j]);
            u[j] = v[j] * u[j] * (s * (1.f + g[j] * (1.f - s)));
            g[j] = v[j] * (g[j] * s);
        }
        spread<FULL>(y + at, 2 * N, cnt, u);
        spread<FULL>(y + at + N, 2 * N, cnt, g);
    } else {
        const size_t at = (size_t)place * N + n;
        float add[C];   // the residual, or z
        if constexpr (PRE) {
#pragma unroll
            for (int j = 0; j < C; ++j) add[j] = x[j];
        } else {
            fetch_extra<FULL, TY>(a, place, cnt, n, add);
        }
        if constexpr (ACT == MOE_ACT_SILU_GRAD || ACT == MOE_ACT_GELU_GRAD) {
#pragma unroll
            for (int j = 0; j < C; ++j) v[j] *= ACT == MOE_ACT_SILU_GRAD ? silu_slope(add[j]) : gelu_slope(add[j]);
        } else {
#pragma unroll
            for (int j = 0; j < C; ++j) v[j] += b;
            if (ACT != MOE_ACT_NONE && z) spread<FULL>(z + at, N, cnt, v);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                if (ACT == MOE_ACT_SILU) v[j] = silu(v[j]);
                if (ACT == MOE_ACT_GELU) v[j] = gelu(v[j]);
                v[j] += add[j];
            }
        }
        spread<FULL>(y + at, N, cnt, v);
    }
}

template <bool FULL, bool PRE, typename TY, int C>
__device__ __forceinline__ void emit_f(const MatmulArgs &a, float (&v)[C], const float (&x)[C], int cnt, int place, int n,
                                       float b, int lane) {
    switch (a.act) {
        case MOE_ACT_NONE: return emit<MOE_ACT_NONE, FULL, PRE, TY, C>(a, v, x, cnt, place, n, b, lane);
        case MOE_ACT_SILU: return emit<MOE_ACT_SILU, FULL, PRE, TY, C>(a, v, x, cnt, place, n, b, lane);
        case MOE_ACT_GELU: return emit<MOE_ACT_GELU, FULL, PRE, TY, C>(a, v, x, cnt, place, n, b, lane);
        case MOE_ACT_SWIGLU: return emit<MOE_ACT_SWIGLU, FULL, PRE, TY, C>(a, v, x, cnt, place, n, b, lane);
        case MOE_ACT_SILU_GRAD: return emit<MOE_ACT_SILU_GRAD, FULL, PRE, TY, C>(a, v, x, cnt, place, n, b, lane);
        case MOE_ACT_GELU_GRAD: return emit<MOE_ACT_GELU_GRAD, FULL, PRE, TY, C>(a, v, x, cnt, place, n, b, lane);
        default: return emit<MOE_ACT_SWIGLU_GRAD, FULL, PRE, TY, C>(a, v, x, cnt, place, n, b, lane);
    }
}
// (with the gated activation N is a multiple of 16, and the lanes of a warp are there or not together)
template <bool PRE, typename TY, int C>
__device__ __forceinline__ void emit_t(const MatmulArgs &a, float (&v)[C], const float (&x)[C], int cnt, int place, int n,
                                       bool in, float b, int lane) {
    if (!in) return;
    if (cnt == C) emit_f<true, PRE, TY, C>(a, v, x, cnt, place, n, b, lane);
    else emit_f<false, PRE, TY, C>(a, v, x, cnt, place, n, b, lane);
}

}  // namespace moe
