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
    int KB;          // blocks of depth
    int ntn;         // column tiles
    // test hook: bound on waits in units of 2^16 cycles; arrivals that never come at a stage's copies, at its products
    uint32_t wait;
    int hold_copies, hold_products;
};

// 1 / (1 + exp(-v)) by the machine's exp and reciprocal: off by (5 + 1.3 |v|) 2^-24 of itself
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

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// C places of a column, FULL: all of them are there, otherwise the first cnt; rows are `step` values apart
template <bool FULL, typename TY, int C>
__device__ __forceinline__ void fetch(const TY *p, size_t step, int cnt, float (&v)[C]) {
#pragma unroll
    for (int j = 0; j < C; ++j, p += step) v[j] = FULL || j < cnt ? to_f(*p) : 0.f;
}
template <bool FULL, typename TY, int C>
__device__ __forceinline__ void spread(TY *p, size_t step, int cnt, const float (&v)[C]) {
#pragma unroll
    for (int j = 0; j < C; ++j, p += step)
        if (FULL || j < cnt) put(p, v[j]);
}

// Products of C places with one column of the tile (lane by lane) to y and z.
//   v : the products; of `cnt` places, the first of which is `place`
//   n : this lane's column of y, which is there
//   b : its bias
// What a place takes here counts beside the products (a tile of 128 x 256 has 16384 cycles of them at K = 2048): bounds and
// what is absent are tested once for all places, not at each (30 instructions a value, then 17000 cycles a tile).
template <int ACT, bool FULL, typename TY, int C>
__device__ __forceinline__ void emit(const MatmulArgs &a, float (&v)[C], int cnt, int place, int n, float b, int lane) {
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
        if constexpr (ACT == MOE_ACT_SILU_GRAD || ACT == MOE_ACT_GELU_GRAD) {
            float f[C];
            fetch<FULL>(z + at, N, cnt, f);
#pragma unroll
            for (int j = 0; j < C; ++j) v[j] *= ACT == MOE_ACT_SILU_GRAD ? silu_slope(f[j]) : gelu_slope(f[j]);
        } else {
            float add[C];
            if (r) {
                fetch<FULL>(r + at, N, cnt, add);
            } else {
#pragma unroll
                for (int j = 0; j < C; ++j) add[j] = 0.f;
            }
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

template <bool FULL, typename TY, int C>
__device__ __forceinline__ void emit_f(const MatmulArgs &a, float (&v)[C], int cnt, int place, int n, float b, int lane) {
    switch (a.act) {
        case MOE_ACT_NONE: return emit<MOE_ACT_NONE, FULL, TY, C>(a, v, cnt, place, n, b, lane);
        case MOE_ACT_SILU: return emit<MOE_ACT_SILU, FULL, TY, C>(a, v, cnt, place, n, b, lane);
        case MOE_ACT_GELU: return emit<MOE_ACT_GELU, FULL, TY, C>(a, v, cnt, place, n, b, lane);
        case MOE_ACT_SWIGLU: return emit<MOE_ACT_SWIGLU, FULL, TY, C>(a, v, cnt, place, n, b, lane);
        case MOE_ACT_SILU_GRAD: return emit<MOE_ACT_SILU_GRAD, FULL, TY, C>(a, v, cnt, place, n, b, lane);
        case MOE_ACT_GELU_GRAD: return emit<MOE_ACT_GELU_GRAD, FULL, TY, C>(a, v, cnt, place, n, b, lane);
        default: return emit<MOE_ACT_SWIGLU_GRAD, FULL, TY, C>(a, v, cnt, place, n, b, lane);
    }
}
// (with the gated activation N is a multiple of 16, and the lanes of a warp are there or not together)
template <typename TY, int C>
__device__ __forceinline__ void emit_t(const MatmulArgs &a, float (&v)[C], int cnt, int place, int n, bool in, float b,
                                       int lane) {
    if (!in) return;
    if (cnt == C) emit_f<true, TY, C>(a, v, cnt, place, n, b, lane);
    else emit_f<false, TY, C>(a, v, cnt, place, n, b, lane);
}

}  // namespace moe
