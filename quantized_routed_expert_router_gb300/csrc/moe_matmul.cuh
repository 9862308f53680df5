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
    uint32_t wait;   // bound on waits in units of 2^16 cycles
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

// Products of C places with one column of the tile (lane by lane) to y and z.
//   v   : the products; of `cnt` places, the first of which is `place`
//   n   : this lane's column of y; in: it is there
//   b   : its bias
// MOE_ACT_SWIGLU: lanes 0 to 15 hold gate columns, lanes 16 to 31 the up columns that belong to them.  Two places at
// a time, either lane of a pair takes one of them: it gives away its product of the other and gets what it lacks.
template <int ACT, typename TY, int C>
__device__ __forceinline__ void emit(const MatmulArgs &a, float (&v)[C], int cnt, int place, int n, bool in, float b,
                                     int lane) {
    const size_t N = (size_t)a.N;
    TY *y = static_cast<TY *>(a.y), *z = static_cast<TY *>(a.z);
    if constexpr (ACT == MOE_ACT_SWIGLU) {
        const int half = lane >> 4;
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] += b;
        if (z) {
            TY *to = z + (size_t)place * 2 * N + half * N + n;
#pragma unroll
            for (int j = 0; j < C; ++j)
                if (in && j < cnt) put(to + (size_t)j * 2 * N, v[j]);
        }
        const TY *r = a.residual ? static_cast<const TY *>(a.residual) + (size_t)place * N + n : nullptr;
        TY *to = y + (size_t)place * N + n;
#pragma unroll
        for (int j0 = 0; j0 < C; j0 += 16) {
            constexpr int P = C < 16 ? C : 16;
            float add[P / 2];
#pragma unroll
            for (int j = 0; j < P; j += 2)
                add[j / 2] = r && in && j0 + j + half < cnt ? to_f(r[(size_t)(j0 + j + half) * N]) : 0.f;
#pragma unroll
            for (int j = 0; j < P; j += 2) {
                const float mine = half ? v[j0 + j + 1] : v[j0 + j], other = half ? v[j0 + j] : v[j0 + j + 1];
                const float got = __shfl_xor_sync(0xFFFFFFFFu, other, 16);
                const float gate = half ? got : mine, up = half ? mine : got;
                if (in && j0 + j + half < cnt) put(to + (size_t)(j0 + j + half) * N, silu(gate) * up + add[j / 2]);
            }
        }
    } else if constexpr (ACT == MOE_ACT_SWIGLU_GRAD) {
        const TY *from = z + (size_t)place * 2 * N + n;
        TY *to = y + (size_t)place * 2 * N + n;
        constexpr int P = C < 8 ? C : 8;
#pragma unroll
        for (int j0 = 0; j0 < C; j0 += P) {
            float g[P], u[P];
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const bool live = in && j0 + j < cnt;
                g[j] = live ? to_f(from[(size_t)(j0 + j) * 2 * N]) : 0.f;
                u[j] = live ? to_f(from[(size_t)(j0 + j) * 2 * N + N]) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < P; ++j) {
                if (!in || j0 + j >= cnt) continue;
                const float s = sigmoid(g[j]);
                put(to + (size_t)(j0 + j) * 2 * N, v[j0 + j] * u[j] * (s * (1.f + g[j] * (1.f - s))));
                put(to + (size_t)(j0 + j) * 2 * N + N, v[j0 + j] * (g[j] * s));
            }
        }
    } else {
        constexpr bool GRAD = ACT == MOE_ACT_SILU_GRAD || ACT == MOE_ACT_GELU_GRAD;
        const TY *r = static_cast<const TY *>(GRAD ? a.z : a.residual);
        if (r) r += (size_t)place * N + n;
        if (z) z += (size_t)place * N + n;
        y += (size_t)place * N + n;
        constexpr int P = C < 16 ? C : 16;
#pragma unroll
        for (int j0 = 0; j0 < C; j0 += P) {
            float add[P];
#pragma unroll
            for (int j = 0; j < P; ++j) add[j] = r && in && j0 + j < cnt ? to_f(r[(size_t)(j0 + j) * N]) : 0.f;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                if (!in || j0 + j >= cnt) continue;
                float f = v[j0 + j];
                if constexpr (GRAD) {
                    f *= ACT == MOE_ACT_SILU_GRAD ? silu_slope(add[j]) : gelu_slope(add[j]);
                } else {
                    f += b;
                    if (ACT != MOE_ACT_NONE && z) put(z + (size_t)(j0 + j) * N, f);
                    if (ACT == MOE_ACT_SILU) f = silu(f);
                    if (ACT == MOE_ACT_GELU) f = gelu(f);
                    f += add[j];
                }
                put(y + (size_t)(j0 + j) * N, f);
            }
        }
    }
}

template <typename TY, int C>
__device__ __forceinline__ void emit_t(const MatmulArgs &a, float (&v)[C], int cnt, int place, int n, bool in, float b,
                                       int lane) {
    switch (a.act) {
        case MOE_ACT_NONE: return emit<MOE_ACT_NONE, TY, C>(a, v, cnt, place, n, in, b, lane);
        case MOE_ACT_SILU: return emit<MOE_ACT_SILU, TY, C>(a, v, cnt, place, n, in, b, lane);
        case MOE_ACT_GELU: return emit<MOE_ACT_GELU, TY, C>(a, v, cnt, place, n, in, b, lane);
        case MOE_ACT_SWIGLU: return emit<MOE_ACT_SWIGLU, TY, C>(a, v, cnt, place, n, in, b, lane);
        case MOE_ACT_SILU_GRAD: return emit<MOE_ACT_SILU_GRAD, TY, C>(a, v, cnt, place, n, in, b, lane);
        case MOE_ACT_GELU_GRAD: return emit<MOE_ACT_GELU_GRAD, TY, C>(a, v, cnt, place, n, in, b, lane);
        default: return emit<MOE_ACT_SWIGLU_GRAD, TY, C>(a, v, cnt, place, n, in, b, lane);
    }
}

}  // namespace moe
