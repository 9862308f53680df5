// moe_topk.cu - the experts of each token and their gating weights from the
// logits of any number of tokens (moe_topk), and the weights' gradient back to
// the logits (moe_topk_grad).
//
// A warp takes a row, VEC * J values a lane.  A logit becomes a 32-bit key whose
// unsigned order is the choice's: larger numbers first, -0 equal to 0, NaN above
// all, 0 for what may not be taken (-inf, past E, chosen already).  Each of the k
// rounds finds the largest key of the warp; where several lanes hold it, the one
// with the lowest index wins.  Slot s of the row ends in lane s.
#include <cuda_bf16.h>
#include <math.h>

#include "moe_around.h"
#include "moe_launch.h"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);   // -0 becomes 0
    if (v != v) return kAll;
    if (u == 0xFF800000u) return 0;
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {   // -inf for 0
    if (key == 0) return -INFINITY;
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
    return v;
}
__device__ __forceinline__ float exp_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}
// sigma(l) exp(-m) for m = min(l's row's largest, 0): what all of a row's sigmas have in common cancels
// in their ratios, so that rows whose sigmas would vanish keep theirs
__device__ __forceinline__ float sigmoid_over(float l, float m) {
    return l >= 0.f ? 1.f / (1.f + expf(-l)) : expf(l - m) / (1.f + expf(l));
}
__device__ __forceinline__ float min0(float v) { return v > 0.f ? 0.f : v; }   // NaN stays

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T *p, float v[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = (float)p[0];
    } else if constexpr (sizeof(T) == 4) {
        const float4 f = *reinterpret_cast<const float4 *>(p);
        v[0] = f.x;
        v[1] = f.y;
        v[2] = f.z;
        v[3] = f.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        v[0] = __uint_as_float(u.x << 16);
        v[1] = __uint_as_float(u.x & 0xFFFF0000u);
        v[2] = __uint_as_float(u.y << 16);
        v[3] = __uint_as_float(u.y & 0xFFFF0000u);
    }
}
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

// sum of exp(l - m) over a row
template <int VEC, int J>
__device__ __forceinline__ float row_sum(const float l[J][VEC], float m) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) s += exp_fast(l[j][i] - m);
    return warp_sum(s);
}

// lane < k holds a chosen logit (-inf: none); m: the largest of the row, all: sum of exp(l - m) over the row where
// the weights are shares of it.  The slot's weight; slope: 1 - sigma(l), or 1 for softmax
__device__ __forceinline__ float weight_of(float l, float m, float all, bool sigmoid, bool renorm, float &slope) {
    const bool some = l != -INFINITY;
    float g;
    slope = 1.f;
    if (sigmoid) {
        g = some ? sigmoid_over(l, renorm ? min0(m) : 0.f) : 0.f;
        slope = some ? sigmoid_over(-l, 0.f) : 0.f;
    } else {
        g = some ? expf(l - m) : 0.f;
    }
    if (renorm) all = warp_sum(g);
    else if (sigmoid) return g;
    return some ? g / all : 0.f;
}

struct TopkArgs {
    const void *logits;
    const uint8_t *valid;
    int32_t *ids;
    float *weights;
    int T, E, k, sigmoid, renorm;
};

template <typename T, int VEC, int J>
__global__ void __launch_bounds__(32 * kWarps) topk_kernel(const TopkArgs a) {
    const int lane = threadIdx.x & 31, t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    int id = -1;
    float w = 0.f;
    if (!a.valid || a.valid[t]) {
        const T *row = static_cast<const T *>(a.logits) + (size_t)t * a.E;
        float l[J][VEC];
        uint32_t key[J][VEC];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int e = 32 * VEC * j + VEC * lane;
#pragma unroll
            for (int i = 0; i < VEC; ++i) l[j][i] = -INFINITY;
            if (e < a.E) load_vec<T, VEC>(row + e, l[j]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) key[j][i] = key_of(l[j][i]);
        }
        uint32_t best = 0, chosen = 0;
        int at = 0;   // of this lane's largest: the lowest index
        const auto look = [&] {
            best = 0;
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (key[j][i] > best) {
                        best = key[j][i];
                        at = 32 * VEC * j + VEC * lane + i;
                    }
        };
        look();
        for (int s = 0; s < a.k; ++s) {
            const uint32_t top = __reduce_max_sync(kAll, best);
            if (top == 0) break;
            const unsigned who = __ballot_sync(kAll, best == top);
            int e = __shfl_sync(kAll, at, __ffs(who) - 1);
            if (who & (who - 1)) e = (int)__reduce_min_sync(kAll, best == top ? (unsigned)at : kAll);
            if (lane == s) {
                id = e;
                chosen = top;
            }
            if (best == top && at == e) {
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if (32 * VEC * j + VEC * lane + i == e) key[j][i] = 0;
                look();
            }
        }
        const float mine = value_of(chosen), m = __shfl_sync(kAll, mine, 0);
        const float all = a.sigmoid || a.renorm ? 0.f : row_sum<VEC, J>(l, m);
        float slope;
        w = weight_of(mine, m, all, a.sigmoid, a.renorm, slope);
    }
    if (lane < a.k) {
        a.ids[(size_t)t * a.k + lane] = id;
        if (a.weights) a.weights[(size_t)t * a.k + lane] = w;
    }
}

struct TopkGradArgs {
    const void *logits, *addend;
    const int32_t *ids;
    const float *dweights;
    void *dlogits;
    int T, E, k, sigmoid, renorm;
};

// ROW: the gradient reaches the whole row (softmax over all E); otherwise the chosen experts
template <typename T, int VEC, int J, bool ROW>
__global__ void __launch_bounds__(32 * kWarps) topk_grad_kernel(const TopkGradArgs a) {
    extern __shared__ float buf[];   // a row a warp
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = blockIdx.x * kWarps + warp;
    if (t >= a.T) return;
    float *at = buf + warp * 32 * VEC * J;
    const T *row = static_cast<const T *>(a.logits) + (size_t)t * a.E;
    int id = lane < a.k ? a.ids[(size_t)t * a.k + lane] : -1;
    if ((unsigned)id >= (unsigned)a.E) id = -1;
    const float mine = id >= 0 ? (float)row[id] : -INFINITY;
    const float d = id >= 0 ? a.dweights[(size_t)t * a.k + lane] : 0.f;
    uint32_t top = key_of(mine);
    float l[J][VEC], all = 0.f;
    if constexpr (ROW) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int e = 32 * VEC * j + VEC * lane;
#pragma unroll
            for (int i = 0; i < VEC; ++i) l[j][i] = -INFINITY;
            if (e < a.E) load_vec<T, VEC>(row + e, l[j]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) top = max(top, key_of(l[j][i]));
        }
    }
    const float m = value_of(__reduce_max_sync(kAll, top));
    if constexpr (ROW) all = row_sum<VEC, J>(l, m);
    float slope;
    const float w = weight_of(mine, m, all, a.sigmoid, a.renorm, slope);
    const bool ratio = a.renorm || !a.sigmoid;
    const float dot = ratio ? warp_sum(id >= 0 ? w * d : 0.f) : 0.f;
    // the row's gradient at the chosen experts, slot by slot: an id that comes twice is added up in order
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) at[32 * VEC * j + VEC * lane + i] = 0.f;
    __syncwarp();
    const float g = ROW ? w * d : slope * w * (d - dot);
    for (int s = 0; s < a.k; ++s) {
        if (lane == s && id >= 0) at[id] += g;
        __syncwarp();
    }
    const float scale = ROW ? dot / all : 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int e = 32 * VEC * j + VEC * lane;
        if (e >= a.E) continue;
        float v[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = 0.f;
        if (a.addend) load_vec<T, VEC>(static_cast<const T *>(a.addend) + (size_t)t * a.E + e, v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float g = at[e + i];
            if constexpr (ROW) {
                // a row without slots has no gradient, whatever its logits are
                if (dot != 0.f && l[j][i] != -INFINITY) g -= exp_fast(l[j][i] - m) * scale;
            }
            v[i] += g;
        }
        store_vec<T, VEC>(static_cast<T *>(a.dlogits) + (size_t)t * a.E + e, v);
    }
}

template <typename T, int VEC, int J>
cudaError_t topk_t(const TopkArgs &a, cudaStream_t s) {
    topk_kernel<T, VEC, J><<<(unsigned)((a.T + kWarps - 1) / kWarps), 32 * kWarps, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename T, int VEC, int J>
cudaError_t topk_t(const TopkGradArgs &a, cudaStream_t s) {
    constexpr int smem = kWarps * 32 * VEC * J * (int)sizeof(float);   // 16 KB at most
    const unsigned grid = (unsigned)((a.T + kWarps - 1) / kWarps);
    if (!a.sigmoid && !a.renorm) topk_grad_kernel<T, VEC, J, true><<<grid, 32 * kWarps, smem, s>>>(a);
    else topk_grad_kernel<T, VEC, J, false><<<grid, 32 * kWarps, smem, s>>>(a);
    return cudaGetLastError();
}

// rows of whole 4-value pieces, or value by value
template <typename T, typename A>
cudaError_t by_width(const A &a, cudaStream_t s) {
    if (a.E % 4 == 0) {
        if (a.E <= 128) return topk_t<T, 4, 1>(a, s);
        if (a.E <= 256) return topk_t<T, 4, 2>(a, s);
        if (a.E <= 512) return topk_t<T, 4, 4>(a, s);
        return topk_t<T, 4, 8>(a, s);
    }
    if (a.E <= 64) return topk_t<T, 1, 2>(a, s);
    if (a.E <= 256) return topk_t<T, 1, 8>(a, s);
    return topk_t<T, 1, 32>(a, s);
}

}  // namespace

cudaError_t launch_topk(const void *logits, int dtype, const uint8_t *valid, int T, int E, int k, int gating,
                        int renormalize, int32_t *ids, float *weights, cudaStream_t s) {
    const TopkArgs a = {logits, valid, ids, weights, T, E, k, gating == MOE_GATE_SIGMOID, renormalize != 0};
    return dtype == MOE_DT_BF16 ? by_width<__nv_bfloat16>(a, s) : by_width<float>(a, s);
}

cudaError_t launch_topk_grad(const void *logits, int dtype, const int32_t *ids, const float *dweights, int T, int E,
                             int k, int gating, int renormalize, const void *addend, void *dlogits, cudaStream_t s) {
    const TopkGradArgs a = {logits, addend, ids, dweights, dlogits, T, E, k, gating == MOE_GATE_SIGMOID,
                            renormalize != 0};
    return dtype == MOE_DT_BF16 ? by_width<__nv_bfloat16>(a, s) : by_width<float>(a, s);
}

}  // namespace moe
