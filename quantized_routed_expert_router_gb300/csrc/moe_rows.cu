// moe_rows.cu - token rows to their places in the order by expert and back,
// with the gating weights applied, and the gradient (moe_dispatch_rows,
// moe_combine_rows, moe_combine_grad).
//
// All three only move rows: each row is read once and written once, V values of
// it a thread, whole 16-byte pieces where the width allows.  Tokens are what the
// blocks are dealt by: a block has a token's k places in hand, so that a token's
// row is read (or written) once for all of them, nothing is added by atomics, and
// the k rows of a piece are on their way at once.  DRAM bounds all three.  On the
// device: combine 8192 x 8 rows of 4096 in bf16 90.8 us (0.98 of the copy rate),
// dispatch 4096 x 8 of 7168 78.5 (0.97), the gradient 8191 x 4 of 2880 65.7 (0.95;
// 86.6 with blocks of 128 threads whose last round over a row was mostly empty).
//   Narrow rows leave threads of a block idle, and rows that are no multiple of 8 values
// go by pairs or single values: 65536 x 8 of 256 in bf16 dispatch 48.5, combine 59.2,
// gradient 91.0 us (0.92, 0.76 and 0.93 of the copy rate), of 128 35.3, 54.5 and 68.6
// (0.64, 0.42, 0.63); 32768 x 8 of 1026 142, 225 and 251 (0.63, 0.40, 0.67), of 1001 210,
// 354 and 305 (0.42, 0.25, 0.54), of 1028 in fp32 199, 222 and 360 (0.90, 0.81, 0.94).
#include <cuda_bf16.h>

#include "moe_around.h"
#include "moe_launch.h"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kSlots = 8;   // slots whose rows are on their way at once
constexpr int kGradThreads = 256;

// V values of a row as they lie in memory, and as numbers
template <typename T, int V>
struct Piece {
    T v[V];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (sizeof(T) * V >= 16) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) * V / 16; ++i)
                reinterpret_cast<uint4 *>(v)[i] = reinterpret_cast<const uint4 *>(p)[i];
        } else if constexpr (sizeof(T) * V == 8) {
            *reinterpret_cast<uint2 *>(v) = *reinterpret_cast<const uint2 *>(p);
        } else if constexpr (sizeof(T) * V == 4) {
            *reinterpret_cast<uint32_t *>(v) = *reinterpret_cast<const uint32_t *>(p);
        } else {
            *reinterpret_cast<uint16_t *>(v) = *reinterpret_cast<const uint16_t *>(p);
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (sizeof(T) * V >= 16) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) * V / 16; ++i)
                reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(v)[i];
        } else if constexpr (sizeof(T) * V == 8) {
            *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(v);
        } else if constexpr (sizeof(T) * V == 4) {
            *reinterpret_cast<uint32_t *>(p) = *reinterpret_cast<const uint32_t *>(v);
        } else {
            *reinterpret_cast<uint16_t *>(p) = *reinterpret_cast<const uint16_t *>(v);
        }
    }
    __device__ __forceinline__ float get(int i) const { return (float)v[i]; }
    __device__ __forceinline__ void set(int i, float f) { v[i] = (T)f; }
};
template <typename T, int V>
struct alignas(16) AlignedPiece : Piece<T, V> {};

struct RowArgs {
    const void *from, *addend;   // rows read: tokens' (dispatch), places' (combine)
    void *to;
    const int32_t *pos;
    const float *weights;
    int T, k, n, M;
    int chunks;                  // blocks a token's row takes
};

// xs[pos[t][s]] = x[t], bit for bit
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const RowArgs a) {
    const int t = blockIdx.x / a.chunks, j = ((blockIdx.x % a.chunks) * kThreads + threadIdx.x) * V;
    if (j >= a.n) return;
    AlignedPiece<T, V> p;
    p.load(static_cast<const T *>(a.from) + (size_t)t * a.n + j);
    for (int s = 0; s < a.k; ++s) {
        const int at = a.pos[(size_t)t * a.k + s];
        if ((unsigned)at < (unsigned)a.M) p.store(static_cast<T *>(a.to) + (size_t)at * a.n + j);
    }
}

// y[t] = addend[t] + sum_s w[t][s] o[pos[t][s]]
template <typename TO, typename TY, int V>
__global__ void __launch_bounds__(kThreads) combine_kernel(const RowArgs a) {
    const int t = blockIdx.x / a.chunks, j = ((blockIdx.x % a.chunks) * kThreads + threadIdx.x) * V;
    if (j >= a.n) return;
    float sum[V] = {};
    if (a.addend) {
        AlignedPiece<TY, V> p;
        p.load(static_cast<const TY *>(a.addend) + (size_t)t * a.n + j);
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] = p.get(i);
    }
    for (int s0 = 0; s0 < a.k; s0 += kSlots) {
        AlignedPiece<TO, V> p[kSlots];
        float w[kSlots];
        bool live[kSlots];
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            const int at = s0 + s < a.k ? a.pos[(size_t)t * a.k + s0 + s] : -1;
            live[s] = (unsigned)at < (unsigned)a.M;
            w[s] = live[s] && a.weights ? a.weights[(size_t)t * a.k + s0 + s] : 1.f;
            if (live[s]) p[s].load(static_cast<const TO *>(a.from) + (size_t)at * a.n + j);
        }
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
            if (live[s]) {
#pragma unroll
                for (int i = 0; i < V; ++i) sum[i] = fmaf(w[s], p[s].get(i), sum[i]);
            }
    }
    AlignedPiece<TY, V> out;
#pragma unroll
    for (int i = 0; i < V; ++i) out.set(i, sum[i]);
    out.store(static_cast<TY *>(a.to) + (size_t)t * a.n + j);
}

struct GradArgs {
    const void *dy, *o;
    void *d_o;
    const int32_t *pos;
    const float *weights;
    float *dweights;
    int T, k, n, M;
    int groups;   // blocks a token's slots take
};

// d_o[pos[t][s]] = w[t][s] dy[t], dweights[t][s] = <o[pos[t][s]], dy[t]>: a block takes whole rows of S slots, so that it
// has the dots to itself
template <typename TO, typename TY, int V, int S>
__global__ void __launch_bounds__(kGradThreads) combine_grad_kernel(const GradArgs a) {
    __shared__ float part[kGradThreads / 32][S];
    const int t = blockIdx.x / a.groups, s0 = (blockIdx.x % a.groups) * S;
    const int have = min(S, a.k - s0), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float w[S], dot[S] = {};
    int at[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        at[s] = s < have ? a.pos[(size_t)t * a.k + s0 + s] : -1;
        if ((unsigned)at[s] >= (unsigned)a.M) at[s] = -1;
        w[s] = at[s] >= 0 && a.weights ? a.weights[(size_t)t * a.k + s0 + s] : 1.f;
    }
    for (int j = threadIdx.x * V; j < a.n; j += blockDim.x * V) {
        AlignedPiece<TY, V> dy;
        AlignedPiece<TO, V> o[S];
        dy.load(static_cast<const TY *>(a.dy) + (size_t)t * a.n + j);
        if (a.dweights) {
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (at[s] >= 0) o[s].load(static_cast<const TO *>(a.o) + (size_t)at[s] * a.n + j);
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (at[s] < 0) continue;
            if (a.dweights) {
#pragma unroll
                for (int i = 0; i < V; ++i) dot[s] = fmaf(o[s].get(i), dy.get(i), dot[s]);
            }
            if (a.d_o) {
                AlignedPiece<TO, V> d;
#pragma unroll
                for (int i = 0; i < V; ++i) d.set(i, w[s] * dy.get(i));
                d.store(static_cast<TO *>(a.d_o) + (size_t)at[s] * a.n + j);
            }
        }
    }
    if (!a.dweights) return;
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) dot[s] += __shfl_xor_sync(0xFFFFFFFFu, dot[s], off);
        if (lane == 0) part[warp][s] = dot[s];
    }
    __syncthreads();
    if (threadIdx.x < have) {
        float sum = part[0][threadIdx.x];
        for (int i = 1; i < (int)blockDim.x / 32; ++i) sum += part[i][threadIdx.x];
        a.dweights[(size_t)t * a.k + s0 + threadIdx.x] = sum;
    }
}

// values of a thread's piece: rows start on a 16-byte boundary, on that of a pair, or of a value
int values(int n) { return n % 8 == 0 ? 8 : n % 2 == 0 ? 2 : 1; }

template <typename T>
cudaError_t dispatch_t(RowArgs a, cudaStream_t s) {
    const int v = values(a.n);
    a.chunks = (a.n + v * kThreads - 1) / (v * kThreads);
    const unsigned grid = (unsigned)((long long)a.T * a.chunks);
    if (v == 8) dispatch_kernel<T, 8><<<grid, kThreads, 0, s>>>(a);
    else if (v == 2) dispatch_kernel<T, 2><<<grid, kThreads, 0, s>>>(a);
    else dispatch_kernel<T, 1><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename TO, typename TY>
cudaError_t combine_t(RowArgs a, cudaStream_t s) {
    const int v = values(a.n);
    a.chunks = (a.n + v * kThreads - 1) / (v * kThreads);
    const unsigned grid = (unsigned)((long long)a.T * a.chunks);
    if (v == 8) combine_kernel<TO, TY, 8><<<grid, kThreads, 0, s>>>(a);
    else if (v == 2) combine_kernel<TO, TY, 2><<<grid, kThreads, 0, s>>>(a);
    else combine_kernel<TO, TY, 1><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename TO, typename TY, int S>
cudaError_t combine_grad_s(GradArgs a, cudaStream_t s) {
    const int v = values(a.n);
    a.groups = (a.k + S - 1) / S;
    const unsigned grid = (unsigned)(a.T * a.groups);
    // the fewest rounds of a block's threads over a row, and of those the same number each
    const int pieces = (a.n + v - 1) / v, rounds = (pieces + kGradThreads - 1) / kGradThreads;
    const int threads = ((pieces + rounds - 1) / rounds + 31) / 32 * 32;
    if (v == 8) combine_grad_kernel<TO, TY, 8, S><<<grid, threads, 0, s>>>(a);
    else if (v == 2) combine_grad_kernel<TO, TY, 2, S><<<grid, threads, 0, s>>>(a);
    else combine_grad_kernel<TO, TY, 1, S><<<grid, threads, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename TO, typename TY>
cudaError_t combine_grad_t(const GradArgs &a, cudaStream_t s) {
    // few rows: a block a slot, and the token's row is read by each
    if ((long long)a.T * a.k <= 4 * num_sms()) return combine_grad_s<TO, TY, 1>(a, s);
    return a.k <= 4 ? combine_grad_s<TO, TY, 4>(a, s) : combine_grad_s<TO, TY, 8>(a, s);
}

}  // namespace

cudaError_t launch_dispatch_rows(const void *x, int dtype, const int32_t *pos, int T, int k, int n, int M, void *xs,
                                 cudaStream_t s) {
    RowArgs a = {};
    a.from = x;
    a.to = xs;
    a.pos = pos;
    a.T = T;
    a.k = k;
    a.n = n;
    a.M = M;
    return dtype == MOE_DT_BF16 ? dispatch_t<__nv_bfloat16>(a, s) : dispatch_t<float>(a, s);
}

cudaError_t launch_combine_rows(const void *o, int dtype, const int32_t *pos, const float *weights, int T, int k,
                                int n, int M, const void *addend, void *y, int ydtype, cudaStream_t s) {
    const RowArgs a = {o, addend, y, pos, weights, T, k, n, M, 0};
    if (dtype == MOE_DT_BF16)
        return ydtype == MOE_DT_BF16 ? combine_t<__nv_bfloat16, __nv_bfloat16>(a, s) : combine_t<__nv_bfloat16, float>(a, s);
    return ydtype == MOE_DT_BF16 ? combine_t<float, __nv_bfloat16>(a, s) : combine_t<float, float>(a, s);
}

cudaError_t launch_combine_grad(const void *dy, int ydtype, const int32_t *pos, const float *weights, int T, int k,
                                int n, int M, const void *o, int dtype, void *d_o, float *dweights, cudaStream_t s) {
    const GradArgs a = {dy, o, d_o, pos, weights, dweights, T, k, n, M, 0};
    if (dtype == MOE_DT_BF16)
        return ydtype == MOE_DT_BF16 ? combine_grad_t<__nv_bfloat16, __nv_bfloat16>(a, s)
                                     : combine_grad_t<__nv_bfloat16, float>(a, s);
    return ydtype == MOE_DT_BF16 ? combine_grad_t<float, __nv_bfloat16>(a, s) : combine_grad_t<float, float>(a, s);
}

}  // namespace moe
