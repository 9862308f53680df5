// moe_router_stats.cu - what a router's choice gives beside the ids: the
// pairs sorted by expert with counts and offsets (moe_expert_order), and the
// balance loss with its gradient (moe_balance_loss).
#include <cuda_bf16.h>

#include "moe_launch.h"

namespace moe {
namespace {

// ---------------------------------------------------------- expert order
//
// A stable counting sort by expert.  The pairs are cut into chunks of
// kOrderChunk, one block each; in a chunk, warp w takes the w-th run of
// 32 * kOrderIters pairs, 32 at a time in order.  Lanes with the same expert
// find one another with a match vote, so a pair's rank among the run's pairs
// of its expert is the run's count so far plus the earlier lanes of its vote:
// no atomics, and the order is that of the pairs.
//   order_count : chunk b's pairs per expert -> hist[b][E]
//   order_place : place = offsets[e] + sum of hist[b' < b][e] + the chunk's
//                 earlier runs + rank
// order_place starts while order_count still runs (its votes need only the
// ids) and waits for it before it reads hist.  One chunk needs no hist:
// order_place counts it itself, in one launch.
// Few pairs: the launches and the chain of votes bound it; many: the votes
// and the 4-byte scatter of rows.
constexpr int kOrderWarps = 32;
constexpr int kOrderThreads = 32 * kOrderWarps;
constexpr int kOrderIters = 8;
constexpr int kOrderChunk = kOrderThreads * kOrderIters;   // 8192; counts in a chunk fit 16 bits

__global__ void __launch_bounds__(kOrderThreads) order_count(const int32_t *__restrict__ ids, int n, int E,
                                                   int32_t *__restrict__ hist) {
    extern __shared__ int32_t cnt[];
    asm volatile("griddepcontrol.launch_dependents;");
    for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = 0;
    __syncthreads();
    const int first = blockIdx.x * kOrderChunk;
#pragma unroll
    for (int j = 0; j < kOrderIters; ++j) {
        const int i = first + j * kOrderThreads + threadIdx.x;
        const int id = i < n ? ids[i] : -1;
        if ((unsigned)id < (unsigned)E) atomicAdd(cnt + id, 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[(size_t)blockIdx.x * E + e] = cnt[e];
}

__global__ void __launch_bounds__(kOrderThreads) order_place(const int32_t *__restrict__ ids, int n, int k, int E,
                                                   const int32_t *hist, int32_t *__restrict__ counts,
                                                   int32_t *__restrict__ offsets, int32_t *__restrict__ rows,
                                                   int32_t *__restrict__ pos) {
    extern __shared__ int32_t sm[];
    int32_t *base = sm;                                          // [E] first place of this chunk's pairs
    int32_t *total = sm + E;                                     // [E] pairs of an expert in all chunks
    uint16_t *run = reinterpret_cast<uint16_t *>(sm + 2 * E);    // [kOrderWarps][E]
    __shared__ int32_t wsum[kOrderWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // this chunk's pairs in runs of 32 * iters, one a warp: few pairs take few votes in a row
    const int chunk0 = blockIdx.x * kOrderChunk, have = min(n - chunk0, kOrderChunk);
    const int iters = (have + kOrderThreads - 1) / kOrderThreads;
    const int used = iters ? (have + 32 * iters - 1) / (32 * iters) : 0;   // warps with pairs
    for (int i = threadIdx.x; i < used * E; i += blockDim.x) run[i] = 0;
    for (int e = threadIdx.x; e < E; e += blockDim.x) base[e] = total[e] = 0;
    __syncthreads();

    // votes: this lane's pairs, their experts and ranks within the warp's run
    const int first = chunk0 + warp * 32 * iters;
    uint16_t *mine = run + warp * E;
    int key[kOrderIters], rank[kOrderIters];
#pragma unroll
    for (int j = 0; j < kOrderIters; ++j) {
        const int i = first + 32 * j + lane;
        const int id = j < iters && i < n ? ids[i] : -1;
        key[j] = (unsigned)id < (unsigned)E ? id : -1;
    }
#pragma unroll
    for (int j = 0; j < kOrderIters; ++j) {
        rank[j] = 0;
        if (j >= iters || first + 32 * j >= n) continue;   // uniform over the warp
        const unsigned same = __match_any_sync(0xFFFFFFFFu, key[j]);
        const int before = __popc(same & ((1u << lane) - 1u));
        const int old = key[j] >= 0 ? mine[key[j]] : 0;
        __syncwarp();
        if (key[j] >= 0 && before == 0) mine[key[j]] = (uint16_t)(old + __popc(same));
        __syncwarp();
        rank[j] = old + before;
    }
    // pairs of the chunks before this one, and of all
    if (hist) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        // P threads share an expert's column of hist (kOrderThreads >= MOE_MAX_EXPERTS: every expert has one)
        const int P = min(kOrderThreads / E, (int)gridDim.x), e = threadIdx.x % E, p = threadIdx.x / E;
        if (p < P) {
            int b = 0, t = 0;
#pragma unroll 16
            for (int ch = p; ch < (int)gridDim.x; ch += P) {
                const int h = hist[(size_t)ch * E + e];
                t += h;
                if (ch < (int)blockIdx.x) b += h;
            }
            if (P == 1) {
                base[e] = b;
                total[e] = t;
            } else {
                atomicAdd(base + e, b);
                atomicAdd(total + e, t);
            }
        }
    }
    __syncthreads();
    // the runs before each run of this chunk
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int sum = 0;
#pragma unroll 8
        for (int w = 0; w < used; ++w) {
            const int c = run[w * E + e];
            run[w * E + e] = (uint16_t)sum;
            sum += c;
        }
        if (!hist) total[e] = sum;
    }
    __syncthreads();
    // offsets: exclusive prefix sums over the experts, one a thread
    const int e = threadIdx.x, c = e < E ? total[e] : 0;
    int s = c;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, s, off);
        if (lane >= off) s += o;
    }
    if (lane == 31) wsum[warp] = s;
    __syncthreads();
    int up = wsum[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, up, off);
        if (lane >= off) up += o;
    }
    const int live = __shfl_sync(0xFFFFFFFFu, up, 31);
    up = warp ? __shfl_sync(0xFFFFFFFFu, up, (warp + 31) & 31) : 0;
    if (e < E) {
        const int o = up + s - c;
        base[e] += o;
        if (blockIdx.x == 0) {
            if (counts) counts[e] = c;
            if (offsets) offsets[e] = o;
        }
    }
    if (blockIdx.x == 0 && e == 0 && offsets) offsets[E] = live;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kOrderIters; ++j) {
        const int i = first + 32 * j + lane;
        if (j >= iters || i >= n) continue;
        const int place = key[j] >= 0 ? base[key[j]] + mine[key[j]] + rank[j] : -1;
        if (pos) pos[i] = place;
        if (rows && place >= 0) rows[place] = (unsigned)i / (unsigned)k;
        if (rows && i >= live) rows[i] = -1;
    }
}

// ---------------------------------------------------------- balance loss
//
// loss = alpha k/N sum_t sum_e f_e p_te with f_e = E c_e / N.  Since the
// probabilities of a token add up to 1, f_e = 1 + d_e with
// d_e = (E c_e - N) / N, whose numerator is exact in integers, gives
//   q_t = sum_e p_te d_e,   loss = alpha k/N sum_t (1 + q_t),
//   dloss/dl_te = alpha k/N p_te (d_e - q_t)   [times 1 - sigma(l_te)]
// and d_e - q_t keeps its digits where f_e - sum f p would lose them (even
// counts: both are close to 1).  The counts are known before the pass, so
// loss and gradient come from one reading of the logits: a warp holds a row,
// its d_e stay in registers, and it walks over the rows.  Bandwidth bounds it.
//
// Sums: a row and a warp's few rows in fp32 (a count holds the ones of 1 + q),
// a block's warps and the blocks in double, in order (the last block to finish
// adds the blocks).  Double arithmetic stays out of the loop: this part has few
// units for it, and one addition a row cost a third of the kernel's time.
// exp and the reciprocal of sigma are the fast ones (2 ulp and |l - m| u, 1 ulp):
// the accurate ones made the kernel issue-bound (70% of issue slots).
constexpr int kBalanceWarps = 8;

struct BalanceArgs {
    const void *logits;
    const int32_t *counts;
    const uint8_t *valid;
    const float *grad_loss;
    float *loss;
    void *dlogits;
    unsigned *ticket;     // ws
    double *partial;      // ws [blocks]
    float alpha;
    int T, E, k;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// VEC consecutive values of a row (VEC 1: any alignment)
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T *p, float v[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = (float)p[0];
    } else if constexpr (sizeof(T) == 4) {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    } else {
        const uint2 a = *reinterpret_cast<const uint2 *>(p);
        v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xFFFF0000u);
        v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xFFFF0000u);
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

// J vectors of VEC values a lane: value i of vector j is expert 32*VEC*j + VEC*lane + i
template <typename T, bool SIGMOID, int VEC, int J>
__global__ void __launch_bounds__(32 * kBalanceWarps) balance_kernel(const BalanceArgs a) {
    __shared__ double part[kBalanceWarps];
    __shared__ int last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E;
    float d[J][VEC];
    long long N = 0;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int e = 32 * VEC * j + VEC * lane + i;
            const int c = e < E ? a.counts[e] : 0;
            N += c;
            d[j][i] = __int_as_float(c);
        }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) N += __shfl_xor_sync(0xFFFFFFFFu, N, off);
    const float coef = N > 0 ? a.alpha * ((float)a.k / (float)N) : 0.f;
    const float gcoef = a.grad_loss ? coef * a.grad_loss[0] : coef;
    const float invN = N > 0 ? 1.f / (float)N : 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) d[j][i] = (float)((long long)__float_as_int(d[j][i]) * E - N) * invN;

    float sum = 0.f;   // of q
    int rows = 0;      // rows that count
    const int step = gridDim.x * kBalanceWarps;
    for (int t = blockIdx.x * kBalanceWarps + warp; t < a.T; t += step) {
        const T *row = static_cast<const T *>(a.logits) + (size_t)t * E;
        T *out = a.dlogits ? static_cast<T *>(a.dlogits) + (size_t)t * E : nullptr;
        float p[J][VEC];
        float m = -INFINITY;
        const bool live = N > 0 && (!a.valid || a.valid[t]);
        if (live) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int e = 32 * VEC * j + VEC * lane;
#pragma unroll
                for (int i = 0; i < VEC; ++i) p[j][i] = -INFINITY;
                if (e < E) load_vec<T, VEC>(row + e, p[j]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) m = fmaxf(m, p[j][i]);
            }
            m = warp_max(m);
        }
        if (!live || m == -INFINITY) {   // uniform over the warp
            if (out) {
                const float zero[VEC] = {};
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int e = 32 * VEC * j + VEC * lane;
                    if (e < E) store_vec<T, VEC>(out + e, zero);
                }
            }
            continue;
        }
        float s = 0.f, q = 0.f;
        float slope[SIGMOID ? J : 1][VEC];   // 1 - sigma(l)
        if constexpr (SIGMOID) {
            // sigma(l) e^-m with m = min(0, the row's largest logit): the
            // factor falls out of the ratio, and rows far below 0 keep their
            // probabilities where sigma itself would vanish
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float l = p[j][i], u = __expf(-fabsf(l)), r = __fdividef(1.f, 1.f + u), ur = u * r;
                    slope[j][i] = l > 0.f ? ur : r;
                    p[j][i] = l > 0.f ? r : m < 0.f ? __expf(l - m) * r : ur;
                }
        } else {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) p[j][i] = __expf(p[j][i] - m);
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                s += p[j][i];
                q = fmaf(p[j][i], d[j][i], q);
            }
        s = warp_sum(s);
        q = warp_sum(q);
        const float inv = __fdiv_rn(1.f, s);
        q *= inv;
        sum += q;
        ++rows;
        if (out) {
            const float g = gcoef * inv;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int e = 32 * VEC * j + VEC * lane;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    p[j][i] *= g * (d[j][i] - q);
                    if constexpr (SIGMOID) p[j][i] *= slope[j][i];
                }
                if (e < E) store_vec<T, VEC>(out + e, p[j]);
            }
        }
    }
    if (!a.loss) return;
    if (lane == 0) part[warp] = (double)sum + rows;
    __syncthreads();
    if (threadIdx.x == 0) {
        double b = 0.0;
        for (int w = 0; w < kBalanceWarps; ++w) b += part[w];
        __stcg(a.partial + blockIdx.x, b);
        __threadfence();
        last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last || warp != 0) return;
    __threadfence();
    double b = 0.0;
    for (int i = lane; i < (int)gridDim.x; i += 32) b += __ldcg(a.partial + i);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) b += __shfl_xor_sync(0xFFFFFFFFu, b, off);
    if (lane == 0) {
        a.loss[0] = (float)((double)a.alpha * b * (N > 0 ? (double)a.k / (double)N : 0.0));
        *a.ticket = 0;   // ready for the next call
    }
}

constexpr int kBalanceBlocks = 1024;   // most blocks of a launch (the workspace's partial sums)

int balance_blocks(int T) {
    // five blocks an SM are resident at most; fewer rows than warps: one row a warp
    const int want = (T + kBalanceWarps - 1) / kBalanceWarps, most = 5 * num_sms();
    const int b = want < most ? want : most;
    return b < 1 ? 1 : b > kBalanceBlocks ? kBalanceBlocks : b;
}

template <typename T, bool SIGMOID>
cudaError_t launch_balance_t(const BalanceArgs &a, cudaStream_t s) {
    const int g = balance_blocks(a.T), th = 32 * kBalanceWarps;
    // rows whose length is a multiple of 4 are read 4 values at a time
    if (a.E % 4 == 0) {
        if (a.E <= 128) balance_kernel<T, SIGMOID, 4, 1><<<g, th, 0, s>>>(a);
        else if (a.E <= 256) balance_kernel<T, SIGMOID, 4, 2><<<g, th, 0, s>>>(a);
        else if (a.E <= 512) balance_kernel<T, SIGMOID, 4, 4><<<g, th, 0, s>>>(a);
        else balance_kernel<T, SIGMOID, 4, 8><<<g, th, 0, s>>>(a);
    } else {
        if (a.E <= 128) balance_kernel<T, SIGMOID, 1, 4><<<g, th, 0, s>>>(a);
        else if (a.E <= 256) balance_kernel<T, SIGMOID, 1, 8><<<g, th, 0, s>>>(a);
        else if (a.E <= 512) balance_kernel<T, SIGMOID, 1, 16><<<g, th, 0, s>>>(a);
        else balance_kernel<T, SIGMOID, 1, 32><<<g, th, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

size_t order_ws_bytes(int T, int k, int E) {
    const long long n = (long long)T * k, chunks = (n + kOrderChunk - 1) / kOrderChunk;
    return chunks > 1 ? (size_t)chunks * E * sizeof(int32_t) : 0;
}

cudaError_t launch_order(const int32_t *ids, int T, int k, int E, int32_t *counts, int32_t *offsets, int32_t *rows,
                         int32_t *pos, void *ws, cudaStream_t s) {
    const int n = T * k;
    const int chunks = n > 0 ? (n + kOrderChunk - 1) / kOrderChunk : 1;
    int32_t *hist = chunks > 1 ? static_cast<int32_t *>(ws) : nullptr;
    // 72 KB at E = 1024
    const size_t smem = (size_t)E * (2 * sizeof(int32_t) + kOrderWarps * sizeof(uint16_t));
    cudaError_t err = cudaSuccess;
    if (smem > 48 * 1024)
        err = cudaFuncSetAttribute(order_place, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)chunks);
    cfg.blockDim = dim3(kOrderThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    if (hist) {
        order_count<<<chunks, kOrderThreads, E * sizeof(int32_t), s>>>(ids, n, E, hist);
        err = cudaGetLastError();
        if (err != cudaSuccess) return err;
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, order_place, ids, n, k, E, (const int32_t *)hist, counts, offsets, rows, pos);
}

size_t balance_ws_bytes() { return 256 + kBalanceBlocks * sizeof(double); }

cudaError_t launch_balance(const void *logits, int dtype, const int32_t *counts, const uint8_t *valid, int T, int E,
                           int k, int gating, float alpha, const float *grad_loss, float *loss, void *dlogits,
                           void *ws, cudaStream_t s) {
    BalanceArgs a;
    a.logits = logits;
    a.counts = counts;
    a.valid = valid;
    a.grad_loss = grad_loss;
    a.loss = loss;
    a.dlogits = dlogits;
    a.ticket = static_cast<unsigned *>(ws);
    a.partial = reinterpret_cast<double *>(static_cast<char *>(ws) + 256);
    a.alpha = alpha;
    a.T = T;
    a.E = E;
    a.k = k;
    if (gating == MOE_GATE_SIGMOID)
        return dtype == MOE_DT_BF16 ? launch_balance_t<__nv_bfloat16, true>(a, s) : launch_balance_t<float, true>(a, s);
    return dtype == MOE_DT_BF16 ? launch_balance_t<__nv_bfloat16, false>(a, s) : launch_balance_t<float, false>(a, s);
}

}  // namespace moe
