// moe_router_stats.cu - what a router's choice gives beside the ids: the
// pairs sorted by expert with counts and offsets (moe_expert_order), and the
// balance loss with its gradient (moe_balance_loss).
#include <cuda_bf16.h>

#include "moe_around.h"
#include "moe_launch.h"
#include "moe_router.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------- expert order
//
// A stable counting sort by expert.  The pairs are cut into chunks of
// kOrderChunk, one block each; in a chunk, warp w takes the w-th run of
// 32 * kOrderIters pairs, 32 at a time in order.  Lanes with the same expert
// find one another with one ballot for each bit of its number (a match vote of
// 32 warps took 2,200 cycles, the ballots take 400), so a pair's rank among the
// run's pairs of its expert is the run's count so far plus the earlier lanes
// of its vote: no atomics, and the order is that of the pairs.
//   order_count : chunk b's pairs per expert -> hist[b][E]
//   order_place : place = offsets[e] + sum of hist[b' < b][e] + the chunk's
//                 earlier runs + rank
// order_place starts while order_count still runs (its votes need only the
// ids) and waits for it before it reads hist.  One chunk needs no hist:
// order_place counts it itself, in one launch.
// Few pairs: the launch and the chain of votes bound it.  Many: the votes, the
// 4-byte scatter of rows, and the counts of the chunks, all of which each block
// reads: 2 MB of hist by 1024 blocks for 2^22 pairs over 1024 experts, 2.1 GB in
// all.  524288 pairs over 256 experts take 11.5 us on the device, 2^20 22, 2^22
// 110; 2^22 over 64 experts 70, over 1024 272.
constexpr int kOrderWarps = 32;
constexpr int kOrderThreads = 32 * kOrderWarps;
constexpr int kOrderIters = 4;
constexpr int kOrderChunk = kOrderThreads * kOrderIters;   // 4096; counts in a chunk fit 16 bits

// counts of a chunk in hist: 16 bits each, rows of whole 16-byte pieces
__host__ __device__ constexpr int hist_pitch(int E) { return (E + 7) & ~7; }
// dynamic shared memory of order_place: base and total in 32 bits, the runs in 16 (72 KB at E = 1024)
constexpr int order_place_smem(int E) {
    return hist_pitch(E) * (int)(2 * sizeof(int32_t) + kOrderWarps * sizeof(uint16_t));
}

__global__ void __launch_bounds__(kOrderThreads) order_count(const int32_t *__restrict__ ids, int n, int E,
                                                   uint16_t *__restrict__ hist) {
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
    const int pitch = hist_pitch(E);
    for (int e = threadIdx.x; e < pitch; e += blockDim.x)
        hist[(size_t)blockIdx.x * pitch + e] = e < E ? (uint16_t)cnt[e] : 0;
}

__global__ void __launch_bounds__(kOrderThreads) order_place(const int32_t *__restrict__ ids, int n, int k, int E,
                                                   const uint16_t *hist, int32_t *__restrict__ counts,
                                                   int32_t *__restrict__ offsets, int32_t *__restrict__ rows,
                                                   int32_t *__restrict__ pos) {
    extern __shared__ int32_t sm[];
    const int pitch = hist_pitch(E), pieces = pitch / 8;
    int32_t *base = sm;                                            // [E] first place of this chunk's pairs
    int32_t *total = sm + pitch;                                   // [E] pairs of an expert in all chunks
    uint16_t *run = reinterpret_cast<uint16_t *>(sm + 2 * pitch);  // [kOrderWarps][pitch]
    __shared__ int32_t wsum[kOrderWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // this chunk's pairs in runs of 32 * iters, one a warp: few pairs take few votes in a row
    const int chunk0 = blockIdx.x * kOrderChunk, have = min(n - chunk0, kOrderChunk);
    const int iters = (have + kOrderThreads - 1) / kOrderThreads;
    const int used = iters ? (have + 32 * iters - 1) / (32 * iters) : 0;   // warps with pairs
    for (int i = threadIdx.x; i < used * pieces; i += blockDim.x)
        reinterpret_cast<uint4 *>(run)[i] = make_uint4(0, 0, 0, 0);
    for (int e = threadIdx.x; e < 2 * pitch; e += blockDim.x) base[e] = 0;   // total too
    __syncthreads();

    // votes: this lane's pairs, their experts and ranks within the warp's run
    const int first = chunk0 + warp * 32 * iters;
    uint16_t *mine = run + warp * pitch;
    const int bits = 32 - __clz(E);   // of 0 .. E: E stands for a pair that takes no part
    int key[kOrderIters], rank[kOrderIters];
#pragma unroll
    for (int j = 0; j < kOrderIters; ++j) {
        const int i = first + 32 * j + lane;
        const int id = j < iters && i < n ? ids[i] : -1;
        key[j] = (unsigned)id < (unsigned)E ? id : E;
    }
    unsigned same[kOrderIters];
#pragma unroll
    for (int j = 0; j < kOrderIters; ++j) same[j] = 0xFFFFFFFFu;
    const auto vote = [&](int j, int b) {
        const bool one = (key[j] >> b) & 1;
        const unsigned with = __ballot_sync(0xFFFFFFFFu, one);
        same[j] &= one ? with : ~with;
    };
    // (not unrolled: a small call is bound by its launch and the fetch of its instructions)
    if (iters == 1) {
#pragma unroll 1
        for (int b = 0; b < bits; ++b) vote(0, b);
    } else {
#pragma unroll 1
        for (int b = 0; b < bits; ++b)
#pragma unroll
            for (int j = 0; j < kOrderIters; ++j) vote(j, b);
    }
#pragma unroll
    for (int j = 0; j < kOrderIters; ++j) {
        rank[j] = 0;
        if (j >= iters || first + 32 * j >= n) continue;   // uniform over the warp
        const int before = __popc(same[j] & ((1u << lane) - 1u));
        const int old = key[j] < E ? mine[key[j]] : 0;
        __syncwarp();
        if (key[j] < E && before == 0) mine[key[j]] = (uint16_t)(old + __popc(same[j]));
        __syncwarp();
        rank[j] = old + before;
    }
    // pairs of the chunks before this one, and of all
    if (hist) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        // a thread takes 8 experts (one 16-byte piece) of every P-th chunk; experts e, e + 1, ... of a piece are
        // `pieces` words apart in base and total until they are read, which keeps the additions free of conflicts
        const int P = kOrderThreads / pieces, q = threadIdx.x % pieces, p = threadIdx.x / pieces;
        if (p < P) {
            int b[8] = {}, s8[8] = {};
#pragma unroll 8
            for (int ch = p; ch < (int)gridDim.x; ch += P) {
                const uint4 v = reinterpret_cast<const uint4 *>(hist + (size_t)ch * pitch)[q];
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                const bool before = ch < (int)blockIdx.x;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int h = (w[i / 2] >> (16 * (i & 1))) & 0xFFFF;
                    s8[i] += h;
                    b[i] += before ? h : 0;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (b[i]) atomicAdd(base + i * pieces + q, b[i]);
                if (s8[i]) atomicAdd(total + i * pieces + q, s8[i]);
            }
        }
    }
    __syncthreads();
    // the runs before each run of this chunk
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int sum = 0;
#pragma unroll 4
        for (int w = 0; w < used; ++w) {
            const int c = run[w * pitch + e];
            run[w * pitch + e] = (uint16_t)sum;
            sum += c;
        }
        if (!hist) total[e] = sum;
    }
    __syncthreads();
    // offsets: exclusive prefix sums over the experts, one a thread
    const int e = threadIdx.x, at = hist ? (e & 7) * pieces + (e >> 3) : e;
    const int c = e < E ? total[at] : 0, before = e < E ? base[at] : 0;
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
        base[e] = before + o;
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
        const int place = key[j] < E ? base[key[j]] + mine[key[j]] + rank[j] : -1;
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
// its d_e stay in registers, and it walks over the rows, the next row's loads
// under way while it adds up one.  The instructions of a row and the chain of
// its reductions bound it: at 65536 x 256 fp32 58% of the issue slots are taken
// and 38% of the DRAM rate, and half the bytes (bf16) take 22.1 us instead of 28.5.
//
// Sums: a row in fp32, a warp's rows in fp32 with the rounding of each addition
// carried over to the next (a count holds the ones of 1 + q), a block's warps
// and the blocks in double, in order (the last block to finish adds the
// blocks).  A plain fp32 sum of a warp's rows (3,450 of 2^24) was off by up to
// 500 u where the rows are alike, u = 2^-24; the carried one by 2.  This part has
// few units for double arithmetic: an addition a row cost a third of the
// kernel's time, and one for every 32 rows, behind a branch, a tenth at E = 8.
// exp and the reciprocal of sigma are the machine's own, flushing below 2^-126
// (exp is off by 2 ulp and |l - m| u, the reciprocal by 1 ulp): with the library
// functions the kernel was bound by issue slots (350 instructions a row of 256).
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

// 1/x for x in [1, 2]
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// J vectors of VEC values a lane: value i of vector j is expert 32*VEC*j + VEC*lane + i.
// Blocks of a launch that share an SM (one row, its d and the next row take 3 to 4 registers a value), 65536 rows fp32:
// E = 256, 8 values: 28.5 us with 4, 31.9 with 2; E = 257, 16 values: 37.6 with 2, 87.5 with 4 (spills); E = 64,
// 2 values: 16.0 with 4, 17.0 with 8.
constexpr int balance_per_sm(int values) { return values <= 8 ? 4 : 2; }

template <typename T, bool SIGMOID, int VEC, int J>
__global__ void __launch_bounds__(32 * kBalanceWarps, balance_per_sm(VEC * J)) balance_kernel(const BalanceArgs a) {
    __shared__ double part[kBalanceWarps];
    __shared__ int last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E;
    const int step = gridDim.x * kBalanceWarps;
    Raw<T, VEC> next[J];
    bool next_live = false;
    const auto fetch = [&](int t) {
        next_live = !a.valid || a.valid[t];
        if (!next_live) return;
        const T *row = static_cast<const T *>(a.logits) + (size_t)t * E;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int e = 32 * VEC * j + VEC * lane;
            if (e < E) next[j].load(row + e);
        }
    };
    int t = blockIdx.x * kBalanceWarps + warp;
    if (t < a.T) fetch(t);   // on its way while the counts are added up
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

    float sum = 0.f, over = 0.f;   // of q; by how much it is too large
    int rows = 0;                  // rows that count
    for (; t < a.T; t += step) {
        T *out = a.dlogits ? static_cast<T *>(a.dlogits) + (size_t)t * E : nullptr;
        float p[J][VEC];
        float m = -INFINITY;
        const bool live = next_live && N > 0;
        if (live) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int e = 32 * VEC * j + VEC * lane;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    p[j][i] = e < E ? next[j].value(i) : -INFINITY;
                    m = max_nan(m, p[j][i]);
                }
            }
        }
        if (t + step < a.T) fetch(t + step);
        if (live) m = warp_max(m);
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
        float ps[SIGMOID ? J : 1][VEC];   // sigma (1 - sigma), up to the factor of p
        if constexpr (SIGMOID) {
            // with u = e^-|l| and r = 1 / (1 + u): sigma is r or u r, 1 - sigma the other one
            if (m >= 0.f) {
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float l = p[j][i], u = exp_fast(-fabsf(l)), r = rcp_fast(1.f + u), ur = u * r;
                        ps[j][i] = ur * r;
                        p[j][i] = l > 0.f ? r : ur;
                    }
            } else {
                // all logits below 0: sigma e^-m with the largest logit m.  The factor falls out of the ratio,
                // and rows far below 0 keep their probabilities where sigma itself would vanish.
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float l = p[j][i], r = rcp_fast(1.f + exp_fast(l));
                        p[j][i] = exp_fast(l - m) * r;
                        ps[j][i] = p[j][i] * r;
                    }
            }
        } else {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) p[j][i] = exp_fast(p[j][i] - m);
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
        const float term = q - over, up = sum + term;
        over = (up - sum) - term;
        sum = up;
        ++rows;
        if (out) {
            const float g = gcoef * inv;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int e = 32 * VEC * j + VEC * lane;
#pragma unroll
                for (int i = 0; i < VEC; ++i) p[j][i] = (SIGMOID ? ps[SIGMOID ? j : 0][i] : p[j][i]) * (g * (d[j][i] - q));
                if (e < E) store_vec<T, VEC>(out + e, p[j]);
            }
        }
    }
    if (!a.loss) return;
    if (lane == 0) part[warp] = (double)(sum - over) + rows;
    __syncthreads();
    if (threadIdx.x == 0) {
        double b = 0.0;
        for (int w = 0; w < kBalanceWarps; ++w) b += part[w];
        __stcg(a.partial + blockIdx.x, b);
        __threadfence();
        last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double b = 0.0;
    for (int i = threadIdx.x; i < (int)gridDim.x; i += 32 * kBalanceWarps) b += __ldcg(a.partial + i);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) b += __shfl_xor_sync(0xFFFFFFFFu, b, off);
    if (lane == 0) part[warp] = b;
    __syncthreads();
    if (threadIdx.x == 0) {
        b = 0.0;
        for (int w = 0; w < kBalanceWarps; ++w) b += part[w];
        a.loss[0] = (float)((double)a.alpha * b * (N > 0 ? (double)a.k / (double)N : 0.0));
        *a.ticket = 0;   // ready for the next call
    }
}

constexpr int kBalanceBlocks = 1024;   // most blocks of a launch (the workspace's partial sums)

template <typename T, bool SIGMOID, int VEC, int J>
void launch_balance_k(const BalanceArgs &a, cudaStream_t s) {
    // all blocks resident at once, each walking over its share of the rows; one row a warp where there are few
    const int want = (a.T + kBalanceWarps - 1) / kBalanceWarps, most = balance_per_sm(VEC * J) * num_sms();
    const int b = min(max(min(want, most), 1), kBalanceBlocks);
    balance_kernel<T, SIGMOID, VEC, J><<<b, 32 * kBalanceWarps, 0, s>>>(a);
}

template <typename T, bool SIGMOID>
cudaError_t launch_balance_t(const BalanceArgs &a, cudaStream_t s) {
    // up to 64 experts: every lane has one or two (65536 x 64: 16.0 us; with 4 a lane half of them idle, 18.2)
    if (a.E <= 64) {
        launch_balance_k<T, SIGMOID, 1, 2>(a, s);
        return cudaGetLastError();
    }
    // rows whose length is a multiple of 4 are read 4 values at a time (16384 x 1024: 36 us, value by value 47;
    // 65536 x 256 bf16: 25.4, 26.8)
    if (a.E % 4 == 0) {
        if (a.E <= 128) launch_balance_k<T, SIGMOID, 4, 1>(a, s);
        else if (a.E <= 256) launch_balance_k<T, SIGMOID, 4, 2>(a, s);
        else if (a.E <= 512) launch_balance_k<T, SIGMOID, 4, 4>(a, s);
        else launch_balance_k<T, SIGMOID, 4, 8>(a, s);
    } else {
        if (a.E <= 128) launch_balance_k<T, SIGMOID, 1, 4>(a, s);
        else if (a.E <= 256) launch_balance_k<T, SIGMOID, 1, 8>(a, s);
        else if (a.E <= 512) launch_balance_k<T, SIGMOID, 1, 16>(a, s);
        else launch_balance_k<T, SIGMOID, 1, 32>(a, s);
    }
    return cudaGetLastError();
}

}  // namespace

size_t order_ws_bytes(int T, int k, int E) {
    const long long n = (long long)T * k, chunks = (n + kOrderChunk - 1) / kOrderChunk;
    return chunks > 1 ? (size_t)chunks * hist_pitch(E) * sizeof(uint16_t) : 0;
}

cudaError_t launch_order(const int32_t *ids, int T, int k, int E, int32_t *counts, int32_t *offsets, int32_t *rows,
                         int32_t *pos, void *ws, cudaStream_t s) {
    const int n = T * k;
    const int chunks = n > 0 ? (n + kOrderChunk - 1) / kOrderChunk : 1;
    uint16_t *hist = chunks > 1 ? static_cast<uint16_t *>(ws) : nullptr;
    const size_t smem = (size_t)order_place_smem(E);
    cudaError_t err = cudaSuccess;
    // The limit belongs to the kernel, not to the launch: one value whatever E is, so that a call on another host
    // thread cannot lower it between here and the launch.
    if (smem > 48 * 1024)
        err = cudaFuncSetAttribute(order_place, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   order_place_smem(MOE_MAX_EXPERTS));
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
    return cudaLaunchKernelEx(&cfg, order_place, ids, n, k, E, (const uint16_t *)hist, counts, offsets, rows, pos);
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
