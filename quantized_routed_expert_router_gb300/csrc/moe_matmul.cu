// moe_matmul.cu - products of bf16 rows with bf16 matrices, dense or grouped by
// expert, with bias, activation and residual in the epilogue (moe_matmul).
//
// A tile is 128 columns of a matrix by up to BT places of one group.  The columns
// are the rows of the tensor cores' first operand, the places the columns of the
// second: TMEM then gives a lane a column and a register a place, so that
//   - the number of places of a product follows the tile's (16, 32, .. BT);
//   - a lane has its bias in a register, and what a warp reads or writes of a
//     place is 32 columns side by side, wherever rows of y start: nothing is
//     turned in shared memory and no row of another group is touched.
// With the gated activation a tile takes 64 columns of y: gate and up rows in
// turns of 16, by one copy whose map has the two as a dimension, so that lanes l
// and l + 16 of a warp hold the gate and the up value of a column.
//
// The warps of a block have roles:
//   warp 0    : TMA copies of matrix tiles, and of rows that lie in order (64
//               values deep, 128-byte swizzle), into a ring of stages
//   warp 1    : one thread issues the products; the sums of a tile stay in one of
//               the TMEM buffers for the whole depth
//   warps 2-3 : rows that are gathered, by 16-byte asynchronous copies that
//               signal the stage when they land
//   warps 4-11: the epilogue, while the products of the next tile run
// Blocks are persistent, one an SM.  Where there are too few tiles for the SMs a
// cluster of blocks splits the depth of a tile and adds its parts through
// distributed shared memory in rank order.
#include <cuda.h>
#include <cuda_bf16.h>

#include "moe_around.h"
#include "moe_launch.h"
#include "moe_matmul.cuh"
#include "moe_tc.cuh"

namespace moe {
namespace {

constexpr int BN = 128;             // matrix rows of a tile (TMEM lanes)
constexpr int BK = 64;              // values of depth of a stage (128 bytes)
constexpr int EPI_FIRST = 4, EPI_WARPS = 8;
constexpr int THREADS = 32 * (EPI_FIRST + EPI_WARPS);
constexpr int GATHER_THREADS = 64;  // warps 2 and 3
constexpr int MAX_SPLIT = 8;        // blocks that share a tile's depth
constexpr int MAX_STAGES = 10;

template <int BT>
struct Shape {
    static constexpr int STAGES = BT == 256 ? 4 : BT == 128 ? 6 : 10;
    static constexpr int W_BYTES = BN * 2 * BK, X_BYTES = BT * 2 * BK, STAGE = W_BYTES + X_BYTES;
    static constexpr int SMEM = STAGES * STAGE + 1024;   // + alignment of the swizzle pattern
    static constexpr int NBUF = BT == 256 ? 2 : 4;       // TMEM buffers
    static constexpr int COLS = NBUF * BT;
    static constexpr int BOX = BT < 64 ? BT : 64;        // places of a copy
    static_assert(STAGES <= MAX_STAGES && COLS <= 512 && 4 * BT * BN <= STAGES * STAGE, "");
};

struct Ctl {
    uint64_t full[MAX_STAGES], done[MAX_STAGES];   // a stage is loaded; its products are done
    uint64_t sums[4], read[4], drain;              // a tile's sums are there; they are read
    uint32_t tmem;
    int abort;
    int goff[MOE_MAX_EXPERTS + 1];     // first place of each group, clamped
    int tstart[MOE_MAX_EXPERTS + 1];   // first tile of places of each group
};

__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t add, uint32_t me) {
    asm volatile(
        "{\n .reg .pred e, p;\n setp.ne.u32 e, %5, 0;\n setp.ne.u32 p, %4, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"(add),
        "r"(me)
        : "memory");
}
__device__ __forceinline__ void tma_3d(void *dst, const CUtensorMap *m, int x, int y, int z, uint64_t *bar, uint32_t me) {
    asm volatile(
        "{\n .reg .pred e;\n setp.ne.u32 e, %6, 0;\n"
        " @e cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];\n}" ::"r"(sa(dst)), "l"(m), "r"(x), "r"(y), "r"(z), "r"(sa(bar)), "r"(me)
        : "memory");
}
__device__ __forceinline__ void tma_5d(void *dst, const CUtensorMap *m, int x, int y, int z, int u, int v, uint64_t *bar,
                                       uint32_t me) {
    asm volatile(
        "{\n .reg .pred e;\n setp.ne.u32 e, %8, 0;\n"
        " @e cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];\n}" ::"r"(sa(dst)), "l"(m), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(sa(bar)), "r"(me)
        : "memory");
}
// shared-memory descriptor of a tile whose depth lies across its rows (128 bytes = 64 columns a row, 128-byte swizzle):
// 8 rows of depth 1024 bytes apart, the next 64 columns 8192 bytes on
__device__ __forceinline__ uint64_t across_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(8192 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

struct Tile {
    int g, first, rows, n0;   // group, first place, places (1..BT), first column of y
};
// tiles of a group: its tiles of places fastest, so that blocks at work at the same time share a matrix tile in L2
template <int BT>
__device__ __forceinline__ Tile tile_at(const Ctl *c, const MatmulArgs &a, int t) {
    const int q = t / a.ntn;
    int lo = 0, hi = a.G;     // tstart[lo] <= q < tstart[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (c->tstart[mid] <= q) lo = mid;
        else hi = mid;
    }
    const int mt = c->tstart[lo + 1] - c->tstart[lo], local = t - c->tstart[lo] * a.ntn;
    Tile r;
    r.g = lo;
    r.n0 = local / mt * (a.act == MOE_ACT_SWIGLU ? BN / 2 : BN);
    r.first = c->goff[lo] + local % mt * BT;
    r.rows = min(BT, c->goff[lo + 1] - r.first);
    return r;
}

// what an epilogue lane needs of its column
struct Column {
    int n;
    bool in;
    float bias;
};
__device__ __forceinline__ Column column_of(const MatmulArgs &a, const Tile &tl, int quad, int lane) {
    Column c;
    const bool gated = a.act == MOE_ACT_SWIGLU;
    c.n = tl.n0 + (gated ? 16 * quad + (lane & 15) : 32 * quad + lane);
    c.in = c.n < a.N;
    const size_t at = gated ? (size_t)tl.g * 2 * a.N + (lane >> 4) * a.N + c.n : (size_t)tl.g * a.N + c.n;
    c.bias = a.bias && c.in ? a.bias[at] : 0.f;
    return c;
}
// places first .. first + cnt - 1 whose row index is bad: their products are 0
template <int C>
__device__ __forceinline__ void clear_bad(const MatmulArgs &a, float (&v)[C], int first, int cnt, int lane) {
    const int row = lane < cnt ? a.rows[first + lane] : 0;
    const unsigned bad = __ballot_sync(0xFFFFFFFFu, (unsigned)row >= (unsigned)a.X);
    if (bad) {
        if (lane == 0) atomicOr(a.status, MOE_DEV_BAD_ROW);
#pragma unroll
        for (int j = 0; j < C; ++j)
            if (bad >> j & 1) v[j] = 0.f;
    }
}

template <int BT, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
    matmul_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw, const MatmulArgs a) {
    using S = Shape<BT>;
    constexpr int STAGES = S::STAGES, NBUF = S::NBUF;
    extern __shared__ uint8_t raw[];
    __shared__ Ctl c;
    uint8_t *stages = raw + ((1024 - (sa(raw) & 1023)) & 1023);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            bar_init(&c.full[i], a.rows ? 1 + GATHER_THREADS : 1);   // TMA's copies, and the gathered rows
            bar_init(&c.done[i], 1);
        }
        for (int i = 0; i < NBUF; ++i) {
            bar_init(&c.sums[i], 1);
            bar_init(&c.read[i], EPI_WARPS);
        }
        bar_init(&c.drain, 1);
        c.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(&c.tmem)),
                     "n"(S::COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (!a.offsets) {
        if (threadIdx.x == 0) {
            c.goff[0] = c.tstart[0] = 0;
            c.goff[1] = a.M;
            c.tstart[1] = (a.M + BT - 1) / BT;
        }
    } else {
        for (int g = threadIdx.x; g <= a.G; g += THREADS) {
            const int o = a.offsets[g], before = g ? a.offsets[g - 1] : 0;
            if (blockIdx.x == 0 && (o < before || o > a.M)) atomicOr(a.status, MOE_DEV_BAD_ROW);
            c.goff[g] = min(max(o, 0), a.M);
        }
        __syncthreads();
        if (warp == EPI_FIRST) {
            // a group ends where the next one begins, never before its own start
            int sum = 0;
            for (int g0 = 0; g0 < a.G; g0 += 32) {
                const int g = g0 + lane;
                const int mt = g < a.G ? (max(c.goff[g + 1] - c.goff[g], 0) + BT - 1) / BT : 0;
                int s = mt;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int o = __shfl_up_sync(0xFFFFFFFFu, s, off);
                    if (lane >= off) s += o;
                }
                if (g < a.G) c.tstart[g] = sum + s - mt;
                sum += __shfl_sync(0xFFFFFFFFu, s, 31);
            }
            if (lane == 0) c.tstart[a.G] = sum;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = c.tmem;
    // Rising offsets have fewer than 2^30 tiles (the launch checks it).  Falling ones let groups overlap and can have
    // many more: no more than 2^30 of them, so that tile numbers stay in 32 bits.
    const int total = (int)min((long long)c.tstart[a.G] * a.ntn, 0x3FFFFFFFll);
    const int rank = SPLIT ? (int)cluster_rank() : 0, parts = SPLIT ? (int)cluster_size() : 1;
    const int t0 = SPLIT ? (int)blockIdx.x / parts : (int)blockIdx.x, dt = SPLIT ? total : (int)gridDim.x;
    const int kb0 = SPLIT ? rank * a.KB / parts : 0, kb1 = SPLIT ? (rank + 1) * a.KB / parts : a.KB;

    if (warp < EPI_FIRST) {
        if (warp == 0) {
            const uint32_t me = elect();
            const bool gated = a.act == MOE_ACT_SWIGLU;
            Ring<STAGES> r;
            int it = 0;
            bool ok = true;
            for (int t = t0; t < total && ok; t += dt) {
                const Tile tl = tile_at<BT>(&c, a, t);
                const int n0 = __shfl_sync(0xFFFFFFFFu, tl.n0, 0), g = __shfl_sync(0xFFFFFFFFu, tl.g, 0);
                const int first = __shfl_sync(0xFFFFFFFFu, tl.first, 0);
                const int boxes = a.rows ? 0 : (__shfl_sync(0xFFFFFFFFu, tl.rows, 0) + S::BOX - 1) / S::BOX;
                const uint32_t bytes = S::W_BYTES + boxes * S::BOX * 2 * BK;
                for (int kb = kb0; kb < kb1; ++kb, ++it, r.next()) {
                    ok = bar_wait(&c.done[r.i], r.phase ^ 1, &c.abort, a.wait, a.status);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    uint8_t *sw = stages + r.i * S::STAGE, *sx = sw + S::W_BYTES;
                    uint64_t *bar = &c.full[r.i];
                    bar_expect(bar, bytes, me);
                    if (gated) {
                        tma_5d(sw, &mw, kb * BK, 0, 0, n0 / 16, g, bar, me);
                    } else if (a.transposed) {
                        tma_3d(sw, &mw, n0, kb * BK, g, bar, me);
                        tma_3d(sw + S::W_BYTES / 2, &mw, n0 + BN / 2, kb * BK, g, bar, me);
                    } else {
                        tma_3d(sw, &mw, kb * BK, n0, g, bar, me);
                    }
                    for (int i = 0; i < boxes; ++i)
                        tma_tile(sx + i * S::BOX * 2 * BK, &mx, kb * BK, first + i * S::BOX, bar, me);
                }
            }
            // copies in flight land, and their products end, before the block ends
            const uint32_t t_out = clock_hi();
            for (int i = it > STAGES ? it - STAGES : 0; i < it; ++i)
                bar_settle(ok ? &c.done[i % STAGES] : &c.full[i % STAGES], (i / STAGES) & 1, t_out);
            __syncwarp();
        } else if (warp == 1) {
            const uint32_t me = elect();
            // 16 values of depth: 32 bytes of a row, or 16 rows across
            const uint64_t step = a.transposed ? 16 * 128 >> 4 : 32 >> 4;
            const uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a.transposed << 15) | ((uint32_t)(BN >> 4) << 24);
            Ring<STAGES> r;
            Ring<NBUF> d;
            bool ok = true;
            for (int t = t0; t < total && ok; t += dt, d.next()) {
                const int rows = __shfl_sync(0xFFFFFFFFu, tile_at<BT>(&c, a, t).rows, 0);
                const uint32_t idesc = idesc0 | ((uint32_t)((rows + 15) >> 4) << 18);
                ok = bar_wait(&c.read[d.i], d.phase ^ 1, &c.abort, a.wait, a.status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                fence_after();
                for (int kb = kb0; kb < kb1; ++kb, r.next()) {
                    ok = bar_wait(&c.full[r.i], r.phase, &c.abort, a.wait, a.status);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    // gathered rows were written through the generic proxy, and the wait made them visible here; the
                    // products read through the async proxy
                    if (a.rows) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    fence_after();
                    const uint32_t sw = sa(stages) + r.i * S::STAGE;
                    const uint64_t ad = a.transposed ? across_desc(sw) : tile_desc(sw), bd = tile_desc(sw + S::W_BYTES);
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k)
                        mma_bf16(tmem + d.i * BT, ad + k * step, bd + 2 * k, idesc, k | (kb - kb0), me);
                    mma_commit(&c.done[r.i], me);
                }
                if (ok) mma_commit(&c.sums[d.i], me);
            }
            if (!ok) {   // products in flight end before TMEM is freed
                mma_commit(&c.drain, me);
                bar_settle(&c.drain, 0, clock_hi());
            }
            __syncwarp();
        } else if (a.rows) {
            // thread: 16 bytes (piece pc) of rows r0, r0 + 8, ...; the swizzle moves piece p of row r to p ^ (r & 7)
            const int id = threadIdx.x - 64, pc = id & 7, r0 = id >> 3;
            const uint32_t to = sa(stages) + S::W_BYTES + r0 * 2 * BK + ((pc ^ r0) << 4);
            const uint8_t *x = reinterpret_cast<const uint8_t *>(a.x);
            Ring<STAGES> r;
            bool ok = true;
            for (int t = t0; t < total && ok; t += dt) {
                const Tile tl = tile_at<BT>(&c, a, t);
                uint32_t row[BT / 8];   // in units of 16 bytes: X K <= 2^36, K / 8 of them a row
#pragma unroll
                for (int i = 0; i < BT / 8; ++i) {
                    const int at = r0 + 8 * i < tl.rows ? a.rows[tl.first + r0 + 8 * i] : 0;
                    row[i] = (uint32_t)((unsigned)at < (unsigned)a.X ? at : 0);
                }
                const int nr = (tl.rows - r0 + 7) >> 3;   // of this thread
                for (int kb = kb0; kb < kb1; ++kb, r.next()) {
                    ok = bar_wait(&c.done[r.i], r.phase ^ 1, &c.abort, a.wait, a.status);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const bool in = kb * BK + 8 * pc < a.K;
                    const uint8_t *src = x + (in ? 2 * (kb * BK + 8 * pc) : 0);
                    const uint32_t bytes = in ? 16 : 0, dst = to + r.i * S::STAGE;
#pragma unroll
                    for (int i = 0; i < BT / 8; ++i)
                        if (i < nr) copy16(dst + i * 8 * 2 * BK, src + (size_t)row[i] * (2 * (size_t)a.K), bytes);
                    // this thread's arrival, once its copies have landed; nobody waits here for them
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sa(&c.full[r.i])) : "memory");
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else {
        const int quad = warp & 3, half = (warp - EPI_FIRST) >> 2;   // TMEM lanes, and every other 32 places
        const uint32_t at0 = tmem + ((uint32_t)(32 * quad) << 16);
        Ring<NBUF> d;
        bool ok = true;
        for (int t = t0; t < total; t += dt, d.next()) {
            const Tile tl = tile_at<BT>(&c, a, t);
            const Column col = column_of(a, tl, quad, lane);
            ok = bar_wait(&c.sums[d.i], d.phase, &c.abort, a.wait, a.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            fence_after();
#pragma unroll 1
            for (int j = 32 * half; j < tl.rows; j += 64) {
                uint32_t u[32];
                tmem_ld32(at0 + d.i * BT + j, u);
                tmem_ld_wait();
                if (SPLIT) {
                    // this block's part, over the stages (every copy and product is done)
                    float *red = reinterpret_cast<float *>(stages) + j * BN + 32 * quad + lane;
#pragma unroll
                    for (int i = 0; i < 32; ++i) red[i * BN] = __uint_as_float(u[i]);
                } else {
                    // (16 at a time, in one piece of code for both: its 14 forms for 32 take minutes to compile)
#pragma unroll 1
                    for (int h = 0; h < 32 && j + h < tl.rows; h += 16) {
                        float v[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(h ? u[16 + i] : u[i]);
                        const int cnt = min(16, tl.rows - j - h), place = tl.first + j + h;
                        if (a.rows) clear_bad(a, v, place, cnt, lane);
                        if (a.ybf16) emit_t<__nv_bfloat16>(a, v, cnt, place, col.n, col.in, col.bias, lane);
                        else emit_t<float>(a, v, cnt, place, col.n, col.in, col.bias, lane);
                    }
                }
            }
            fence_before();
            bar_arrive(&c.read[d.i], lane == 0);
        }
    }
    if (SPLIT) {
        __syncwarp();
        cluster_sync();
        if (warp >= EPI_FIRST && t0 < total && !*(volatile int *)&c.abort) {
            // each block takes every parts-th 4 places, and adds them over the cluster in rank order
            const int quad = warp & 3, half = (warp - EPI_FIRST) >> 2;
            const Tile tl = tile_at<BT>(&c, a, t0);
            const Column col = column_of(a, tl, quad, lane);
            const uint32_t red = sa(stages) + 4 * (32 * quad + lane);
#pragma unroll 1
            for (int j = 4 * (rank + parts * half); j < tl.rows; j += 8 * parts) {
                float p[MAX_SPLIT][4], v[4];
#pragma unroll
                for (int i = 0; i < MAX_SPLIT; ++i)
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        if (i < parts) p[i][h] = ld_peer1(red + (j + h) * 4 * BN, i);
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    v[h] = p[0][h];
#pragma unroll
                    for (int i = 1; i < MAX_SPLIT; ++i)
                        if (i < parts) v[h] += p[i][h];
                }
                const int cnt = min(4, tl.rows - j);
                if (a.rows) clear_bad(a, v, tl.first + j, cnt, lane);
                if (a.ybf16) emit_t<__nv_bfloat16>(a, v, cnt, tl.first + j, col.n, col.in, col.bias, lane);
                else emit_t<float>(a, v, cnt, tl.first + j, col.n, col.in, col.bias, lane);
            }
        }
        cluster_sync();   // parts are read before their block ends
    }
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::COLS));
    }
}

// ------------------------------------------------------------------ host

bool encode(CUtensorMap *m, int dims, const void *p, const cuuint64_t *size, const cuuint64_t *stride,
            const cuuint32_t *box) {
    const cuuint32_t steps[5] = {1, 1, 1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)dims, const_cast<void *>(p), size, stride, box,
                       steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_w(CUtensorMap *m, const MatmulArgs &a) {
    const cuuint64_t K = (cuuint64_t)a.K, N = (cuuint64_t)a.N, G = (cuuint64_t)a.G;
    if (a.act == MOE_ACT_SWIGLU) {   // depth, 16 rows, gate or up, which 16, group
        const cuuint64_t size[5] = {K, 16, 2, N / 16, G}, stride[4] = {2 * K, 2 * N * K, 32 * K, 4 * N * K};
        const cuuint32_t box[5] = {BK, 16, 2, BN / 32, 1};
        return encode(m, 5, a.w, size, stride, box);
    }
    if (a.transposed) {
        const cuuint64_t size[3] = {N, K, G}, stride[2] = {2 * N, 2 * N * K};
        const cuuint32_t box[3] = {64, BK, 1};
        return encode(m, 3, a.w, size, stride, box);
    }
    const cuuint64_t size[3] = {K, N, G}, stride[2] = {2 * K, 2 * N * K};
    const cuuint32_t box[3] = {BK, BN, 1};
    return encode(m, 3, a.w, size, stride, box);
}

template <int BT, bool SPLIT>
cudaError_t launch_t(const MatmulArgs &a, int grid, int split, cudaStream_t s) {
    CUtensorMap mx, mw;
    const cuuint64_t size[2] = {(cuuint64_t)a.K, (cuuint64_t)a.X}, stride[1] = {2 * (cuuint64_t)a.K};
    const cuuint32_t box[2] = {BK, (cuuint32_t)Shape<BT>::BOX};
    if (!encode_fn()) return cudaErrorSymbolNotFound;
    if (!encode(&mx, 2, a.x, size, stride, box) || !encode_w(&mw, a)) return cudaErrorInvalidValue;
    auto *k = matmul_kernel<BT, SPLIT>;
    cudaError_t err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<BT>::SMEM);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = Shape<BT>::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    if (SPLIT) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)split;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, k, mx, mw, a);
}

}  // namespace

cudaError_t launch_matmul(MatmulArgs a, cudaStream_t s) {
    a.KB = (a.K + BK - 1) / BK;
    a.ntn = a.act == MOE_ACT_SWIGLU ? (a.N + 63) / 64 : (a.N + 127) / 128;
    a.wait = kWaitLimit;
    // most tiles there can be: a group's last one may be short
    const long long sms = num_sms(), groups = a.offsets ? (a.G < a.M ? a.G : a.M) : 1;
    const auto tiles = [&](int bt) { return (a.offsets ? a.M / bt + groups : (a.M + bt - 1) / bt) * a.ntn; };
    if (tiles(32) > 0x3FFFFFFF) return cudaErrorNotSupported;
    const long long rows = a.M / groups;   // of a group on average
    const int bt = rows <= 32 ? 32 : rows > 128 && tiles(256) >= sms ? 256 : 128;
    const long long n = tiles(bt);
    int split = 1;
    while (split < MAX_SPLIT && n * split * 2 <= sms && a.KB >= split * 8) split *= 2;
    const int grid = (int)(split > 1 ? n * split : n < sms ? n : sms);
    if (split > 1) return bt == 32 ? launch_t<32, true>(a, grid, split, s) : launch_t<128, true>(a, grid, split, s);
    if (bt == 32) return launch_t<32, false>(a, grid, 1, s);
    return bt == 128 ? launch_t<128, false>(a, grid, 1, s) : launch_t<256, false>(a, grid, 1, s);
}

}  // namespace moe
