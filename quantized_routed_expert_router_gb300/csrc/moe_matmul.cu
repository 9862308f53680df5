// moe_matmul.cu - products of bf16 rows with bf16 matrices, dense or grouped by
// expert, with bias, activation and residual in the epilogue (moe_matmul).
//
// A tile is 128 columns of a matrix a block by up to BT places of one group.  The
// columns are the rows of the tensor cores' first operand, the places the columns of the
// second: TMEM then gives a lane a column and a register a place, so that
//   - the number of places of a product follows the tile's (16, 32, .. BT);
//   - a lane has its bias in a register, and what a warp reads or writes of a
//     place is 32 columns side by side, wherever rows of y start: nothing is
//     turned in shared memory and no row of another group is touched.
// With the gated activation a block's 128 columns are 64 of y: gate and up rows in
// turns of 16, by one copy whose map has the two as a dimension, so that lanes l
// and l + 16 of a warp hold the gate and the up value of a column.
//
// The warps of a block have roles:
//   warp 0    : TMA copies of matrix tiles, and of rows that lie in order (64
//               values deep, 128-byte swizzle), into a ring of stages
//   warp 1    : one thread issues the products into one of the TMEM buffers
//   warps 2-3 : rows that are gathered, by 16-byte asynchronous copies that
//               signal the stage when they land
//   warps 4-11: the epilogue, while the products of the next tile run
// Blocks are persistent, one an SM.  What bounds the large tiles is their feed: a stage of 32 KB a block
// comes in 560 to 600 cycles where its products take 512 (8192 x 2048 by 7168 x 2048 129 us, 1.86 PFLOP/s, 0.96 of the
// bf16 rate; without the copies of rows it would be 2.04); one block a tile, 48 KB a stage, took 165.  Few places a
// group are bound by the matrices' bytes (64 rows over 32 of 2880 x 2880: 64.5 us on the device, 0.9 of the copy rate).
//   Pairs: two blocks share a tile of 256 columns by 256 places.  Each holds its 128
// columns and half of the places; the first one issues products that read both
// halves (cta_group::2).  The other's warp 1 passes on that its stage is loaded, so that either
// block has barriers of its own for its copies.
//   Split depth: where there are too few tiles for the SMs, a cluster of blocks
// splits the depth of a tile and adds its parts through distributed shared memory
// in rank order.
//
// Sums.  The tensor cores cut off what they add below the 24 bits of a running sum, always towards zero.  Over K values that
// is about K 2^-30 of the results where terms have both signs (1.7e-6 at K = 2048), and more where they have one: 4e-6 at
// 2048, 3.3e-5 at 8192, 1.8e-4 at 32768, 1.9e-3 at 262144.  So running sums are bounded and added up in fp32 (RUNS): for fp32
// results 640 values long at most, which leaves 4e-7 to 8e-7 at any K, the more the larger a few channels of the rows
// are (768 long: 6e-7 to 9e-7); for bf16 results, which are rounded by up to 2^-8, 8192 long, so that most have one.
#include <cuda.h>
#include <cuda_bf16.h>

#include "moe_around.h"
#include "moe_device.h"
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
// registers a thread: at the launch, and where the epilogue takes some of the feeding warps'
constexpr int LAUNCH_REGS = 168, FEED_REGS = 88, EPI_REGS = 208;
// stages of a running sum of fp32 results: of a tile's first two, which the products can fill while the epilogue is busy with
// the tile before, and of the others
constexpr int FIRST_RUNS = 10, RUN = 8;
constexpr int WHOLE = 128;   // of bf16 results

template <int BT, bool PAIR>
struct Shape {
    static constexpr int PLACES = PAIR ? BT / 2 : BT;   // of a block's stage
    static constexpr int STAGES = BT == 32 ? 10 : PAIR && BT == 128 ? 9 : 6;
    static constexpr int W_BYTES = BN * 2 * BK, X_BYTES = PLACES * 2 * BK, STAGE = W_BYTES + X_BYTES;
    static constexpr int SMEM = STAGES * STAGE + 1024;   // + alignment of the swizzle pattern
    static constexpr int NBUF = BT == 256 ? 2 : 4;       // TMEM buffers
    static constexpr int COLS = NBUF * BT;
    static constexpr int BOX = PLACES, LESS = PLACES == 128 ? 64 : PLACES;   // places of a copy, of one for few places
    static constexpr int PIECES = BT < 64 ? 1 : BT / 64;   // 32 places each, of an epilogue warp
    static_assert(STAGES <= MAX_STAGES && COLS <= 512 && 4 * BT * BN <= STAGES * STAGE, "");
};

struct Ctl {
    uint64_t full[MAX_STAGES], done[MAX_STAGES];   // a stage is loaded; its products are done
    uint64_t other[MAX_STAGES];                    // the pair's other block has loaded its part of a stage
    uint64_t sums[4], read[4], drain;              // a tile's sums are there; they are read
    uint32_t tmem;
    int abort;
    int goff[MOE_MAX_EXPERTS + 1];     // first place of each group, clamped
    int tstart[MOE_MAX_EXPERTS + 1];   // first tile of places of each group
};

template <bool PAIR>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t add, uint32_t me) {
    if constexpr (PAIR)
        asm volatile(
            "{\n .reg .pred e, p;\n setp.ne.u32 e, %5, 0;\n setp.ne.u32 p, %4, 0;\n"
            " @e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(ad), "l"(bd), "r"(idesc),
            "r"(add), "r"(me)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred e, p;\n setp.ne.u32 e, %5, 0;\n setp.ne.u32 p, %4, 0;\n"
            " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(ad), "l"(bd), "r"(idesc),
            "r"(add), "r"(me)
            : "memory");
}
// the barrier is told when the products so far are done; of a pair, whose first block is `lead` of the cluster, that of either
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t *bar, int lead, uint32_t me) {
    if constexpr (PAIR)
        asm volatile(
            "{\n .reg .pred e;\n setp.ne.u32 e, %1, 0;\n"
            " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n}" ::"r"(
                sa(bar)), "r"(me), "h"((uint16_t)(3 << lead))
            : "memory");
    else
        mma_commit(bar, me);
}
__device__ __forceinline__ void tma_3d(void *dst, const CUtensorMap *m, int x, int y, int z, uint64_t *bar, uint32_t me) {
    asm volatile(
        "{\n .reg .pred e;\n setp.ne.u32 e, %6, 0;\n"
        " @e cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];\n}" ::"r"(sa(dst)), "l"(m), "r"(x), "r"(y), "r"(z), "r"(sa(bar)), "r"(me)
        : "memory");
}
__device__ __forceinline__ void tma_4d(void *dst, const CUtensorMap *m, int x, int y, int z, int u, uint64_t *bar,
                                       uint32_t me) {
    asm volatile(
        "{\n .reg .pred e;\n setp.ne.u32 e, %7, 0;\n"
        " @e cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];\n}" ::"r"(sa(dst)), "l"(m), "r"(x), "r"(y), "r"(z), "r"(u), "r"(sa(bar)), "r"(me)
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
    int g, first, rows, n0;   // group, first place, places (1..BT), this block's first column of y
};
// Tiles of a group: its tiles of places fastest, so that blocks at work at the same time share a matrix tile in L2.  Whole
// column tiles of all groups come first, then those that are cut off by the matrix's end: they take less time, and fill up
// the last round (3108 rows over 32 of 2880 x 2880: 384 tiles of pairs, 352 of them whole, on 76 pairs).
template <int BT, bool PAIR>
__device__ __forceinline__ Tile tile_at(const Ctl *c, const MatmulArgs &a, int t, int rank) {
    const int whole = (int)((unsigned)c->tstart[a.G] * (unsigned)a.whole);   // (taken where it is at most t)
    const bool cut = a.whole != a.ntn && (long long)c->tstart[a.G] * a.whole <= t;
    const int q = cut ? t - whole : t / a.whole;
    int lo = 0, hi = a.G;     // tstart[lo] <= q < tstart[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (c->tstart[mid] <= q) lo = mid;
        else hi = mid;
    }
    const int mt = c->tstart[lo + 1] - c->tstart[lo], local = cut ? q - c->tstart[lo] : t - c->tstart[lo] * a.whole;
    const int ct = cut ? a.whole : local / mt;
    Tile r;
    r.g = lo;
    r.n0 = (PAIR ? 2 * ct + rank : ct) * (a.act == MOE_ACT_SWIGLU ? BN / 2 : BN);
    r.first = c->goff[lo] + (cut ? local : local % mt) * BT;
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
// what an fp32 epilogue reads (the residual, or z) for places lo .. hi - 1 of a tile into L2; thread `id` of the epilogue's
template <typename TY>
__device__ __forceinline__ void prefetch_rows(const MatmulArgs &a, const TY *p, const Tile &tl, int lo, int hi, int id) {
    constexpr int LINE = 128 / (int)sizeof(TY), LINES = BN / LINE;   // of a place
    const bool both = a.act == MOE_ACT_SWIGLU_GRAD;
    const int have = min(a.act == MOE_ACT_SWIGLU ? BN / 2 : BN, a.N - tl.n0), i = id % LINES * LINE;
    if (i >= have) return;
    const size_t pitch = both ? 2 * (size_t)a.N : (size_t)a.N;
    for (int j = lo + id / LINES; j < hi; j += 32 * EPI_WARPS / LINES)
        for (int h = 0; h <= (both ? 1 : 0); ++h) {
            const TY *at = p + (size_t)(tl.first + j) * pitch + (size_t)h * a.N + tl.n0;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at + i));
            if (i == 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + have - 1));   // (a row can start inside a line)
        }
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

// places of a tile that one of a pair's blocks loads (a product takes them in 32s)
__device__ __forceinline__ int half_of(int rows) { return ((rows + 31) >> 5) << 4; }

template <int BT, bool PAIR, bool SPLIT, bool RUNS, typename TY>
__global__ void __launch_bounds__(THREADS, 1)
    matmul_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mx_less,
                  const __grid_constant__ CUtensorMap mw, const MatmulArgs a) {
    using S = Shape<BT, PAIR>;
    constexpr int STAGES = S::STAGES, NBUF = S::NBUF;
    extern __shared__ uint8_t raw[];
    __shared__ Ctl c;
    uint8_t *stages = raw + ((1024 - (sa(raw) & 1023)) & 1023);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // of the cluster: this block, the first one of its pair; of the pair: this block; of the depth: this block's part
    const int in_cluster = PAIR || SPLIT ? (int)cluster_rank() : 0, lead = in_cluster & ~1;
    const int rank = PAIR ? in_cluster & 1 : 0, part = SPLIT ? in_cluster / (PAIR ? 2 : 1) : 0;
    const int size = PAIR || SPLIT ? (int)cluster_size() : 1, parts = SPLIT ? size / (PAIR ? 2 : 1) : 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            bar_init(&c.full[i], (a.rows ? 1 + GATHER_THREADS : 1) + a.hold_copies);   // TMA's copies, the gathered rows
            bar_init(&c.done[i], 1 + a.hold_products);
            bar_init(&c.other[i], 1);
        }
        for (int i = 0; i < NBUF; ++i) {
            bar_init(&c.sums[i], 1 + a.hold_products);
            bar_init(&c.read[i], PAIR ? 2 * EPI_WARPS : EPI_WARPS);
        }
        bar_init(&c.drain, 1);
        c.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(&c.tmem)),
                         "n"(S::COLS) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(&c.tmem)),
                         "n"(S::COLS) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
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
    if (PAIR) cluster_sync();   // the other block's barriers are there
    fence_after();
    const uint32_t tmem = c.tmem;
    // Rising offsets have fewer than 2^30 tiles (the launch checks it).  Falling ones let groups overlap and can have
    // many more: no more than 2^30 of them, so that tile numbers stay in 32 bits.
    const int total = (int)min((long long)c.tstart[a.G] * a.ntn, 0x3FFFFFFFll);
    const int t0 = (int)blockIdx.x / size, dt = SPLIT ? total : (int)gridDim.x / size;
    const int kb0 = SPLIT ? part * a.KB / parts : 0, kb1 = SPLIT ? (part + 1) * a.KB / parts : a.KB;
    const auto run_end = [&](int kb) {   // of the running sum that starts with stage kb
        return !RUNS ? kb1 : min(kb + (sizeof(TY) == 2 ? WHOLE : kb < kb0 + 2 * FIRST_RUNS ? FIRST_RUNS : RUN), kb1);
    };

    // Registers: the running sums take 128, beside 32 on their way.
    constexpr bool MOVE = RUNS && PAIR && !SPLIT;
    static_assert(FEED_REGS * 32 * EPI_FIRST + EPI_REGS * 32 * EPI_WARPS <= LAUNCH_REGS * THREADS, "");
    if (warp < EPI_FIRST) {
        if (MOVE) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FEED_REGS));
        if (warp == 0) {
            const uint32_t me = elect();
            Ring<STAGES> r;
            int it = 0;
            bool ok = true;
            for (int t = t0; t < total && ok; t += dt) {
                const Tile tl = tile_at<BT, PAIR>(&c, a, t, rank);
                const int n0 = __shfl_sync(0xFFFFFFFFu, tl.n0, 0), g = __shfl_sync(0xFFFFFFFFu, tl.g, 0);
                const int rows = __shfl_sync(0xFFFFFFFFu, tl.rows, 0), h = PAIR ? half_of(rows) : 0;
                const int first = __shfl_sync(0xFFFFFFFFu, tl.first, 0) + rank * h;
                const int mine = PAIR ? (rank ? max(rows - h, 0) : min(rows, h)) : rows;
                // (one copy each of matrix and rows: with two of 64 rows a stage 8192 x 2048 by 7168 x 2048 took 4% more)
                const CUtensorMap *rows_map = mine > S::LESS ? &mx : &mx_less;
                const int box = a.rows || mine <= 0 ? 0 : mine > S::LESS ? S::BOX : S::LESS;
                const uint32_t bytes = S::W_BYTES + box * 2 * BK;
                for (int kb = kb0; kb < kb1; ++kb, ++it, r.next()) {
                    ok = bar_wait<PAIR>(&c.done[r.i], r.phase ^ 1, &c.abort, a.wait, a.status);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    uint8_t *sw = stages + r.i * S::STAGE, *sx = sw + S::W_BYTES;
                    uint64_t *bar = &c.full[r.i];
                    bar_expect(bar, bytes, me);
                    // (by the dimensions that the map has)
                    if (a.wdims == 5) {
                        tma_5d(sw, &mw, kb * BK, 0, 0, n0 / 16, g, bar, me);
                    } else if (a.wdims == 4) {
                        tma_4d(sw, &mw, 0, kb * BK, n0 / 64, g, bar, me);
                    } else if (a.transposed) {
                        tma_3d(sw, &mw, n0, kb * BK, g, bar, me);
                        tma_3d(sw + S::W_BYTES / 2, &mw, n0 + BN / 2, kb * BK, g, bar, me);
                    } else {
                        tma_3d(sw, &mw, kb * BK, n0, g, bar, me);
                    }
                    if (box) tma_tile(sx, rows_map, kb * BK, first, bar, me);
                }
            }
            // copies in flight land, and their products end, before the block ends
            const uint32_t t_out = clock_hi();
            for (int i = it > STAGES ? it - STAGES : 0; i < it; ++i)
                bar_settle(ok ? &c.done[i % STAGES] : &c.full[i % STAGES], (i / STAGES) & 1, t_out);
            __syncwarp();
        } else if (warp == 1 && rank && PAIR) {
            // this block's part of a stage is loaded: the first block may take it
            const uint32_t me = elect();
            Ring<STAGES> r;
            bool ok = true;
            for (int t = t0; t < total && ok; t += dt)
                for (int kb = kb0; kb < kb1; ++kb, r.next()) {
                    ok = bar_wait(&c.full[r.i], r.phase, &c.abort, a.wait, a.status);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    if (a.rows) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    bar_arrive_at(&c.other[r.i], lead, me);
                }
            __syncwarp();
        } else if (warp == 1) {
            const uint32_t me = elect();
            // 16 values of depth: 32 bytes of a row, or 16 rows across
            const uint64_t step = a.transposed ? 16 * 128 >> 4 : 32 >> 4;
            const uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a.transposed << 15) |
                                    ((uint32_t)((PAIR ? 2 * BN : BN) >> 4) << 24);
            Ring<STAGES> r;
            Ring<NBUF> d;
            bool ok = true;
            for (int t = t0; t < total && ok; t += dt) {
                const int rows = __shfl_sync(0xFFFFFFFFu, (tile_at<BT, PAIR>(&c, a, t, rank).rows), 0);
                const uint32_t idesc = idesc0 | ((uint32_t)(PAIR ? half_of(rows) >> 3 : (rows + 15) >> 4) << 18);
                for (int kb = kb0; kb < kb1 && ok;) {
                    const int first = kb, end = run_end(kb);
                    ok = bar_wait<PAIR>(&c.read[d.i], d.phase ^ 1, &c.abort, a.wait, a.status);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    fence_after();
                    for (; kb < end; ++kb, r.next()) {
                        ok = bar_wait(&c.full[r.i], r.phase, &c.abort, a.wait, a.status) &&
                             (!PAIR || bar_wait<PAIR>(&c.other[r.i], r.phase, &c.abort, a.wait, a.status));
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok) break;
                        // gathered rows were written through the generic proxy, and the wait made them visible here; the
                        // products read through the async proxy (the other block's rows have passed a fence there; one for
                        // the cluster's shared memory here: 8191 x 4 rows over 32 experts 1588 us instead of 725)
                        if (a.rows) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        fence_after();
                        const uint32_t sw = sa(stages) + r.i * S::STAGE;
                        const uint64_t ad = a.transposed ? across_desc(sw) : tile_desc(sw), bd = tile_desc(sw + S::W_BYTES);
#pragma unroll
                        for (int k = 0; k < BK / 16; ++k)
                            mma_bf16<PAIR>(tmem + d.i * BT, ad + k * step, bd + 2 * k, idesc, k | (kb - first), me);
                        commit<PAIR>(&c.done[r.i], lead, me);
                    }
                    if (ok) {
                        commit<PAIR>(&c.sums[d.i], lead, me);
                        d.next();
                    }
                }
            }
            if (!ok) {   // products in flight end before TMEM is freed
                commit<PAIR>(&c.drain, lead, me);
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
                const Tile tl = tile_at<BT, PAIR>(&c, a, t, rank);
                const int h = PAIR ? half_of(tl.rows) : 0, first = tl.first + rank * h;
                const int mine = PAIR ? (rank ? max(tl.rows - h, 0) : min(tl.rows, h)) : tl.rows;
                uint32_t row[S::PLACES / 8];   // in units of 16 bytes (X K <= 2^35 values)
#pragma unroll
                for (int i = 0; i < S::PLACES / 8; ++i) {
                    const int at = r0 + 8 * i < mine ? a.rows[first + r0 + 8 * i] : 0;
                    row[i] = (uint32_t)((unsigned)at < (unsigned)a.X ? at : 0) * (uint32_t)(a.K >> 3);
                }
                const int nr = (mine - r0 + 7) >> 3;   // of this thread
                for (int kb = kb0; kb < kb1; ++kb, r.next()) {
                    ok = bar_wait<PAIR>(&c.done[r.i], r.phase ^ 1, &c.abort, a.wait, a.status);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const bool in = kb * BK + 8 * pc < a.K;
                    const uint8_t *src = x + (in ? 2 * (kb * BK + 8 * pc) : 0);
                    const uint32_t bytes = in ? 16 : 0, dst = to + r.i * S::STAGE;
                    if (nr == S::PLACES / 8) {
#pragma unroll
                        for (int i = 0; i < S::PLACES / 8; ++i) copy16(dst + i * 8 * 2 * BK, src + 16 * (uint64_t)row[i], bytes);
                    } else {
#pragma unroll
                        for (int i = 0; i < S::PLACES / 8; ++i)
                            if (i < nr) copy16(dst + i * 8 * 2 * BK, src + 16 * (uint64_t)row[i], bytes);
                    }
                    // this thread's arrival, once its copies have landed; nobody waits here for them
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sa(&c.full[r.i])) : "memory");
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else {
        if (MOVE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
        const int quad = warp & 3, half = (warp - EPI_FIRST) >> 2;   // TMEM lanes, and every other 32 places
        const uint32_t at0 = tmem + ((uint32_t)(32 * quad) << 16);
        Ring<NBUF> d;
        bool ok = true;
        // the sums of a buffer are read
        const auto give_back = [&] {
            fence_before();
            __syncwarp();
            if (PAIR) bar_arrive_at(&c.read[d.i], lead, lane == 0);
            else bar_arrive(&c.read[d.i], lane == 0);
            d.next();
        };
        for (int t = t0; t < total; t += dt) {
            const Tile tl = tile_at<BT, PAIR>(&c, a, t, rank);
            const Column col = column_of(a, tl, quad, lane);
            // 16 places of this warp to the others of the cluster (over the stages: every copy and product is done), or out
            const auto pass_on = [&](float(&v)[16], const float(&x)[16], int j) {
                if (SPLIT) {
                    float *red = reinterpret_cast<float *>(stages) + j * BN + 32 * quad + lane;
#pragma unroll
                    for (int i = 0; i < 16; ++i) red[i * BN] = v[i];
                } else {
                    const int cnt = min(16, tl.rows - j), place = tl.first + j;
                    if (a.rows) clear_bad(a, v, place, cnt, lane);
                    emit_t<MOVE, TY>(a, v, x, cnt, place, col.n, col.in, col.bias, lane);
                }
            };
            if constexpr (RUNS) {
                // The running sums are added in registers and go out from there, so that the buffers are free for the next
                // tile's (held in TMEM meanwhile, they kept the products waiting: 206 us with a residual, 2048 deep).
                float acc[S::PIECES][32] = {};
                const auto place_of = [&](int q) { return 32 * half + 64 * (q >> 1) + 16 * (q & 1); };
                // Pairs: the residual of the next 16 places is on its way while 16 go out (and of the first ones while the
                // products run): waited for 16 by 16 it took 8000 of a tile's 27000 cycles, 2048 deep.
                float x[16];
                const auto extra = [&](int j) {
                    if (!MOVE || a.act == MOE_ACT_SWIGLU || a.act == MOE_ACT_SWIGLU_GRAD || !col.in) return;
                    if (j + 16 <= tl.rows) fetch_extra<true, TY>(a, tl.first + j, 16, col.n, x);
                    else fetch_extra<false, TY>(a, tl.first + j, tl.rows - j, col.n, x);
                };
                extra(place_of(0));
                // All that the tile's 16s read comes into L2 while its products run, in shares: 8192 x 2048 by 7168 x 2048
                // with a residual takes 202 us so, 214 with all of it asked for at once, 227 with none.  (bf16 results have
                // half the bytes and no shares to wait for: 144 us either way, z's SwiGLU slopes 112 without and 114 with.)
                const TY *extras = SPLIT ? nullptr : static_cast<const TY *>(a.act >= MOE_ACT_SILU_GRAD ? a.z : a.residual);
                int asked = 0;
                for (int kb = kb0; kb < kb1; kb = run_end(kb)) {
                    if (extras) {
                        const int upto = (int)((long long)tl.rows * (run_end(kb) - kb0) / (kb1 - kb0));
                        prefetch_rows(a, extras, tl, asked, upto, (int)threadIdx.x - 32 * EPI_FIRST);
                        asked = upto;
                    }
                    ok = bar_wait<PAIR>(&c.sums[d.i], d.phase, &c.abort, a.wait, a.status);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    fence_after();
#pragma unroll
                    for (int p = 0; p < S::PIECES; ++p) {
                        const int j = 32 * half + 64 * p;
                        if (j >= tl.rows) continue;
                        uint32_t u[32];
                        tmem_ld32(at0 + d.i * BT + j, u);
#pragma unroll
                        for (int i = 0; i < 32; ++i) acc[p][i] += __uint_as_float(u[i]);
                    }
                    give_back();
                }
                if (!ok) break;
                // (one piece of code for all 16s: unrolled, its forms take minutes to compile)
#pragma unroll 1
                for (int q = 0; q < 2 * S::PIECES; ++q) {
                    const int j = place_of(q);
                    if (j >= tl.rows) break;
                    float v[16], now[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        v[i] = acc[0][i];
                        now[i] = x[i];
                    }
#pragma unroll
                    for (int k = 1; k < 2 * S::PIECES; ++k)
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = q == k ? acc[k >> 1][16 * (k & 1) + i] : v[i];
                    extra(place_of(q + 1));
                    pass_on(v, now, j);
                }
            } else {
                ok = bar_wait<PAIR>(&c.sums[d.i], d.phase, &c.abort, a.wait, a.status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                fence_after();
#pragma unroll 1
                for (int j = 32 * half; j < tl.rows; j += 64) {
                    uint32_t u[32];
                    tmem_ld32(at0 + d.i * BT + j, u);
#pragma unroll 1
                    for (int h = 0; h < 32 && j + h < tl.rows; h += 16) {
                        float v[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(h ? u[16 + i] : u[i]);
                        pass_on(v, v, j + h);
                    }
                }
                give_back();
            }
        }
    }
    if (SPLIT) {
        __syncwarp();
        cluster_sync();
        if (warp >= EPI_FIRST && t0 < total && !*(volatile int *)&c.abort) {
            // Each block takes every parts-th C places, and adds them over the cluster's parts of its columns in order.  A load
            // takes a microsecond, so a warp has many on their way; and it takes 32 columns side by side (four places of a column
            // at a time, a row apart, were slower: 128 x 4096 by 1000 x 4096 14.5 us instead of 10.6).
            constexpr int C = PAIR ? 16 : BT == 32 ? 4 : 8, PARTS = PAIR ? MAX_SPLIT / 2 : MAX_SPLIT;
            const int quad = warp & 3, half = (warp - EPI_FIRST) >> 2;
            const Tile tl = tile_at<BT, PAIR>(&c, a, t0, rank);
            const Column col = column_of(a, tl, quad, lane);
            const uint32_t red = sa(stages) + 4 * (32 * quad + lane);
#pragma unroll 1
            for (int j = C * (part + parts * half); j < tl.rows; j += 2 * C * parts) {
                float p[PARTS][C], v[C];
#pragma unroll
                for (int i = 0; i < PARTS; ++i)
                    if (i < parts) {
#pragma unroll
                        for (int h = 0; h < C; ++h) p[i][h] = ld_peer1(red + (j + h) * 4 * BN, PAIR ? 2 * i + rank : i);
                    }
#pragma unroll
                for (int h = 0; h < C; ++h) {
                    v[h] = p[0][h];
#pragma unroll
                    for (int i = 1; i < PARTS; ++i)
                        if (i < parts) v[h] += p[i][h];
                }
                const int cnt = min(C, tl.rows - j);
                if (a.rows) clear_bad(a, v, tl.first + j, cnt, lane);
                emit_t<false, TY>(a, v, v, cnt, tl.first + j, col.n, col.in, col.bias, lane);
            }
        }
        cluster_sync();   // parts are read before their block ends
    }
    fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();   // the first block's products are done, and the other's arrivals there
    if (warp == 1) {
        fence_after();
        if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::COLS));
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::COLS));
    }
}

// ------------------------------------------------------------------ host

int current_device() {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}

bool encode(CUtensorMap *m, int dims, const void *p, const cuuint64_t *size, const cuuint64_t *stride,
            const cuuint32_t *box) {
    const cuuint32_t steps[5] = {1, 1, 1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)dims, const_cast<void *>(p), size, stride, box,
                       steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_w(CUtensorMap *m, const MatmulArgs &a) {
    const cuuint64_t K = (cuuint64_t)a.K, N = (cuuint64_t)a.N, G = (cuuint64_t)a.G;
    if (a.wdims == 5) {   // depth, 16 rows, gate or up, which 16, group
        const cuuint64_t size[5] = {K, 16, 2, N / 16, G}, stride[4] = {2 * K, 2 * N * K, 32 * K, 4 * N * K};
        const cuuint32_t box[5] = {BK, 16, 2, BN / 32, 1};
        return encode(m, 5, a.w, size, stride, box);
    }
    if (a.wdims == 4) {   // 64 columns, depth, which 64, group
        const cuuint64_t size[4] = {64, K, N / 64, G}, stride[3] = {2 * N, 128, 2 * N * K};
        const cuuint32_t box[4] = {64, BK, BN / 64, 1};
        return encode(m, 4, a.w, size, stride, box);
    }
    if (a.transposed) {   // columns, depth, group
        const cuuint64_t size[3] = {N, K, G}, stride[2] = {2 * N, 2 * N * K};
        const cuuint32_t box[3] = {64, BK, 1};
        return encode(m, 3, a.w, size, stride, box);
    }
    const cuuint64_t size[3] = {K, N, G}, stride[2] = {2 * K, 2 * N * K};   // depth, rows, group
    const cuuint32_t box[3] = {BK, BN, 1};
    return encode(m, 3, a.w, size, stride, box);
}

template <int BT, bool PAIR, bool SPLIT, bool RUNS, typename TY>
cudaError_t launch_t(const MatmulArgs &a, int grid, int cluster, cudaStream_t s) {
    using S = Shape<BT, PAIR>;
    CUtensorMap mx, mx_less, mw;
    const cuuint64_t size[2] = {(cuuint64_t)a.K, (cuuint64_t)a.X}, stride[1] = {2 * (cuuint64_t)a.K};
    const cuuint32_t box[2] = {BK, (cuuint32_t)S::BOX}, less[2] = {BK, (cuuint32_t)S::LESS};
    if (!encode_fn()) return cudaErrorSymbolNotFound;
    if (!encode(&mx, 2, a.x, size, stride, box) || !encode(&mx_less, 2, a.x, size, stride, less) || !encode_w(&mw, a))
        return cudaErrorInvalidValue;
    auto *k = matmul_kernel<BT, PAIR, SPLIT, RUNS, TY>;
    cudaError_t err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (err != cudaSuccess) return err;
    if (PAIR && !SPLIT && RUNS) {   // the registers that its warps hand on have to be there
        static PerDevice registers;
        const int have = registers.get(current_device(), [k] {
            cudaFuncAttributes at;
            return cudaFuncGetAttributes(&at, k) == cudaSuccess ? at.numRegs : -1;
        });
        if (have < LAUNCH_REGS) return cudaErrorInvalidConfiguration;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    if (PAIR || SPLIT) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)cluster;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, k, mx, mx_less, mw, a);
}

// clusters of SIZE blocks that fit the GPU at once (its SMs come in groups, and a cluster lies within one); negative: not known
template <int BT, bool PAIR, typename TY, int SIZE>
int clusters_at_once() {
    static PerDevice clusters;
    return clusters.get(current_device(), [] {
        auto *k = matmul_kernel<BT, PAIR, true, sizeof(TY) == 4, TY>;   // (RUNS asks for the same threads and memory)
        constexpr int smem = Shape<BT, PAIR>::SMEM;
        int n = 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(SIZE);
        cfg.blockDim = dim3(THREADS);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = SIZE;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess) {
            cudaGetLastError();   // this call goes on without
            return -1;
        }
        return n;
    });
}
// how many parts of the depth n tiles can have: every part with 4 blocks of depth and an SM (a pair: two) of its own, and all
// clusters at once (16 of 8 blocks did not fit: 64 x 7168 by 2048 x 7168 18.8 us in 8 parts, 14.5 in 4; 64 x 8192 by
// 512 x 8192 11.5 in 8, 14.6 in 4, 22.7 in 2; 64 x 4096 by 1000 x 4096 10.4, 12.5 and 14.7)
template <int BT, bool PAIR, typename TY>
int parts_of(long long n, int KB) {
    const auto room = [&](int parts, int clusters) {
        return KB >= 4 * parts && n * parts * (PAIR ? 2 : 1) <= num_sms() && n <= clusters;
    };
    if (!room(2, clusters_at_once<BT, PAIR, TY, PAIR ? 4 : 2>())) return 1;
    if (!room(4, clusters_at_once<BT, PAIR, TY, PAIR ? 8 : 4>())) return 2;
    if (PAIR || !room(MAX_SPLIT, clusters_at_once<BT, PAIR, TY, 8>())) return 4;
    return MAX_SPLIT;
}
template <int BT, bool PAIR, bool RUNS, typename TY>
cudaError_t launch_tiles_t(const MatmulArgs &a, long long n, int parts, cudaStream_t s) {
    constexpr int PER = PAIR ? 2 : 1;
    if constexpr (!PAIR || BT == 256) {   // (of pairs with fewer places there are many)
        if (parts > 1) return launch_t<BT, PAIR, true, RUNS, TY>(a, (int)n * parts * PER, parts * PER, s);
    }
    const long long most = num_sms() / PER;
    return launch_t<BT, PAIR, false, RUNS, TY>(a, (int)(n < most ? n : most) * PER, PER, s);
}
template <int BT, bool PAIR, typename TY>
cudaError_t launch_tiles(MatmulArgs a, int wide, long long n, int parts, cudaStream_t s) {
    constexpr int PER = PAIR ? 2 : 1;
    a.ntn = (wide + PER * BN - 1) / (PER * BN);
    a.whole = wide / (PER * BN);
    if constexpr (sizeof(TY) == 2) {
        if ((a.KB + parts - 1) / parts <= WHOLE) return launch_tiles_t<BT, PAIR, false, TY>(a, n, parts, s);
    }
    return launch_tiles_t<BT, PAIR, true, TY>(a, n, parts, s);
}

template <typename TY>
cudaError_t launch_matmul_t(const MatmulArgs &a, cudaStream_t s) {
    const int wide = a.act == MOE_ACT_SWIGLU ? 2 * a.N : a.N;
    // most tiles there can be: a group's last one may be short
    const long long sms = num_sms(), groups = a.offsets ? (a.G < a.M ? a.G : a.M) : 1;
    const auto tiles = [&](int bt, int bn) {
        return (a.offsets ? a.M / bt + groups : (a.M + bt - 1) / bt) * ((wide + bn - 1) / bn);
    };
    if (tiles(32, BN) > 0x3FFFFFFF) return cudaErrorNotSupported;
    const long long rows = a.M / groups;   // of a group on average
    const long long n32 = tiles(32, BN), n128 = tiles(128, BN), n256 = tiles(256, 2 * BN);
    if (rows <= 32) return launch_tiles<32, false, TY>(a, wide, n32, parts_of<32, false, TY>(n32, a.KB), s);
    const int single = parts_of<128, false, TY>(n128, a.KB);
    if (a.offsets) {
        // Pairs where that leaves one of them for every other SM.  Few places a group: shorter stages, and more of them on
        // their way, until many groups take a second tile (us by 128, by 256 places: 70 places a group of 128 of 1536 x 2048
        // 138.8, 144.4; 97 of 32 of 2880 x 2880 101.8, 106.5; 110 of 16 of 4096 x 4096 93.5, 101.7, of 64 of 2048 x 1408 72.4,
        // 70.9; 128 108.1, 108.8 and 110.6, 103.1 and 77.5, 72.0; 160 140.2, 112.9 and 124.3, 104.9 and 99.4, 74.8).
        if (rows <= 64 || 2 * n256 < sms) return launch_tiles<128, false, TY>(a, wide, n128, single, s);
        return rows <= 110 ? launch_tiles<128, true, TY>(a, wide, tiles(128, 2 * BN), 1, s)
                           : launch_tiles<256, true, TY>(a, wide, n256, 1, s);
    }
    // One matrix: what takes fewer cycles.  A stage of either comes in about 560 (32 KB from L2); pairs have a longer start and
    // end, and an exchange between parts its own.  us, by pairs and by one block a tile: 256 x 2048 by 7168 x 2048 16.2, 13.9;
    // 512 17.9, 22.7; 2048 37.5, 58.1; 512 x 7168 by 2048 x 7168 26.1, 21.5; 1024 27.3, 33.6; 512 x 4096 by 4096 x 4096 22.4,
    // 22.7; 1024 x 4096 by 1536 x 4096 19.5, 21.2; 512 x 2880 by 2880 x 2880 16.8, 16.2; 2048 x 4096 by 512 x 4096 19.0, 15.5;
    // 256 x 1024 by 8192 x 1024 13.3, 9.3 (128 to 4096 rows by these seven matrices: the faster, or within 4% of it).
    const int both = parts_of<256, true, TY>(n256, a.KB);
    const auto cycles = [&](long long n, int parts, long long slots, int stage, int fixed, int exchange) {
        return (n + slots - 1) / slots * ((a.KB + parts - 1) / parts) * stage + fixed + (parts > 1 ? exchange : 0);
    };
    if (cycles(n256, both, both > 1 ? n256 : sms / 2, 550, 18000, 6000) <
        cycles(n128, single, single > 1 ? n128 : sms, 575, 9000, 4000))
        return launch_tiles<256, true, TY>(a, wide, n256, both, s);
    return launch_tiles<128, false, TY>(a, wide, n128, single, s);
}

}  // namespace

static long long g_wait = 0;   // 0: the kernel's own bound
static int g_hold = 0;
void hold_matmul(int hold, long long cycles) {
    g_hold = hold;
    g_wait = cycles;
}

cudaError_t launch_matmul(MatmulArgs a, cudaStream_t s) {
    a.KB = (a.K + BK - 1) / BK;
    a.wait = g_wait > 0 && (g_wait >> 16) < kWaitLimit ? (uint32_t)(g_wait >> 16) : kWaitLimit;
    a.hold_copies = g_hold == 1;
    a.hold_products = g_hold == 2;
    a.wdims = a.act == MOE_ACT_SWIGLU ? 5 : a.transposed && a.N % 64 == 0 ? 4 : 3;
    if (matmul_few_rows(a)) return launch_matmul_rows(a, s);
    return a.ybf16 ? launch_matmul_t<__nv_bfloat16>(a, s) : launch_matmul_t<float>(a, s);
}

}  // namespace moe
