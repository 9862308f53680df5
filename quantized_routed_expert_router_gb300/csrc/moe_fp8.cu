// moe_fp8.cu - products of e4m3 rows with e4m3 matrices whose scales cover
// blocks of 128 (moe_fp8_matmul), dense or grouped by expert.
//
//   y[i][n] = sum_b sx[r_i][b] sw[g][n/128][b] * D_b[i][n],
//   D_b[i][n] = sum over the 128 values of block b of x8[r_i][.] w[g][n][.]
//
// D_b is one 128-deep product on the tensor cores (four tcgen05.mma of depth
// 32, accumulated in TMEM in fp32); the scales change from block to block, so
// every D_b is read back and added to fp32 registers with its scale.  The
// warps of a block have roles that work on different blocks b at once:
//   warp 0    : TMA copies of w tiles, and of x tiles where the rows are in
//               order (128 bytes deep, 128-byte swizzle), into a ring of stages
//   warp 1    : one thread issues the products into one of the TMEM buffers
//   warps 2-3 : rows that are gathered, by 16-byte asynchronous copies
//   warps 4.. : acc += (sx * sw) * D_b, 64 columns a warp.  TMEM gives lane i of
//               the tile to thread i, so sx is one number a thread and sw one a
//               warp: the scaling is one (packed) multiply-add a value
// A tile is 128 places of one group by BN columns.  Blocks beyond the ends of
// x, w or K are zero-filled; rows of other groups that a tile happens to load
// only reach accumulators that are not stored.
//
// Large products are persistent blocks, one an SM, over the tiles (BN 256).
// When there are fewer tiles than SMs, a cluster of S blocks splits the depth of
// a tile and adds its parts through distributed shared memory in rank order.
#include <cuda.h>
#include <cuda_bf16.h>

#include "moe_common.cuh"
#include "moe_launch.h"

namespace moe {
namespace {

constexpr int BM = 128;             // places of a tile (TMEM lanes)
constexpr int BK = 128;             // bytes of depth of a stage (one scale block)
constexpr int EPI_FIRST = 4;        // first accumulating warp
constexpr int HC = 64;              // columns of an accumulating warp
constexpr int GATHER_LAG = 2;       // stages of gathered rows in flight before one is handed over
constexpr int RED_PITCH = BM + 1;   // fp32 partial tiles, column by column
// bound on every device-side wait, in SM clock cycles (under a second)
constexpr long long FP8_WAIT_CYCLES = 800ll * 1000ll * 1000ll;

template <int BN>
struct Shape {
    static constexpr int STAGES = BN == 256 ? 4 : 6;
    static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE = A_BYTES + B_BYTES;
    static constexpr int SMEM = STAGES * STAGE + 1024;   // + alignment of the swizzle pattern
    static constexpr int NBUF = 512 / BN;                // TMEM buffers
    static constexpr int AHEAD = BN == 256 ? 2 : 4;      // 16-column loads on their way in an accumulating warp
    static constexpr int EPI_WARPS = 4 * (BN / HC), THREADS = 32 * (EPI_FIRST + EPI_WARPS);
};

struct Fp8Args {
    const uint8_t *x;
    const float *xs, *ws;
    const int32_t *rows, *offsets;
    void *y;
    unsigned *status;
    int X, M, G, N, K, KB, NB, ntn;
    int xbox;      // rows of an x copy (ungathered)
};

struct Ctl {
    uint64_t full[6], empty[6], dfull[4], dempty[4], drain;
    uint32_t tmem;
    int abort;
    int goff[MOE_MAX_EXPERTS + 1];     // first place of each group, clamped
    int tstart[MOE_MAX_EXPERTS + 1];   // first 128-place tile of each group
};

// ------------------------------------------------------------ PTX helpers

__device__ __forceinline__ uint32_t sa(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t *b, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(sa(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(sa(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(sa(b)) : "memory");
}
__device__ __forceinline__ bool bar_test(uint64_t *b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(sa(b)), "r"(parity) : "memory");
    return ok != 0;
}
// one lane of a converged warp.  The single-thread instructions (copies, products,
// commits) sit behind this inside loops that the whole warp runs: behind a
// test of the lane number one stage's four products took 540-800 cycles to issue.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
// wait for a phase; false once this block has given up (the first wait to run
// out says so to the others and in the status word)
__device__ __noinline__ bool bar_wait_slow(uint64_t *b, uint32_t parity, Ctl *c, unsigned *status) {
    const long long t0 = clock64();
    while (!bar_test(b, parity)) {
        if (*(volatile int *)&c->abort) return false;
        if (clock64() - t0 > FP8_WAIT_CYCLES) {
            *(volatile int *)&c->abort = 1;
            atomicOr(status, MOE_DEV_TIMEOUT);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool bar_wait(uint64_t *b, uint32_t parity, Ctl *c, unsigned *status) {
    return bar_test(b, parity) || bar_wait_slow(b, parity, c, status);
}
// wait on the way out of a block that has given up: for its own copies and
// products in flight, bounded by itself
__device__ __noinline__ void bar_settle(uint64_t *b, uint32_t parity) {
    const long long t0 = clock64();
    while (!bar_test(b, parity))
        if (clock64() - t0 > FP8_WAIT_CYCLES) return;
}
__device__ __forceinline__ void tma_tile(void *dst, const CUtensorMap *m, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            sa(dst)), "l"(m), "r"(x), "r"(y), "r"(sa(bar))
        : "memory");
}
// 16 bytes, or 16 zeros where `bytes` is 0
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// shared-memory descriptor of a K-major tile with 128-byte rows and the
// 128-byte swizzle: 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"(add)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(sa(bar)) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t v[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}
// waits for this thread's loads; the values pass through it, so that none is used before it
__device__ __forceinline__ void tmem_ld_wait(uint32_t v[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 ::"memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// acc (two fp32) += {lo, hi} * {s, s}
__device__ __forceinline__ void fma2(uint64_t &acc, uint32_t lo, uint32_t hi, uint64_t ss) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(d), "l"(ss));
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float ld_peer(uint32_t addr, uint32_t rank) {
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

// -------------------------------------------------------------- the tile

struct Tile {
    int g, first, rows, n0;   // group, first place, places (1..128), first column
};
// tiles of a group: its 128-place tiles fastest, so that blocks at work at the
// same time share a matrix tile in L2
__device__ __forceinline__ Tile tile_at(const Ctl *c, const Fp8Args &a, int t, int BN) {
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
    r.n0 = local / mt * BN;
    r.first = c->goff[lo] + local % mt * BM;
    r.rows = min(BM, c->goff[lo + 1] - r.first);
    return r;
}

template <typename TY>
__device__ __forceinline__ void store_cols(TY *y, const uint64_t *acc, int cols, bool vec);
// 32 columns: whole 16-byte pieces where the row is aligned, one by one else
template <>
__device__ __forceinline__ void store_cols<float>(float *y, const uint64_t *acc, int cols, bool vec) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float4 v;
        v.x = __uint_as_float((uint32_t)acc[2 * i]);
        v.y = __uint_as_float((uint32_t)(acc[2 * i] >> 32));
        v.z = __uint_as_float((uint32_t)acc[2 * i + 1]);
        v.w = __uint_as_float((uint32_t)(acc[2 * i + 1] >> 32));
        if (vec && 4 * i + 4 <= cols) {
            *reinterpret_cast<float4 *>(y + 4 * i) = v;
        } else {
            if (4 * i < cols) y[4 * i] = v.x;
            if (4 * i + 1 < cols) y[4 * i + 1] = v.y;
            if (4 * i + 2 < cols) y[4 * i + 2] = v.z;
            if (4 * i + 3 < cols) y[4 * i + 3] = v.w;
        }
    }
}
template <>
__device__ __forceinline__ void store_cols<__nv_bfloat16>(__nv_bfloat16 *y, const uint64_t *acc, int cols, bool vec) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint64_t v = acc[4 * i + j];
            h[j] = __floats2bfloat162_rn(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
        }
        if (vec && 8 * i + 8 <= cols) {
            const uint32_t *w = reinterpret_cast<const uint32_t *>(h);
            *reinterpret_cast<uint4 *>(y + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (8 * i + 2 * j < cols) y[8 * i + 2 * j] = h[j].x;
                if (8 * i + 2 * j + 1 < cols) y[8 * i + 2 * j + 1] = h[j].y;
            }
        }
    }
}

template <int BN, typename TY, bool SPLIT>
__global__ void __launch_bounds__(Shape<BN>::THREADS, 1)
    fp8_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw, const Fp8Args a) {
    using S = Shape<BN>;
    constexpr int THREADS = S::THREADS, NBUF = S::NBUF;
    extern __shared__ uint8_t raw[];
    __shared__ Ctl c;
    uint8_t *stages = raw + ((1024 - (sa(raw) & 1023)) & 1023);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            bar_init(&c.full[i], a.rows ? 3 : 1);   // the w copy, and the two gathering warps
            bar_init(&c.empty[i], 1);
        }
        for (int i = 0; i < NBUF; ++i) {
            bar_init(&c.dfull[i], 1);
            bar_init(&c.dempty[i], S::EPI_WARPS);
        }
        bar_init(&c.drain, 1);
        c.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(&c.tmem)),
                     "n"(NBUF * BN) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (!a.offsets) {
        if (threadIdx.x == 0) {
            c.goff[0] = c.tstart[0] = 0;
            c.goff[1] = a.M;
            c.tstart[1] = (a.M + BM - 1) / BM;
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
                const int mt = g < a.G ? (max(c.goff[g + 1] - c.goff[g], 0) + BM - 1) / BM : 0;
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
    const int total = c.tstart[a.G] * a.ntn;
    const int rank = SPLIT ? (int)cluster_rank() : 0, parts = SPLIT ? (int)cluster_size() : 1;
    const int t0 = SPLIT ? (int)blockIdx.x / parts : (int)blockIdx.x, dt = SPLIT ? total : (int)gridDim.x;
    const int kb0 = SPLIT ? rank * a.KB / parts : 0, kb1 = SPLIT ? (rank + 1) * a.KB / parts : a.KB;

    if (warp == 0) {
        const uint32_t bytes = (a.rows ? 0 : a.xbox) * BK + S::B_BYTES;
        int it = 0;
        bool ok = true;
        for (int t = t0; t < total && ok; t += dt) {
            const Tile tl = tile_at(&c, a, t, BN);
            const int wrow = __shfl_sync(0xFFFFFFFFu, tl.g * a.N + tl.n0, 0);
            const int xrow = __shfl_sync(0xFFFFFFFFu, tl.first, 0);
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int st = it % S::STAGES;
                ok = bar_wait(&c.empty[st], ((it / S::STAGES) & 1) ^ 1, &c, a.status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                uint8_t *sx = stages + st * S::STAGE;
                if (elect()) {
                    bar_expect(&c.full[st], bytes);
                    tma_tile(sx + S::A_BYTES, &mw, kb * BK, wrow, &c.full[st]);
                    if (!a.rows) tma_tile(sx, &mx, kb * BK, xrow, &c.full[st]);
                }
                __syncwarp();
            }
        }
        // copies in flight land, and their stages are handed back, before the block ends
        for (int i = it > S::STAGES ? it - S::STAGES : 0; i < it; ++i)
            bar_settle(ok ? &c.empty[i % S::STAGES] : &c.full[i % S::STAGES], (i / S::STAGES) & 1);
        __syncwarp();
    } else if (warp == 1) {
        constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
        int it = 0;
        bool ok = true;
        for (int t = t0; t < total && ok; t += dt) {
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int st = it % S::STAGES, buf = it % NBUF;
                ok = bar_wait(&c.dempty[buf], ((it / NBUF) & 1) ^ 1, &c, a.status) &&
                     bar_wait(&c.full[st], (it / S::STAGES) & 1, &c, a.status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                fence_after();
                const uint32_t sx = sa(stages) + st * S::STAGE;
                const uint64_t ad = tile_desc(sx), bd = tile_desc(sx + S::A_BYTES);
                if (elect()) {
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)   // 32 bytes of depth: 2 units of 16 bytes
                        mma_e4m3(tmem + buf * BN, ad + 2 * k, bd + 2 * k, idesc, k);
                    mma_commit(&c.empty[st]);
                    mma_commit(&c.dfull[buf]);
                }
                __syncwarp();
            }
        }
        if (!ok) {   // products in flight end before TMEM is freed
            if (elect()) mma_commit(&c.drain);
            __syncwarp();
            bar_settle(&c.drain, 0);
        }
        __syncwarp();
    } else if (warp < EPI_FIRST) {
        if (a.rows) {
            // thread: 16 bytes (piece pc) of rows r0, r0 + 8, ...; the swizzle moves piece p of row r to p ^ (r & 7)
            const int id = threadIdx.x - 64, pc = id & 7, r0 = id >> 3;
            const uint32_t to = sa(stages) + r0 * BK + ((pc ^ r0) << 4);
            int it = 0;
            bool ok = true;
            for (int t = t0; t < total && ok; t += dt) {
                const Tile tl = tile_at(&c, a, t, BN);
                int row[BM / 8];
#pragma unroll
                for (int i = 0; i < BM / 8; ++i) {
                    const int r = r0 + 8 * i < tl.rows ? a.rows[tl.first + r0 + 8 * i] : 0;
                    row[i] = (unsigned)r < (unsigned)a.X ? r : 0;
                }
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int st = it % S::STAGES;
                    ok = bar_wait(&c.empty[st], ((it / S::STAGES) & 1) ^ 1, &c, a.status);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const int at = kb * BK + 16 * pc;
                    const uint32_t bytes = at < a.K ? 16 : 0;
                    const uint8_t *src = a.x + (bytes ? at : 0);
#pragma unroll
                    for (int i = 0; i < BM / 8; ++i)
                        if (r0 + 8 * i < tl.rows)
                            copy16(to + st * S::STAGE + i * 8 * BK, src + (size_t)row[i] * a.K, bytes);
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    if (it >= GATHER_LAG) {
                        asm volatile("cp.async.wait_group %0;" ::"n"(GATHER_LAG) : "memory");
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) bar_arrive(&c.full[(it - GATHER_LAG) % S::STAGES]);
                    }
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                for (int i = it > GATHER_LAG ? it - GATHER_LAG : 0; i < it; ++i) bar_arrive(&c.full[i % S::STAGES]);
        }
    } else {
        const int quad = warp & 3, part = (warp - EPI_FIRST) >> 2;   // TMEM lanes and columns of this warp
        const int lrow = 32 * quad + lane;
        int it = 0;
        bool ok = true;
        for (int t = t0; t < total && ok; t += dt) {
            const Tile tl = tile_at(&c, a, t, BN);
            const int n0 = tl.n0 + part * HC;
            const bool mine = lrow < tl.rows;
            const bool work = 32 * quad < tl.rows && n0 < a.N;   // uniform over the warp
            int row = mine ? tl.first + lrow : 0;
            bool bad = false;
            if (a.rows && mine) {
                row = a.rows[row];
                bad = (unsigned)row >= (unsigned)a.X;
                if (bad) {
                    row = 0;
                    atomicOr(a.status, MOE_DEV_BAD_ROW);
                }
            }
            const float *xs = a.xs + (size_t)row * a.KB;
            const float *ws = a.ws + ((size_t)tl.g * a.NB + (work ? n0 / BK : 0)) * a.KB;
            uint64_t acc[HC / 2];
#pragma unroll
            for (int i = 0; i < HC / 2; ++i) acc[i] = 0;
            float nx = 0.f, nw = 0.f;
            if (work) {
                nx = xs[kb0];
                nw = ws[kb0];
            }
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int buf = it % NBUF;
                const float s = nx * nw;
                if (work && kb + 1 < kb1) {
                    nx = xs[kb + 1];
                    nw = ws[kb + 1];
                }
                ok = bar_wait(&c.dfull[buf], (it / NBUF) & 1, &c, a.status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                fence_after();
                if (work) {
                    uint64_t ss;
                    asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "r"(__float_as_uint(s)));
                    const uint32_t at = tmem + buf * BN + part * HC + ((uint32_t)(32 * quad) << 16);
                    // Beside running products a load takes about 250 cycles, however much is on its way, so as
                    // much is as the registers beside the sums hold: all 64 columns (BN 128), or the next 16
                    // while 16 are added (BN 256).  The buffer goes back before the last columns are added.
                    uint32_t u[S::AHEAD][16];
                    if constexpr (S::AHEAD == 4) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) tmem_ld16(at + 16 * j, u[j]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) tmem_ld_wait(u[j]);
                    } else {
                        tmem_ld16(at, u[0]);
                    }
#pragma unroll
                    for (int j = 0; j < HC / 16; ++j) {
                        uint32_t *v = u[j % S::AHEAD];
                        if constexpr (S::AHEAD == 2) {
                            tmem_ld_wait(v);
                            if (j + 1 < HC / 16) tmem_ld16(at + 16 * (j + 1), u[(j + 1) % 2]);
                        }
                        if (j == (S::AHEAD == 4 ? 0 : HC / 16 - 1)) {
                            fence_before();
                            if (lane == 0) bar_arrive(&c.dempty[buf]);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) fma2(acc[8 * j + i], v[2 * i], v[2 * i + 1], ss);
                    }
                } else if (lane == 0) {
                    bar_arrive(&c.dempty[buf]);
                }
            }
            if (!ok) break;
            if (bad) {
#pragma unroll
                for (int i = 0; i < HC / 2; ++i) acc[i] = 0;
            }
            if (SPLIT) {
                // this block's part, over the stages (every copy and product is done)
                float *red = reinterpret_cast<float *>(stages);
                if (mine && work) {
#pragma unroll
                    for (int i = 0; i < HC / 2; ++i) {
                        red[(part * HC + 2 * i) * RED_PITCH + lrow] = __uint_as_float((uint32_t)acc[i]);
                        red[(part * HC + 2 * i + 1) * RED_PITCH + lrow] = __uint_as_float((uint32_t)(acc[i] >> 32));
                    }
                }
            } else if (mine && work) {
                TY *y = static_cast<TY *>(a.y) + (size_t)(tl.first + lrow) * a.N + n0;
                const bool vec = a.N % (16 / (int)sizeof(TY)) == 0;
#pragma unroll
                for (int j = 0; j < HC; j += 32)
                    if (n0 + j < a.N) store_cols<TY>(y + j, acc + j / 2, a.N - n0 - j, vec);
            }
        }
    }
    if (SPLIT) {
        __syncwarp();
        cluster_sync();
        if (warp >= EPI_FIRST && t0 < total && !*(volatile int *)&c.abort) {
            // each block adds its share of the columns over the cluster, in rank order
            const Tile tl = tile_at(&c, a, t0, BN);
            const int C = BN / parts, c0 = rank * C;
            const uint32_t red = sa(stages);
            for (int i = threadIdx.x - 32 * EPI_FIRST; i < tl.rows * C; i += S::EPI_WARPS * 32) {
                const int col = c0 + i % C, r = i / C;
                if (tl.n0 + col >= a.N) continue;
                float v = 0.f;
                for (int p = 0; p < parts; ++p) v += ld_peer(red + (col * RED_PITCH + r) * 4, p);
                static_cast<TY *>(a.y)[(size_t)(tl.first + r) * a.N + tl.n0 + col] = (TY)v;
            }
        }
        cluster_sync();   // parts are read before their block ends
    }
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(NBUF * BN));
    }
}

// ------------------------------------------------------------------ host

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (EncodeTiled)p;
    }();
    return fn;
}

// rows x depth bytes, copied in boxes of `box` rows by 128 bytes
bool encode(CUtensorMap *m, const void *p, size_t rows, size_t depth, int box) {
    const cuuint64_t dims[2] = {depth, rows}, strides[1] = {depth};
    const cuuint32_t boxes[2] = {BK, (cuuint32_t)box}, steps[2] = {1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, boxes, steps,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, typename TY, bool SPLIT>
cudaError_t launch_t(const CUtensorMap &mx, const CUtensorMap &mw, const Fp8Args &a, int grid, int split, cudaStream_t s) {
    constexpr int smem = Shape<BN>::SMEM;
    auto *k = fp8_kernel<BN, TY, SPLIT>;
    cudaError_t err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(Shape<BN>::THREADS);
    cfg.dynamicSmemBytes = smem;
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

template <typename TY>
cudaError_t launch_fp8_t(Fp8Args a, const void *x8, const void *w, int K, cudaStream_t s) {
    // most 128-place tiles there can be: a group's last tile may be short
    const long long sms = num_sms();
    const long long mt = a.offsets ? (long long)(a.M / BM) + (a.G < a.M ? a.G : a.M) : (a.M + BM - 1) / BM;
    const long long t128 = mt * ((a.N + 127) / 128), t256 = mt * ((a.N + 255) / 256);
    if (t256 > 0x3FFFFFFF || t128 > 0x3FFFFFFF) return cudaErrorNotSupported;
    int split = 1;
    while (split < 8 && t128 * split * 2 <= sms && a.KB >= split * 4) split *= 2;
    const bool wide = split == 1 && t256 >= sms && a.M >= 64 * mt;
    CUtensorMap mx, mw;
    a.xbox = a.M >= BM || a.offsets ? BM : (a.M + 7) / 8 * 8;
    if (!encode_fn()) return cudaErrorSymbolNotFound;
    if (!encode(&mx, x8, (size_t)a.X, (size_t)K, a.xbox) ||
        !encode(&mw, w, (size_t)a.G * a.N, (size_t)K, wide ? 256 : 128))
        return cudaErrorInvalidValue;
    a.ntn = wide ? (a.N + 255) / 256 : (a.N + 127) / 128;
    if (split > 1) return launch_t<128, TY, true>(mx, mw, a, (int)(t128 * split), split, s);
    if (wide) return launch_t<256, TY, false>(mx, mw, a, (int)(t256 < sms ? t256 : sms), 1, s);
    return launch_t<128, TY, false>(mx, mw, a, (int)(t128 < sms ? t128 : sms), 1, s);
}

}  // namespace

cudaError_t launch_fp8(const void *x8, const float *x_scale, int X, const int32_t *rows, int M, const int32_t *offsets,
                       int G, const void *w, const float *w_scale, int N, int K, void *y, int ydtype,
                       unsigned *status, cudaStream_t s) {
    Fp8Args a = {};
    a.x = static_cast<const uint8_t *>(x8);
    a.xs = x_scale;
    a.ws = w_scale;
    a.rows = rows;
    a.offsets = offsets;
    a.y = y;
    a.status = status;
    a.X = X;
    a.M = M;
    a.G = G;
    a.N = N;
    a.K = K;
    a.KB = (K + BK - 1) / BK;
    a.NB = (N + BK - 1) / BK;
    return ydtype == MOE_DT_BF16 ? launch_fp8_t<__nv_bfloat16>(a, x8, w, K, s) : launch_fp8_t<float>(a, x8, w, K, s);
}

}  // namespace moe
