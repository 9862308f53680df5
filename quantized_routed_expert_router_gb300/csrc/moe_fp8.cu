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
//   warps 2-3 : rows that are gathered, by 16-byte asynchronous copies that
//               signal the stage when they land
//   warps 4.. : acc += (sx * sw) * D_b, 64 columns a warp.  TMEM gives lane i of
//               the tile to thread i, so sx is one number a thread and sw one a
//               warp: the scaling is one multiply-add (half a packed one) a value
// A tile is 128 places of one group by BN columns.  Blocks beyond the ends of
// x, w or K are zero-filled; rows of other groups that a tile happens to load
// only reach accumulators that are not stored.
//
// Large products are persistent blocks, one an SM, over the tiles.  When there
// are too few tiles for the SMs, a cluster of S blocks splits the depth of a
// tile and adds its parts through distributed shared memory in rank order.
#include <cuda.h>
#include <cuda_bf16.h>

#include "moe_around.h"
#include "moe_common.cuh"
#include "moe_launch.h"
#include "moe_tc.cuh"

namespace moe {
namespace {

constexpr int BM = 128;             // places of a tile (TMEM lanes)
constexpr int BK = 128;             // bytes of depth of a stage (one scale block)
constexpr int EPI_FIRST = 4;        // first accumulating warp
constexpr int HC = 64;              // columns of an accumulating warp
constexpr int GATHER_THREADS = 64;  // warps 2 and 3
constexpr int MAX_SPLIT = 8;        // blocks that share a tile's depth
constexpr int RED_PITCH = BM + 4;   // fp32 partial tiles, column by column; 16-byte pieces free of bank conflicts

// What bounds the tiles is how the sums come back: a TMEM load beside running
// products takes about 250 cycles however wide it is, so a warp has all of its
// 64 columns on their way at once, 64 registers beside its 64 sums.  128 x 192
// is the widest tile whose sums and loads fit the register file (12 warps, 122
// registers); at 128 x 256 a warp could have 16 columns on their way, and a block
// of depth took 950 cycles where its products take 512.  Moving registers from
// the feeding warps to the accumulating ones gained 1 to 3% and is not done.
template <int BN>
struct Shape {
    static constexpr int STAGES = BN == 192 ? 5 : 6;
    static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE = A_BYTES + B_BYTES;
    static constexpr int SMEM = STAGES * STAGE + 1024;   // + alignment of the swizzle pattern
    static constexpr int NBUF = 512 / BN;                // TMEM buffers
    static constexpr int EPI_WARPS = 4 * (BN / HC), THREADS = 32 * (EPI_FIRST + EPI_WARPS);
    // a split tile's part and the sums of a block's share lie over the stages
    static_assert(4 * (BN * RED_PITCH + BM * (BN / 2 + 4)) <= STAGES * STAGE, "");
};
struct Ctl {
    uint64_t full[6], done[6];   // a stage is loaded; its products are done (the stage is free, the sums are there)
    uint64_t dempty[4], drain;   // a TMEM buffer is read
    uint32_t tmem;
    int abort;
    int goff[MOE_MAX_EXPERTS + 1];     // first place of each group, clamped
    int tstart[MOE_MAX_EXPERTS + 1];   // first 128-place tile of each group
};

// ------------------------------------------------------------ PTX helpers

// wait for a phase; false once this block has given up.  Inline: a call would take registers that the accumulating warps
// do not have.
__device__ __forceinline__ bool bar_wait(uint64_t *b, uint32_t parity, Ctl *c, const Fp8Args &a) {
    return bar_wait(b, parity, &c->abort, a.wait, a.status);
}
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t add, uint32_t me) {
    asm volatile(
        "{\n .reg .pred e, p;\n setp.ne.u32 e, %5, 0;\n setp.ne.u32 p, %4, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"(add),
        "r"(me)
        : "memory");
}
// two sums += {lo, hi} * {s, s}
__device__ __forceinline__ void fma2(uint64_t &acc, uint32_t lo, uint32_t hi, uint64_t ss) {
    asm volatile("{\n .reg .b64 d;\n mov.b64 d, {%1, %2};\n fma.rn.f32x2 %0, d, %3, %0;\n}"
                 : "+l"(acc) : "r"(lo), "r"(hi), "l"(ss));
}
// sum i of a warp's packed ones
__device__ __forceinline__ float sum_of(const uint64_t *acc, int i) {
    return __uint_as_float((uint32_t)(acc[i / 2] >> (32 * (i & 1))));
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

// 32 columns of a row of which `align` bytes are aligned, 32 or 16: 32 bytes a lane
// (whole sectors) or 16; a tile's last columns value by value.
__device__ __forceinline__ void store32(void *p, const uint32_t w[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
template <typename TY>
__device__ __forceinline__ void store_cols(TY *y, const uint64_t *acc, int cols, int align) {
    constexpr int PER = 32 / (int)sizeof(TY);   // values of a 32-byte piece
#pragma unroll
    for (int i = 0; i < 32 / PER; ++i) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (sizeof(TY) == 4) {
                w[j] = __float_as_uint(sum_of(acc, 8 * i + j));
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(sum_of(acc, 16 * i + 2 * j), sum_of(acc, 16 * i + 2 * j + 1));
                w[j] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        TY *to = y + PER * i;
        if (align >= 32 && PER * i + PER <= cols) {
            store32(to, w);
        } else if (PER * i + PER <= cols) {
            *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4 *>(to + PER / 2) = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                if (PER * i + j >= cols) break;
                if constexpr (sizeof(TY) == 4) to[j] = __uint_as_float(w[j]);
                else to[j] = __ushort_as_bfloat16((unsigned short)(w[j / 2] >> (16 * (j & 1))));
            }
        }
    }
}

// The sums of a warp where rows of y are not aligned to 16 bytes (an odd N): 32 rows
// by 8 words at a time turn in shared memory and leave value by value, columns side
// by side.  Straight from the lanes each store touched 32 rows: 3221 x 6993 x 768
// took 219 us, and takes 49.
constexpr int TURN_PITCH = 9;   // words, free of bank conflicts
template <typename TY>
__device__ __forceinline__ void store_turned(TY *y, size_t N, const uint64_t *acc, int rows, int cols, uint32_t *turn,
                                             int lane) {
    constexpr int PER = 32 / (int)sizeof(TY);   // values of a row's 8 words
#pragma unroll
    for (int i = 0; i < HC / PER; ++i) {
        if (PER * i >= cols) break;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (sizeof(TY) == 4) {
                turn[TURN_PITCH * lane + j] = __float_as_uint(sum_of(acc, 8 * i + j));
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(sum_of(acc, 16 * i + 2 * j), sum_of(acc, 16 * i + 2 * j + 1));
                turn[TURN_PITCH * lane + j] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        __syncwarp();
        const int col = lane % PER;
        if (PER * i + col < cols) {
#pragma unroll 4
            for (int r = lane / PER; r < 32; r += 32 / PER)
                if (r < rows)
                    y[r * N + PER * i + col] = reinterpret_cast<const TY *>(turn + TURN_PITCH * r)[col];
        }
    }
}

// 4 columns of a row, of which `cols` are there
template <typename TY>
__device__ __forceinline__ void store4(TY *y, float4 v, int cols, bool aligned) {
    if (aligned && cols >= 4) {
        if constexpr (sizeof(TY) == 4) {
            *reinterpret_cast<float4 *>(y) = v;
        } else {
            const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
            *reinterpret_cast<uint2 *>(y) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
        }
    } else {
        if (cols > 0) y[0] = (TY)v.x;
        if (cols > 1) y[1] = (TY)v.y;
        if (cols > 2) y[2] = (TY)v.z;
        if (cols > 3) y[3] = (TY)v.w;
    }
}

template <int BN, typename TY, bool SPLIT, bool TURN>
__global__ void __launch_bounds__(Shape<BN>::THREADS, 1)
    fp8_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw, const Fp8Args a) {
    using S = Shape<BN>;
    constexpr int THREADS = S::THREADS, NBUF = S::NBUF, STAGES = S::STAGES - (TURN ? 1 : 0);
    static_assert(!TURN || 4 * 32 * TURN_PITCH * S::EPI_WARPS <= S::STAGE, "");
    extern __shared__ uint8_t raw[];
    __shared__ Ctl c;
    uint8_t *stages = raw + ((1024 - (sa(raw) & 1023)) & 1023);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            bar_init(&c.full[i], (a.rows ? 1 + GATHER_THREADS : 1) + a.hold_copies);   // TMA's copies, and the gathered rows
            bar_init(&c.done[i], 1 + a.hold_products);
        }
        for (int i = 0; i < NBUF; ++i) bar_init(&c.dempty[i], S::EPI_WARPS);
        bar_init(&c.drain, 1);
        c.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(&c.tmem)),
                     "n"(512) : "memory");
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
    // Rising offsets have fewer than 2^30 tiles (the launch checks it).  Falling ones let groups overlap and can have up to
    // G / 2 times as many: no more than 2^30 of them, so that tile numbers stay in 32 bits.
    const int total = (int)min((long long)c.tstart[a.G] * a.ntn, 0x3FFFFFFFll);
    const int rank = SPLIT ? (int)cluster_rank() : 0, parts = SPLIT ? (int)cluster_size() : 1;
    const int t0 = SPLIT ? (int)blockIdx.x / parts : (int)blockIdx.x, dt = SPLIT ? total : (int)gridDim.x;
    const int kb0 = SPLIT ? rank * a.KB / parts : 0, kb1 = SPLIT ? (rank + 1) * a.KB / parts : a.KB;

    if (warp < EPI_FIRST) {
        if (warp == 0) {
            const uint32_t bytes = (a.rows ? 0 : a.xbox) * BK + S::B_BYTES, me = elect();
            Ring<STAGES> r;
            int it = 0;
            bool ok = true;
            for (int t = t0; t < total && ok; t += dt) {
                const Tile tl = tile_at(&c, a, t, BN);
                const int wrow = __shfl_sync(0xFFFFFFFFu, tl.g * a.N + tl.n0, 0);
                const int xrow = __shfl_sync(0xFFFFFFFFu, tl.first, 0);
                for (int kb = kb0; kb < kb1; ++kb, ++it, r.next()) {
                    ok = bar_wait(&c.done[r.i], r.phase ^ 1, &c, a);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    uint8_t *sx = stages + r.i * S::STAGE;
                    bar_expect(&c.full[r.i], bytes, me);
                    tma_tile(sx + S::A_BYTES, &mw, kb * BK, wrow, &c.full[r.i], me);
                    if (!a.rows) tma_tile(sx, &mx, kb * BK, xrow, &c.full[r.i], me);
                }
            }
            // copies in flight land, and their products end, before the block ends
            const uint32_t t_out = clock_hi();
            for (int i = it > STAGES ? it - STAGES : 0; i < it; ++i)
                bar_settle(ok ? &c.done[i % STAGES] : &c.full[i % STAGES], (i / STAGES) & 1, t_out);
            __syncwarp();
        } else if (warp == 1) {
            constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
            const uint32_t me = elect();
            Ring<STAGES> r;
            Ring<NBUF> d;
            bool ok = true;
            for (int t = t0; t < total && ok; t += dt) {
                for (int kb = kb0; kb < kb1; ++kb, r.next(), d.next()) {
                    ok = bar_wait(&c.dempty[d.i], d.phase ^ 1, &c, a) && bar_wait(&c.full[r.i], r.phase, &c, a);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    // gathered rows were written through the generic proxy, and the wait made them visible here; the
                    // products read through the async proxy
                    if (a.rows) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    fence_after();
                    const uint32_t sx = sa(stages) + r.i * S::STAGE;
                    const uint64_t ad = tile_desc(sx), bd = tile_desc(sx + S::A_BYTES);
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)   // 32 bytes of depth: 2 units of 16 bytes
                        mma_e4m3(tmem + d.i * BN, ad + 2 * k, bd + 2 * k, idesc, k, me);
                    mma_commit(&c.done[r.i], me);
                }
            }
            if (!ok) {   // products in flight end before TMEM is freed
                mma_commit(&c.drain, me);
                bar_settle(&c.drain, 0, clock_hi());
            }
            __syncwarp();
        } else {
            if (a.rows) {
                // thread: 16 bytes (piece pc) of rows r0, r0 + 8, ...; the swizzle moves piece p of row r to p ^ (r & 7)
                const int id = threadIdx.x - 64, pc = id & 7, r0 = id >> 3;
                const uint32_t to = sa(stages) + r0 * BK + ((pc ^ r0) << 4);
                Ring<STAGES> r;
                bool ok = true;
                for (int t = t0; t < total && ok; t += dt) {
                    const Tile tl = tile_at(&c, a, t, BN);
                    uint32_t row[BM / 8];   // in units of 16 bytes (X K <= 2^36)
#pragma unroll
                    for (int i = 0; i < BM / 8; ++i) {
                        const int x = r0 + 8 * i < tl.rows ? a.rows[tl.first + r0 + 8 * i] : 0;
                        row[i] = (uint32_t)((unsigned)x < (unsigned)a.X ? x : 0) * (uint32_t)(a.K >> 4);
                    }
                    const int nr = (tl.rows - r0 + 7) >> 3;   // of this thread
                    for (int kb = kb0; kb < kb1; ++kb, r.next()) {
                        ok = bar_wait(&c.done[r.i], r.phase ^ 1, &c, a);
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok) break;
                        const bool in = kb * BK + 16 * pc < a.K;
                        const uint8_t *src = a.x + (in ? kb * BK + 16 * pc : 0);
                        const uint32_t bytes = in ? 16 : 0, dst = to + r.i * S::STAGE;
                        if (nr == BM / 8) {
#pragma unroll
                            for (int i = 0; i < BM / 8; ++i) copy16(dst + i * 8 * BK, src + 16 * (uint64_t)row[i], bytes);
                        } else {
#pragma unroll
                            for (int i = 0; i < BM / 8; ++i)
                                if (i < nr) copy16(dst + i * 8 * BK, src + 16 * (uint64_t)row[i], bytes);
                        }
                        // this thread's arrival, once its copies have landed; nobody waits here for them
                        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sa(&c.full[r.i])) : "memory");
                    }
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
            }
        }
    } else {
        const int quad = warp & 3, part = (warp - EPI_FIRST) >> 2;   // TMEM lanes and columns of this warp
        const int lrow = 32 * quad + lane;
        Ring<STAGES> r;
        Ring<NBUF> d;
        bool ok = true;
        for (int t = t0; t < total; t += dt) {
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
            // Nothing in this loop hangs on whether a wait gave up: it ends by itself, its warps stay together,
            // and nothing is stored.  What need not come after the sums stands between their load and the wait for it.
            const uint32_t at0 = tmem + part * HC + ((uint32_t)(32 * quad) << 16);
            for (int kb = kb0; kb < kb1; ++kb) {
                if (ok) ok = bar_wait(&c.done[r.i], r.phase, &c, a);
                __syncwarp();
                fence_after();
                r.next();
                if (work) {
                    // all 64 columns on their way at once; the buffer goes back before they are added
                    uint32_t u[2][32];
                    tmem_ld32_begin(at0 + d.i * BN, u[0]);
                    tmem_ld32_begin(at0 + d.i * BN + 32, u[1]);
                    uint64_t ss;
                    asm volatile("mov.b64 %0, {%1, %1};" : "=l"(ss) : "r"(__float_as_uint(nx * nw)));
                    if (kb + 1 < kb1) {
                        nx = xs[kb + 1];
                        nw = ws[kb + 1];
                    }
                    tmem_landed(u[0]);
                    tmem_landed(u[1]);
                    fence_before();
                    bar_arrive(&c.dempty[d.i], lane == 0);
#pragma unroll
                    for (int i = 0; i < 32; ++i) fma2(acc[i], u[i / 16][2 * (i % 16)], u[i / 16][2 * (i % 16) + 1], ss);
                } else {
                    bar_arrive(&c.dempty[d.i], lane == 0);
                }
                d.next();
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) continue;
            if (bad) {
#pragma unroll
                for (int i = 0; i < HC / 2; ++i) acc[i] = 0;
            }
            if (SPLIT) {
                // this block's part, over the stages (every copy and product is done)
                float *red = reinterpret_cast<float *>(stages);
                if (mine && work) {
#pragma unroll
                    for (int i = 0; i < HC; ++i) red[(part * HC + i) * RED_PITCH + lrow] = sum_of(acc, i);
                }
            } else if (TURN) {
                // in shared memory beside the stages in use
                if (work)
                    store_turned<TY>(static_cast<TY *>(a.y) + (size_t)(tl.first + 32 * quad) * a.N + n0, (size_t)a.N, acc,
                                     tl.rows - 32 * quad, a.N - n0,
                                     reinterpret_cast<uint32_t *>(stages + STAGES * S::STAGE) +
                                         (warp - EPI_FIRST) * 32 * TURN_PITCH,
                                     lane);
            } else if (mine && work) {
                TY *y = static_cast<TY *>(a.y) + (size_t)(tl.first + lrow) * a.N + n0;
#pragma unroll
                for (int j = 0; j < HC; j += 32)
                    if (n0 + j < a.N) store_cols<TY>(y + j, acc + j / 2, a.N - n0 - j, a.yalign);
            }
        }
    }
    if (SPLIT) {
        __syncwarp();
        cluster_sync();
        if (warp >= EPI_FIRST && t0 < total && !*(volatile int *)&c.abort) {
            // Each block adds its share of the columns over the cluster, in rank order: a warp a column, four rows a
            // lane (512 bytes of a part in a piece: with columns side by side a tile of 128 rows in 8 parts took 6 us
            // to add), then from its own shared memory to y with columns side by side.
            const Tile tl = tile_at(&c, a, t0, BN);
            const int lc = 31 - __clz(BN / parts), C = 1 << lc, c0 = rank * C;   // parts: a power of two
            const int pitch = C + 4;
            const uint32_t red = sa(stages) + (c0 * RED_PITCH + 4 * lane) * 4;
            float *sum = reinterpret_cast<float *>(stages) + BN * RED_PITCH;
            // (two columns at a time; otherwise short code, as it runs once, from a cold cache)
#pragma unroll 1
            for (int col = warp - EPI_FIRST; col < C; col += 2 * S::EPI_WARPS) {
                if (4 * lane >= tl.rows) continue;
                float4 part[2][MAX_SPLIT];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int p = 0; p < MAX_SPLIT; ++p)
                        if (p < parts) part[h][p] = ld_peer(red + (col + h * S::EPI_WARPS) * RED_PITCH * 4, p);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float4 v = part[h][0];
#pragma unroll
                    for (int p = 1; p < MAX_SPLIT; ++p)
                        if (p < parts) {
                            v.x += part[h][p].x;
                            v.y += part[h][p].y;
                            v.z += part[h][p].z;
                            v.w += part[h][p].w;
                        }
                    float *to = sum + 4 * lane * pitch + col + h * S::EPI_WARPS;
                    to[0] = v.x;
                    to[pitch] = v.y;
                    to[2 * pitch] = v.z;
                    to[3 * pitch] = v.w;
                }
            }
            asm volatile("bar.sync 1, %0;" ::"n"(S::EPI_WARPS * 32) : "memory");   // the accumulating warps
            TY *y = static_cast<TY *>(a.y) + (size_t)tl.first * a.N + tl.n0 + c0;
            const int cols = min(C, a.N - tl.n0 - c0);
#pragma unroll 1
            for (int i = 4 * (threadIdx.x - 32 * EPI_FIRST); i < tl.rows << lc; i += 4 * S::EPI_WARPS * 32) {
                const int r = i >> lc, col = i & (C - 1);
                const float4 v = *reinterpret_cast<const float4 *>(sum + r * pitch + col);
                store4(y + (size_t)r * a.N + col, v, cols - col, a.yalign >= 16);
            }
        }
        cluster_sync();   // parts are read before their block ends
    }
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512));
    }
}

// ------------------------------------------------------------------ host

// rows x depth bytes, copied in boxes of `box` rows by 128 bytes
bool encode(CUtensorMap *m, const void *p, size_t rows, size_t depth, int box) {
    const cuuint64_t dims[2] = {depth, rows}, strides[1] = {depth};
    const cuuint32_t boxes[2] = {BK, (cuuint32_t)box}, steps[2] = {1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, boxes, steps,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, typename TY, bool SPLIT, bool TURN>
cudaError_t launch_t(const CUtensorMap &mx, const CUtensorMap &mw, const Fp8Args &a, int grid, int split, cudaStream_t s) {
    constexpr int smem = Shape<BN>::SMEM;
    auto *k = fp8_kernel<BN, TY, SPLIT, TURN>;
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
cudaError_t launch_fp8_t(Fp8Args a, cudaStream_t s) {
    // most 128-place tiles there can be: a group's last tile may be short
    const long long sms = num_sms();
    const long long mt = a.offsets ? (long long)(a.M / BM) + (a.G < a.M ? a.G : a.M) : (a.M + BM - 1) / BM;
    const long long t128 = mt * ((a.N + 127) / 128), t192 = mt * ((a.N + 191) / 192);
    if (t128 > 0x3FFFFFFF) return cudaErrorNotSupported;
    // Depth in parts while all parts still have an SM of their own and 4 blocks of depth.  Whole tiles leave SMs idle
    // and each takes a whole depth's time (us in parts, and whole): 256 x 2048 x 7168 11.8, 19.6; 64 x 2048 x 7168
    // 14.4, 19.2; 512 x 1000 x 4096 10.0, 13.7.  At the shallow end, 64 x 7168 x 2048, it is 9.1 and 8.1.
    int split = 1;
    while (split < MAX_SPLIT && t128 * split * 2 <= sms && a.KB >= split * 4) split *= 2;
    // 192 columns where that leaves a tile for every SM and the tiles are at least half full on average: fewer reads of x
    // and w a product.  us with 192, and with 128: 8192 x 2048 x 7168 121, 126; 8192 x 7168 x 2048 131, 140; 128 experts
    // of 1536 x 4096, 65536 rows 499, 525; 32 of 2880 x 2880, 4096 rows 66, 70.  Below the bounds: 1024 x 2048 x 7168
    // (88 tiles) 26.1, 20.8; 256 experts of 512 x 2048, 16384 rows 58.4, 52.6; but 128 of 1536 x 4096, 6216 rows 136, 142.
    // (Tiles are counted as if the rows fell on as many groups as there can be: a batch whose rows fall on few groups
    // has fewer, and its depth stays whole.)
    const bool wide = split == 1 && t192 >= sms && a.M >= 64 * mt;
    CUtensorMap mx, mw;
    a.xbox = a.M >= BM || a.offsets ? BM : (a.M + 7) / 8 * 8;
    const size_t rows_at = (size_t)(uintptr_t)a.y | ((size_t)a.N * sizeof(TY));
    a.yalign = rows_at % 32 == 0 ? 32 : rows_at % 16 == 0 ? 16 : 0;
    if (!encode_fn()) return cudaErrorSymbolNotFound;
    if (!encode(&mx, a.x, (size_t)a.X, (size_t)a.K, a.xbox) ||
        !encode(&mw, a.w, (size_t)a.G * a.N, (size_t)a.K, wide ? 192 : 128))
        return cudaErrorInvalidValue;
    a.ntn = wide ? (a.N + 191) / 192 : (a.N + 127) / 128;
    if (split > 1) return launch_t<128, TY, true, false>(mx, mw, a, (int)(t128 * split), split, s);
    const int grid = (int)(wide ? (t192 < sms ? t192 : sms) : (t128 < sms ? t128 : sms));
    if (a.yalign < 16)
        return wide ? launch_t<192, TY, false, true>(mx, mw, a, grid, 1, s) : launch_t<128, TY, false, true>(mx, mw, a, grid, 1, s);
    return wide ? launch_t<192, TY, false, false>(mx, mw, a, grid, 1, s) : launch_t<128, TY, false, false>(mx, mw, a, grid, 1, s);
}

}  // namespace

static long long g_wait = 0;   // 0: the kernel's own bound
static int g_hold = 0;
void hold_fp8(int hold, long long cycles) {
    g_hold = hold;
    g_wait = cycles;
}

cudaError_t launch_fp8(const void *x8, const float *x_scale, int X, const int32_t *rows, int M, const int32_t *offsets,
                       int G, const void *w, const float *w_scale, int N, int K, void *y, int ydtype,
                       unsigned *status, cudaStream_t s) {
    Fp8Args a = {};
    a.x = static_cast<const uint8_t *>(x8);
    a.w = static_cast<const uint8_t *>(w);
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
    a.wait = g_wait > 0 && (g_wait >> 16) < kWaitLimit ? (uint32_t)(g_wait >> 16) : kWaitLimit;
    a.hold_copies = g_hold == 1;
    a.hold_products = g_hold == 2;
    if (fp8_few_rows(a)) return launch_fp8_rows(a, ydtype, s);
    return ydtype == MOE_DT_BF16 ? launch_fp8_t<__nv_bfloat16>(a, s) : launch_fp8_t<float>(a, s);
}

}  // namespace moe
