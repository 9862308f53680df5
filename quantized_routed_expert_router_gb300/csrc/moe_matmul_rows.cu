// moe_matmul_rows.cu - moe_matmul for few rows: decode of one token to a few.
//
// The weights are read once and bound the call, so nothing is staged: a warp
// loads 16 matrix rows of 32-deep chunks straight into the registers of its
// matrix instructions (m16n8k16, weights as the 16 rows, places as the 8
// columns).  A lane's 16-byte pieces of a matrix row and of an x row hold the same
// depths, and a sum does not mind the order of its terms, so the pieces serve as
// fragments as they are: words 0, 1 for one instruction, 2, 3 for the next.
// Chunks are dealt to the warps of a block; DEPTH of them are on their way at
// once and summed by the tensor cores, these sums and then the warps' in fp32, in
// order.
//
// A block takes 16 matrix rows for a chunk of up to 8 NT places of one group (16
// columns of y; with the gated activation 8 gate rows and the 8 up rows that
// belong to them, which a thread of the epilogue has side by side); chunks start
// at a group's first place.  Against the tiles of moe_matmul.cu this saves the
// tensor maps, the ring's start and the cluster's exchange.  What is left above the
// weights' bytes is a chain of latencies: launch, offsets, weights, the warps' sums
// (8 rows over 8 of 256 experts of 2 x 512 x 2048: 8.9 us on the device, 3.8 TB/s; with
// 80 registers instead of 64 not all of its 512 blocks ran at once, and it took 2 more).
#include <cuda_bf16.h>

#include "moe_around.h"
#include "moe_launch.h"
#include "moe_matmul.cuh"

namespace moe {
namespace {

constexpr int RB = 16;   // matrix rows of a block

__device__ __forceinline__ void mma16816(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 16 bytes of a weight row, read once
__device__ __forceinline__ uint4 ld_weight(const __nv_bfloat16 *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <int NT, int WARPS, int DEPTH, typename TY>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 8 ? NT == 1 ? 4 : NT == 2 ? 3 : 2 : 1) matmul_rows_kernel(const MatmulArgs a) {
    constexpr int CHUNK = 8 * NT;   // places of a block
    __shared__ float red[WARPS][RB][CHUNK + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g8 = lane >> 2, t4 = lane & 3;
    const bool gated = a.act == MOE_ACT_SWIGLU;
    // The row indexes of the places from blockIdx.y on are on their way while the group is looked for: a chunk starts there, or
    // the block has nothing to do.
    int g = 0, first = a.offsets ? blockIdx.y : blockIdx.y * CHUNK, end = a.M;
    int row[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        row[j] = first + 8 * j + g8;
        if (a.rows) row[j] = row[j] < a.M ? a.rows[row[j]] : 0;
    }
    if (a.offsets) {
        // the group of place blockIdx.y: the last one that does not start after it; every warp looks for itself
        int n = 0, start = 0;
        for (int i = lane; i <= a.G; i += 32) {
            const int o = a.offsets[i];
            n += o <= first;
            if (o <= first) start = max(start, o);
            else end = min(end, o);
            if (blockIdx.x == 0 && blockIdx.y == 0 && warp == 0) {
                const int before = i ? a.offsets[i - 1] : 0;
                if (o < before || o > a.M) atomicOr(a.status, MOE_DEV_BAD_ROW);
            }
        }
        n = __reduce_add_sync(0xFFFFFFFFu, n);
        start = __reduce_max_sync(0xFFFFFFFFu, start);
        end = __reduce_min_sync(0xFFFFFFFFu, end);
        if (n < 1 || n > a.G || (first - start) % CHUNK) return;
        g = n - 1;
    }
    const int rows = min(CHUNK, end - first), n0 = blockIdx.x * (gated ? RB / 2 : RB);
    // x rows of this lane's columns.  Columns past the chunk, rows past N and bad indexes read something that is there;
    // nothing of it is stored.
    const __nv_bfloat16 *x[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        if (8 * j + g8 >= rows) {
            row[j] = 0;
        } else if ((unsigned)row[j] >= (unsigned)a.X) {
            atomicOr(a.status, MOE_DEV_BAD_ROW);
            row[j] = 0;
        }
        x[j] = a.x + (size_t)row[j] * a.K;
    }
    const size_t wide = gated ? 2 * (size_t)a.N : (size_t)a.N;
    const int second = gated ? a.N + n0 + g8 : n0 + g8 + 8;
    const __nv_bfloat16 *w = a.w + g * wide * a.K;
    const __nv_bfloat16 *w0 = w + (size_t)min(n0 + g8, a.N - 1) * a.K;
    const __nv_bfloat16 *w1 = w + (size_t)min(second, (int)wide - 1) * a.K;
    float acc[NT][4] = {};
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const int chunks = (a.K + 31) / 32;
    for (int c0 = warp * DEPTH; c0 < chunks; c0 += DEPTH * WARPS) {
        // everything of DEPTH chunks on its way before the first product; past K: zeros
        uint4 wa[DEPTH], wb[DEPTH], xb[DEPTH][NT];
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
            const int k = (c0 + i) * 32 + 8 * t4;
            wa[i] = k < a.K ? ld_weight(w0 + k) : zero;
            wb[i] = k < a.K ? ld_weight(w1 + k) : zero;
#pragma unroll
            for (int j = 0; j < NT; ++j) xb[i][j] = k < a.K ? *reinterpret_cast<const uint4 *>(x[j] + k) : zero;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float d[4] = {};
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) {
                mma16816(d, wa[i].x, wb[i].x, wa[i].y, wb[i].y, xb[i][j].x, xb[i][j].y);
                mma16816(d, wa[i].z, wb[i].z, wa[i].w, wb[i].w, xb[i][j].z, xb[i][j].w);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] += d[i];
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[warp][g8 + 8 * (i >> 1)][8 * j + 2 * t4 + (i & 1)] = acc[j][i];
    __syncthreads();
    const int cols = gated ? RB / 2 : RB;
    for (int i = threadIdx.x; i < rows * cols; i += 32 * WARPS) {
        const int n = i % cols, m = i / cols;
        if (n0 + n >= a.N) continue;
        float v = 0.f, up = 0.f;
#pragma unroll
        for (int k = 0; k < WARPS; ++k) v += red[k][n][m];
        if (gated) {
#pragma unroll
            for (int k = 0; k < WARPS; ++k) up += red[k][n + RB / 2][m];
        }
        if (a.rows && (unsigned)a.rows[first + m] >= (unsigned)a.X) v = up = 0.f;   // (a NaN weight would outlive the zeros)
        finish<TY>(a, g, first + m, n0 + n, v, up);
    }
}

template <int NT, int WARPS, int DEPTH>
cudaError_t launch_t(const MatmulArgs &a, dim3 grid, cudaStream_t s) {
    if (a.ybf16) matmul_rows_kernel<NT, WARPS, DEPTH, __nv_bfloat16><<<grid, 32 * WARPS, 0, s>>>(a);
    else matmul_rows_kernel<NT, WARPS, DEPTH, float><<<grid, 32 * WARPS, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Up to 16 places (us here, and by tiles): one by 7168 x 2048 6.4, 10.5, by 2048 x 7168 8.4, 18.6; 16 by them 8.4, 10.8 and
// 8.4, 18.6; 8 over 8 of 256 experts of 2 x 512 x 2048 10.4, 12.5; 16 over 14 of 32 of 2 x 2880 x 2880 55.5, 55.2; 16 over
// 16 of 128 of 1536 x 2048 20.5, 20.8.  Up to 32 of a single matrix that has too few tiles for the SMs: 32 by 2048 x 7168
// 12.4, 14.5, but by 7168 x 2048 14.5, 12.5.
bool matmul_few_rows(const MatmulArgs &a) {
    if (a.transposed) return false;
    const int wide = a.act == MOE_ACT_SWIGLU ? 2 * a.N : a.N;
    return a.M <= 16 || (a.M <= 32 && !a.offsets && wide <= 16 * num_sms());
}

cudaError_t launch_matmul_rows(const MatmulArgs &a, cudaStream_t s) {
    const bool two = !a.offsets && a.M > 8, four = !a.offsets && a.M > 16;   // more sets of 8 columns beside the first
    const int cols = a.act == MOE_ACT_SWIGLU ? RB / 2 : RB;
    const dim3 grid((unsigned)((a.N + cols - 1) / cols), (unsigned)(a.offsets ? a.M : 1));
    // 16 warps a block share deep sums where every block has an SM to itself (us with 16, 8 warps: one row by 2048 x 7168 8.4,
    // 10.5, by 512 x 8192 7.2, 10.7, by 2048 x 2048 4.1, 4.7; 16 rows by 2048 x 7168 8.9, 14.1; shallower: by 2048 x 1024
    // one row 3.1, 2.9, 16 rows 3.5, 3.9; more blocks than SMs: one row by 7168 x 2048 9.3, 7.1)
    const bool wide = a.K >= 2048 && (long long)grid.x * grid.y <= num_sms();
    if (four) return wide ? launch_t<4, 16, 2>(a, grid, s) : launch_t<4, 8, 2>(a, grid, s);
    if (two) return wide ? launch_t<2, 16, 2>(a, grid, s) : launch_t<2, 8, 2>(a, grid, s);
    return wide ? launch_t<1, 16, 4>(a, grid, s) : launch_t<1, 8, 4>(a, grid, s);
}

}  // namespace moe
