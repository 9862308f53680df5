// moe_fp8_rows.cu - moe_fp8_matmul for few rows: decode of one token to a few.
//
// The weights are read once and bound the call, so nothing is staged: a warp
// loads 16 matrix rows of a 128-deep block straight into the registers of its
// matrix instructions (m16n8k32, weights as the 16 rows, tokens as the 8
// columns).  A lane's 16-byte pieces of a matrix row and of an x row hold the
// same depths, and a sum does not mind the order of its terms, so the pieces
// serve as fragments as they are: registers 0, 1 for one instruction, 2, 3 for
// the next.  Depth blocks are dealt to the warps of a block, each scaled as it
// is done (sx * sw, fp32), and the warps' sums are added in warp order.
//
// A block takes 16 columns of y for a chunk of up to 8 NT places of one group;
// chunks start at a group's first place.  Against the tiles of moe_fp8.cu this
// saves the tensor maps, the ring's start and the cluster's exchange.
#include <cuda_bf16.h>

#include "moe_around.h"
#include "moe_common.cuh"
#include "moe_launch.h"

namespace moe {
namespace {

constexpr int RB = 16;   // matrix rows of a block

__device__ __forceinline__ void mma16832(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 16 bytes of a weight row, read once
__device__ __forceinline__ uint4 ld_weight(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <int NT, int WARPS, typename TY>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 8 ? 3 : 1) fp8_rows_kernel(const Fp8Args a) {
    constexpr int CHUNK = 8 * NT, DEPTH = NT == 1 ? 2 : 1;   // places of a block; depth blocks a warp has on their way
    __shared__ float red[WARPS][RB][CHUNK + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g8 = lane >> 2, t4 = lane & 3;
    int g = 0, first = blockIdx.y * CHUNK, end = a.M;
    if (a.offsets) {
        // the group of place blockIdx.y: the last one that does not start after it; every warp looks for itself
        const int place = blockIdx.y;
        int n = 0;
        for (int i = lane; i <= a.G; i += 32) {
            const int o = a.offsets[i];
            n += o <= place;
            if (blockIdx.x == 0 && blockIdx.y == 0 && warp == 0) {
                const int before = i ? a.offsets[i - 1] : 0;
                if (o < before || o > a.M) atomicOr(a.status, MOE_DEV_BAD_ROW);
            }
        }
        n = __reduce_add_sync(0xFFFFFFFFu, n);
        if (n < 1 || n > a.G) return;
        g = n - 1;
        const int start = max(a.offsets[g], 0);
        end = min(a.offsets[g + 1], a.M);
        if (place < start || place >= end || (place - start) % CHUNK) return;
        first = place;
    }
    const int rows = min(CHUNK, end - first), n0 = blockIdx.x * RB;
    // x rows of this lane's columns: as a product's operand (column g8), and of its sums (columns 2 t4, 2 t4 + 1).
    // Columns past the chunk, rows past N and bad indexes read something that is there; nothing of it is stored.
    const uint8_t *x[NT];
    const float *xs[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const auto row_of = [&](int m) {
            int r = first + (m < rows ? m : 0);
            if (a.rows) r = a.rows[r];
            if ((unsigned)r >= (unsigned)a.X) {
                atomicOr(a.status, MOE_DEV_BAD_ROW);
                r = 0;
            }
            return (size_t)r;
        };
        x[j] = a.x + row_of(8 * j + g8) * a.K;
#pragma unroll
        for (int h = 0; h < 2; ++h) xs[j][h] = a.xs + row_of(8 * j + 2 * t4 + h) * a.KB;
    }
    const float *ws = a.ws + ((size_t)g * a.NB + n0 / 128) * a.KB;
    const uint8_t *w0 = a.w + ((size_t)g * a.N + min(n0 + g8, a.N - 1)) * a.K;
    const uint8_t *w1 = a.w + ((size_t)g * a.N + min(n0 + g8 + 8, a.N - 1)) * a.K;
    float acc[NT][4] = {};
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int kb0 = warp; kb0 < a.KB; kb0 += DEPTH * WARPS) {
        // everything of DEPTH blocks on its way before the first product; past K and KB: zeros
        uint4 wa[DEPTH][2], wb[DEPTH][2], xb[DEPTH][NT][2];
        float sw[DEPTH], sx[DEPTH][NT][2];
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
            const int kb = min(kb0 + i * WARPS, a.KB - 1);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int k = (kb0 + i * WARPS) * 128 + 64 * p + 16 * t4;
                wa[i][p] = k < a.K ? ld_weight(w0 + k) : zero;
                wb[i][p] = k < a.K ? ld_weight(w1 + k) : zero;
#pragma unroll
                for (int j = 0; j < NT; ++j) xb[i][j][p] = k < a.K ? *reinterpret_cast<const uint4 *>(x[j] + k) : zero;
            }
            sw[i] = ws[kb];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                sx[i][j][0] = xs[j][0][kb];
                sx[i][j][1] = xs[j][1][kb];
            }
        }
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
            if (kb0 + i * WARPS >= a.KB) break;   // uniform over the warp
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float d[4] = {};
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const uint4 b = xb[i][j][p];
                    mma16832(d, wa[i][p].x, wb[i][p].x, wa[i][p].y, wb[i][p].y, b.x, b.y);
                    mma16832(d, wa[i][p].z, wb[i][p].z, wa[i][p].w, wb[i][p].w, b.z, b.w);
                }
                const float s0 = sx[i][j][0] * sw[i], s1 = sx[i][j][1] * sw[i];
                acc[j][0] = fmaf(d[0], s0, acc[j][0]);
                acc[j][1] = fmaf(d[1], s1, acc[j][1]);
                acc[j][2] = fmaf(d[2], s0, acc[j][2]);
                acc[j][3] = fmaf(d[3], s1, acc[j][3]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[warp][g8 + 8 * (i >> 1)][8 * j + 2 * t4 + (i & 1)] = acc[j][i];
    __syncthreads();
    for (int i = threadIdx.x; i < rows * RB; i += 32 * WARPS) {
        const int n = i % RB, m = i / RB;
        if (n0 + n >= a.N) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += red[w][n][m];
        if (a.rows && (unsigned)a.rows[first + m] >= (unsigned)a.X) v = 0.f;   // (a NaN weight would outlive the zeros)
        static_cast<TY *>(a.y)[(size_t)(first + m) * a.N + n0 + n] = (TY)v;
    }
}

template <int NT, int WARPS>
cudaError_t launch_t(const Fp8Args &a, int ydtype, dim3 grid, cudaStream_t s) {
    if (ydtype == MOE_DT_BF16) fp8_rows_kernel<NT, WARPS, __nv_bfloat16><<<grid, 32 * WARPS, 0, s>>>(a);
    else fp8_rows_kernel<NT, WARPS, float><<<grid, 32 * WARPS, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Up to 16 places: one matrix of 2048 x 7168 takes 4.6 us for one row and 6.6 for 16 where tiles take 11.8 and 12.4
// (7168 x 2048: 4.4 and 5.6 against 8.2 and 8.5); experts of 1536 x 4096, 8 rows over 8 of them: 14.9 against 14.9, 16
// over 16: 23.7 against 27.5; of 512 x 2048, 8 over 8: 5.2 against 8.0; but of 4096 x 1536: 17.0 against 14.8.  At 24
// rows and more a second reading of the weights brings them level (one matrix: 8.4 against 7.5) and, over many experts,
// short blocks fall behind the tiles' queues of copies (64 rows over 48 experts of 1536 x 4096: 61 against 52).
bool fp8_few_rows(const Fp8Args &a) {
    return a.M <= 16;
}

cudaError_t launch_fp8_rows(const Fp8Args &a, int ydtype, cudaStream_t s) {
    const bool two = !a.offsets && a.M > 8;   // a second set of 8 columns beside the first
    const dim3 grid((unsigned)((a.N + RB - 1) / RB), (unsigned)(a.offsets ? a.M : 1));
    // one block an SM or fewer, and two blocks of depth for each warp: sixteen warps to a block (2048 x 7168, one row:
    // 5.4 us, with eight 7.4); more: eight, so that blocks share an SM (7168 x 2048: 5.0, with sixteen 7.4; 8 rows over 8
    // experts of 4096 x 1536: 15.8, 31.4)
    const bool wide = a.KB >= 32 && (long long)grid.x * grid.y <= num_sms();
    if (two) return wide ? launch_t<2, 16>(a, ydtype, grid, s) : launch_t<2, 8>(a, ydtype, grid, s);
    return wide ? launch_t<1, 16>(a, ydtype, grid, s) : launch_t<1, 8>(a, ydtype, grid, s);
}

}  // namespace moe
