// moe_matmul.cu - products of bf16 rows with bf16 matrices, dense or grouped by
// expert, with bias, activation and residual in the epilogue (moe_matmul).
// A block of TB x TB threads takes TB places of a group by TB columns.
#include <cuda_bf16.h>

#include "moe_around.h"
#include "moe_launch.h"
#include "moe_matmul.cuh"

namespace moe {
namespace {

constexpr int TB = 32;

__global__ void __launch_bounds__(TB * TB) matmul_kernel(const MatmulArgs a) {
    __shared__ float xs[TB][TB + 1], ws[2][TB][TB + 1];
    __shared__ int s_g, s_first, s_end;
    const int tx = threadIdx.x % TB, ty = threadIdx.x / TB;
    if (threadIdx.x == 0) {
        int tile = blockIdx.y;   // numbered group by group
        s_g = -1;
        for (int g = 0; g < a.G; ++g) {
            const int lo = a.offsets ? a.offsets[g] : 0, hi = a.offsets ? a.offsets[g + 1] : a.M;
            if (hi < lo || lo < 0 || hi > a.M) atomicOr(a.status, MOE_DEV_BAD_ROW);
            const int first = min(max(lo, 0), a.M), end = min(max(hi, 0), a.M);
            const int tiles = (max(end - first, 0) + TB - 1) / TB;
            if (tile < tiles) {
                s_g = g;
                s_first = first + tile * TB;
                s_end = end;
                break;
            }
            tile -= tiles;
        }
    }
    __syncthreads();
    if (s_g < 0) return;
    const int g = s_g, place = s_first + ty, n0 = blockIdx.x * TB, n = n0 + tx;
    const bool gated = a.act == MOE_ACT_SWIGLU;
    const int wide = gated ? 2 * a.N : a.N;
    int row = place < s_end ? (a.rows ? a.rows[place] : place) : 0;
    const bool bad = (unsigned)row >= (unsigned)a.X;
    if (bad) {
        atomicOr(a.status, MOE_DEV_BAD_ROW);
        row = 0;
    }
    float acc[2] = {};
    for (int k0 = 0; k0 < a.K; k0 += TB) {
        xs[ty][tx] = k0 + tx < a.K && place < s_end ? __bfloat162float(a.x[(size_t)row * a.K + k0 + tx]) : 0.f;
        for (int h = 0; h < (gated ? 2 : 1); ++h) {
            if (a.transposed)
                ws[h][tx][ty] = k0 + ty < a.K && n < a.N ? __bfloat162float(a.w[((size_t)g * a.K + k0 + ty) * a.N + n]) : 0.f;
            else
                ws[h][ty][tx] = k0 + tx < a.K && n0 + ty < a.N
                                    ? __bfloat162float(a.w[((size_t)g * wide + h * a.N + n0 + ty) * a.K + k0 + tx])
                                    : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < TB; ++k) {
            acc[0] = fmaf(xs[ty][k], ws[0][tx][k], acc[0]);
            if (gated) acc[1] = fmaf(xs[ty][k], ws[1][tx][k], acc[1]);
        }
        __syncthreads();
    }
    if (place >= s_end || n >= a.N) return;
    if (bad) acc[0] = acc[1] = 0.f;
    finish(a, place, g, n, acc[0], acc[1]);
}

}  // namespace

cudaError_t launch_matmul(const MatmulArgs &a, cudaStream_t s) {
    const long long tiles = (long long)(a.M / TB) + (a.offsets ? (a.G < a.M ? a.G : a.M) : 1);
    if (tiles > 65535) return cudaErrorNotSupported;
    matmul_kernel<<<dim3((unsigned)((a.N + TB - 1) / TB), (unsigned)tiles), TB * TB, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
