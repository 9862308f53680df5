// moe_norm.cu - residual addition, RMS norm and 8-bit rows (moe_add_rmsnorm).
//
//   s = x + residual,  v = s / sqrt(mean(s^2) + eps) * weight,
//   q8 records of v (the library's rule) and / or e4m3 codes with a scale for
//   each 128 values.
//
// One pass over the data: a block holds its row in registers between the sum
// of squares and the scaling, so x and the residual are read once and each
// output is written once.  A lane holds 8 consecutive values per chunk and a
// warp 256 of them, which is one q8 block (quant_store8's layout) and two
// e4m3 groups: their maxima are taken among 32 and 16 lanes, without shared
// memory.  Bandwidth bounds it for many rows, latency for few.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "moe_around.h"
#include "moe_common.cuh"
#include "moe_launch.h"

namespace moe {
namespace {

template <typename T>
__device__ __forceinline__ void load8(const T *p, float v[8]);
template <>
__device__ __forceinline__ void load8<float>(const float *p, float v[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float v[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float v[8]);
template <>
__device__ __forceinline__ void store8<float>(float *p, const float v[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16 *p, const float v[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// smallest maximum whose inverse 448/amax is finite with room to spare
constexpr float kFp8MinAmax = 0x1p-119f;

// (a NaN is the larger one)
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// e4m3 codes of a lane's 8 values, the scale shared by its 16 lanes.  A NaN stays one in the scale and its codes.
__device__ __forceinline__ void fp8_store8(const float v[8], bool active, int e0, uint8_t *row, float *scale,
                                           int lane) {
    float am = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) am = max_nan(am, fabsf(v[i]));
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, off));
    float d = 0.f, inv = 0.f;
    if (!(am < kFp8MinAmax)) {
        d = __fdiv_rn(am, 448.f);
        inv = __fdiv_rn(448.f, am);
    }
    if (!active) return;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<uint2 *>(row + e0) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    if ((lane & 15) == 0) scale[e0 >> 7] = d;
}

struct NormArgs {
    const void *x, *residual;
    const float *weight;
    void *residual_out, *y;
    uint8_t *xq, *x8;
    float *x8_scale;
    float eps, inv_n;
    int n, nscale;
    size_t xq_row;
};

// Sums over a warp of VPT chunks' numbers at once: number j ends up in the lanes from 32 / VPT * j on.  Where there are
// several, half of the lanes go on with each half of them.  Each is added by the same tree (lanes 16, 8, 4, 2, 1 apart)
// whatever VPT, so a chunk's sum has the same bits in every layout.
template <int VPT>
__device__ __forceinline__ float chunk_sums(const float s[VPT], int lane) {
    float v;
    if constexpr (VPT == 1) {
        v = s[0] + __shfl_xor_sync(0xFFFFFFFFu, s[0], 16);
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
    } else if constexpr (VPT == 2) {
        const bool up = lane & 16;
        v = (up ? s[1] : s[0]) + __shfl_xor_sync(0xFFFFFFFFu, up ? s[0] : s[1], 16);
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
    } else {
        static_assert(VPT == 4, "");
        const bool up = lane & 16, odd = lane & 8;
        const float a = (up ? s[2] : s[0]) + __shfl_xor_sync(0xFFFFFFFFu, up ? s[0] : s[2], 16);
        const float b = (up ? s[3] : s[1]) + __shfl_xor_sync(0xFFFFFFFFu, up ? s[1] : s[3], 16);
        v = (odd ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 8);
    }
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

constexpr int kMaxChunks = MOE_MAX_NORM_WIDTH / 256;

// One row per block.  Warp w takes the 256-value chunks w, w + W, ...: at most
// VPT of them.  The squares of each chunk are added by themselves, then the
// chunks in their order, so a row's bits do not hang on its layout and with it
// on the number of rows.  x and residual are read through plain loads: residual_out may
// be either of them, and a thread writes only where it has read.
template <typename TX, typename TY, int VPT>
__global__ void __launch_bounds__(VPT == 4 ? 512 : 1024) norm_kernel(const NormArgs a) {
    __shared__ float part[kMaxChunks];   // a chunk's sum of squares
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5, n = a.n;
    const size_t at = (size_t)blockIdx.x * n;
    const TX *x = static_cast<const TX *>(a.x) + at;
    const TX *r = a.residual ? static_cast<const TX *>(a.residual) + at : nullptr;
    float s[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int e0 = 256 * (warp + j * W) + 8 * lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j][i] = 0.f;
        if (e0 < n) load8<TX>(x + e0, s[j]);
    }
    if (r) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int e0 = 256 * (warp + j * W) + 8 * lane;
            if (e0 < n) {
                float b[8];
                load8<TX>(r + e0, b);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[j][i] += b[i];
            }
        }
    }
    float sq[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        sq[j] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sq[j] = fmaf(s[j][i], s[j][i], sq[j]);
    }
    constexpr int PER = 32 / VPT;   // lanes that hold a chunk's sum
    const float sum = chunk_sums<VPT>(sq, lane);
    if (lane % PER == 0) part[warp + lane / PER * W] = sum;
    if (a.residual_out) {
        TX *out = static_cast<TX *>(a.residual_out) + at;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int e0 = 256 * (warp + j * W) + 8 * lane;
            if (e0 < n) store8<TX>(out + e0, s[j]);
        }
    }
    __syncthreads();
    const int parts = VPT * W;   // past the row's last chunk: zeros
    float ss = lane < parts ? part[lane] : 0.f;
    if (VPT > 1 && lane + 32 < parts) ss += part[lane + 32];
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
    const float rstd = __fdiv_rn(1.f, __fsqrt_rn(fmaf(ss, a.inv_n, a.eps)));
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c0 = 256 * (warp + j * W), e0 = c0 + 8 * lane;
        if (c0 >= n) break;   // uniform over the warp
        const bool active = e0 < n;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
        if (active) load8<float>(a.weight + e0, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (s[j][i] * rstd) * v[i];
        if (a.y && active) store8<TY>(static_cast<TY *>(a.y) + at + e0, v);
        if (a.x8) fp8_store8(v, active, e0, a.x8 + at, a.x8_scale + (size_t)blockIdx.x * a.nscale, lane);
        if (a.xq) quant_store8(v, active, n, c0, a.xq + (size_t)blockIdx.x * a.xq_row, lane);
    }
}

template <typename TX, typename TY>
cudaError_t launch_norm_t(const NormArgs &a, int T, cudaStream_t s) {
    const int chunks = (a.n + 255) / 256;
    // A row an SM or fewer: one chunk a warp (two past 8192), so that a row's loads are all in flight at once over as
    // many warps as it has chunks: 16 x 7168 bf16 3.1 us, with two a warp 3.4.  More rows: up to 16 chunks one a warp as
    // well (fp32 out, 16384 x 4096: 113 us, with two 122, with four 110; 32768 x 2880: 158, 166, 153), and four a warp
    // beyond, so that several rows share an SM and one loads while another waits at its sum: 8192 x 7168 fp32 out 99.1 us,
    // with two 122, with one 117.
    const bool few = T <= num_sms();
    if (chunks <= (few ? 32 : 16)) norm_kernel<TX, TY, 1><<<T, 32 * chunks, 0, s>>>(a);
    else if (few) norm_kernel<TX, TY, 2><<<T, 32 * ((chunks + 1) / 2), 0, s>>>(a);
    else norm_kernel<TX, TY, 4><<<T, 32 * ((chunks + 3) / 4), 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(const void *x, const void *residual, const float *weight, float eps, int T, int n, int dtype,
                        void *residual_out, void *y, int ydtype, uint8_t *xq, uint8_t *x8, float *x8_scale,
                        cudaStream_t s) {
    NormArgs a;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.residual_out = residual_out;
    a.y = y;
    a.xq = xq;
    a.x8 = x8;
    a.x8_scale = x8_scale;
    a.eps = eps;
    a.inv_n = 1.f / (float)n;
    a.n = n;
    a.nscale = (n + MOE_FP8_GROUP - 1) / MOE_FP8_GROUP;
    a.xq_row = xq ? q8_row_bytes(n) : 0;
    if (dtype == MOE_DT_BF16)
        return ydtype == MOE_DT_BF16 ? launch_norm_t<__nv_bfloat16, __nv_bfloat16>(a, T, s)
                                     : launch_norm_t<__nv_bfloat16, float>(a, T, s);
    return ydtype == MOE_DT_BF16 ? launch_norm_t<float, __nv_bfloat16>(a, T, s)
                                 : launch_norm_t<float, float>(a, T, s);
}

}  // namespace moe
