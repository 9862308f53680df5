// moe_around.h - internal launcher declarations of the calls around the
// experts (moe_norm.cu, moe_router_stats.cu, moe_fp8.cu, moe_fp8_rows.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

cudaError_t launch_norm(const void *x, const void *residual, const float *weight, float eps, int T, int n, int dtype,
                        void *residual_out, void *y, int ydtype, uint8_t *xq, uint8_t *x8, float *x8_scale,
                        cudaStream_t s);

size_t order_ws_bytes(int T, int k, int E);
cudaError_t launch_order(const int32_t *ids, int T, int k, int E, int32_t *counts, int32_t *offsets, int32_t *rows,
                         int32_t *pos, void *ws, cudaStream_t s);

size_t balance_ws_bytes();
cudaError_t launch_balance(const void *logits, int dtype, const int32_t *counts, const uint8_t *valid, int T, int E,
                           int k, int gating, float alpha, const float *grad_loss, float *loss, void *dlogits,
                           void *ws, cudaStream_t s);

// moe_fp8_matmul: tiles through TMA and tcgen05 (moe_fp8.cu), or few rows (moe_fp8_rows.cu)
struct Fp8Args {
    const uint8_t *x, *w;
    const float *xs, *ws;
    const int32_t *rows, *offsets;
    void *y;
    unsigned *status;
    int X, M, G, N, K;
    int KB, NB;    // blocks of 128 in K and N
    int ntn;       // column tiles
    int xbox;      // rows of an x copy (ungathered)
    int yalign;    // bytes that rows of y are aligned to: 32, 16 or less
    // test hook: bound on waits in units of 2^16 cycles; arrivals that never come at a stage's copies, at its products
    uint32_t wait;
    int hold_copies, hold_products;
};
cudaError_t launch_fp8(const void *x8, const float *x_scale, int X, const int32_t *rows, int M, const int32_t *offsets,
                       int G, const void *w, const float *w_scale, int N, int K, void *y, int ydtype,
                       unsigned *status, cudaStream_t s);
void hold_fp8(int hold, long long cycles);   // moe_debug_hold_fp8_matmul
bool fp8_few_rows(const Fp8Args &a);
cudaError_t launch_fp8_rows(const Fp8Args &a, int ydtype, cudaStream_t s);

}  // namespace moe
