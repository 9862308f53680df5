// moe_api.cu - the C ABI declared in include/moe.h: argument validation and
// launches.  Every check happens before anything is enqueued.
#include <math.h>
#include <string.h>

#include <initializer_list>

#include "moe_around.h"
#include "moe_common.cuh"
#include "moe_launch.h"
#include "moe_matmul.cuh"

using namespace moe;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

bool dtype_ok(int d) { return d == MOE_DT_F32 || d == MOE_DT_BF16; }

bool expert_format(int q) {
    return q == MOE_Q8_0 || q == MOE_Q4_K || q == MOE_Q2_K || q == MOE_MXFP4 || q == MOE_Q6_K || q == MOE_Q3_K;
}

// columns a packed matrix of this format accepts
bool cols_ok(int q, int cols) {
    if (cols <= 0) return false;
    if (q == MOE_MXFP4) return cols % 32 == 0;
    return cols % 256 == 0;
}

size_t packed_bytes(int q, int rows, int cols) {
    if (rows <= 0 || rows % 32 || !expert_format(q) || !cols_ok(q, cols)) return 0;
    size_t tile;
    switch (q) {
        case MOE_Q4_K: tile = FQ4K::tile_bytes(cols); break;
        case MOE_Q2_K: tile = FQ2K::tile_bytes(cols); break;
        case MOE_Q8_0: tile = FQ80::tile_bytes(cols); break;
        case MOE_Q6_K: tile = FQ6K::tile_bytes(cols); break;
        case MOE_Q3_K: tile = FQ3K::tile_bytes(cols); break;
        default: tile = FMX4::tile_bytes(cols); break;
    }
    return (size_t)(rows / 32) * tile;
}

moe_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return MOE_OK;
    if (e == cudaErrorInvalidConfiguration || e == cudaErrorNotSupported) return MOE_ERR_UNSUPPORTED;
    return MOE_ERR_CUDA;
}

size_t route_ws(int T, int E, int H) {
    const int nseg = (H + 1023) / 1024;
    return 256 + (size_t)T * E * nseg * sizeof(float);
}

bool pool_ok(const moe_pool *p, bool shared) {
    if (!p || !p->experts || !expert_format(p->qtype)) return false;
    if (p->H <= 0 || p->I <= 0 || p->H % 32 || p->I % 32) return false;
    if (shared ? p->E != 1 : (p->E < 1 || p->E > MOE_MAX_EXPERTS)) return false;
    return true;
}

// formats whose records span 256 columns need 256-blocks of activations
bool pool_shape_ok(const moe_pool *p) {
    if (!cols_ok(p->qtype, p->H) || !cols_ok(p->qtype, p->I)) return false;
    return act_block(p->H) != 0 && act_block(p->I) != 0;
}

bool topk_ok(int T, int E, int k, int dtype, int gating) {
    if (T < 0 || T > MOE_MAX_ROWS || E < 1 || E > MOE_MAX_EXPERTS || k < 1 || k > E || k > MOE_MAX_K) return false;
    return dtype_ok(dtype) && (gating == MOE_GATE_SOFTMAX || gating == MOE_GATE_SIGMOID);
}

bool rows_ok(int T, int k, int n, int M) {
    if (T < 0 || T > MOE_MAX_ROWS || M < 0 || M > MOE_MAX_ROWS || k < 1 || k > MOE_MAX_K) return false;
    if (n < 1 || n > 65536 || (long long)T * k > MOE_MAX_PAIRS) return false;
    return (long long)T * n <= (1ll << 36) && (long long)M * n <= (1ll << 36);
}

}  // namespace

namespace moe {
moe_status ffn_check_args(const void *xq, int T, const int32_t *ids, const float *weights, int k,
                          const moe_pool *pool, const moe_pool *shared, const float *shared_scale, const float *y) {
    if (T < 0 || T > MOE_MAX_TOKENS || k < 1 || k > MOE_MAX_K) return MOE_ERR_INVALID_ARG;
    if (!pool_ok(pool, false)) return MOE_ERR_INVALID_ARG;
    if (shared && !pool_ok(shared, true)) return MOE_ERR_INVALID_ARG;
    if (!pool_shape_ok(pool)) return MOE_ERR_UNSUPPORTED;
    if (shared && (shared->H != pool->H || !pool_shape_ok(shared))) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!xq || !ids || !weights || !y || !aligned16(xq) || !aligned16(y)) return MOE_ERR_INVALID_ARG;
    if (shared_scale && !shared) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}
}  // namespace moe

extern "C" {

int moe_act_block(int n) { return act_block(n); }

size_t moe_q8_row_bytes(int n) { return q8_row_bytes(n); }

size_t moe_packed_bytes(moe_qtype qtype, int rows, int cols) { return packed_bytes(qtype, rows, cols); }

moe_status moe_pack_weights(const void *blocks, moe_qtype qtype, int rows, int cols, void *packed,
                            cudaStream_t stream) {
    if (!blocks || !packed) return MOE_ERR_INVALID_ARG;
    if (rows <= 0 || cols <= 0) return MOE_ERR_INVALID_ARG;
    if (packed_bytes(qtype, rows, cols) == 0) return MOE_ERR_UNSUPPORTED;
    if (!aligned16(packed)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_pack((const uint8_t *)blocks, qtype, rows, cols, (uint8_t *)packed, stream));
}

moe_status moe_quantize_q8K(const float *x, int T, int n, void *xq, cudaStream_t stream) {
    if (T < 0 || T > MOE_MAX_TOKENS * 64) return MOE_ERR_INVALID_ARG;
    if (!act_block(n)) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!x || !xq || !aligned16(x) || !aligned16(xq)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_quantize(x, T, n, (uint8_t *)xq, stream));
}

size_t moe_route_workspace_bytes(int T, int E, int H) {
    if (T <= 0 || E <= 0 || H <= 0) return 0;
    return route_ws(T, E, H);
}

moe_status moe_route(const float *hidden, const void *xq, int T, int H, const void *w_router, moe_qtype rtype,
                     int E, const float *router_bias, int k, moe_gating gating, int renormalize, int32_t *ids,
                     float *weights, float *logits_out, const float *shared_gate, float *shared_scale, void *ws,
                     size_t ws_bytes, cudaStream_t stream) {
    if (T < 0 || T > MOE_MAX_TOKENS || H <= 0 || H % 32 || E < 1 || E > MOE_MAX_EXPERTS) return MOE_ERR_INVALID_ARG;
    if (k < 1 || k > E || k > MOE_MAX_K) return MOE_ERR_INVALID_ARG;
    if (gating != MOE_GATE_SOFTMAX && gating != MOE_GATE_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (rtype != MOE_F32 && rtype != MOE_Q8_0) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!w_router || !ids || !weights) return MOE_ERR_INVALID_ARG;
    if (!aligned16(w_router)) return MOE_ERR_INVALID_ARG;
    if (rtype == MOE_F32 && (!hidden || !aligned16(hidden))) return MOE_ERR_INVALID_ARG;
    if (rtype == MOE_Q8_0) {
        if (H % 256) return MOE_ERR_UNSUPPORTED;
        if (!xq || !aligned16(xq)) return MOE_ERR_INVALID_ARG;
    }
    if ((shared_gate == nullptr) != (shared_scale == nullptr)) return MOE_ERR_INVALID_ARG;
    if (shared_gate && (!hidden || !aligned16(hidden) || !aligned16(shared_gate))) return MOE_ERR_INVALID_ARG;
    if (!ws || ws_bytes < route_ws(T, E, H) || !aligned16(ws)) return MOE_ERR_WORKSPACE;
    RouteArgs a;
    a.hidden = hidden;
    a.xq = (const uint8_t *)xq;
    a.w = w_router;
    a.bias = router_bias;
    a.ids = ids;
    a.weights = weights;
    a.logits_out = logits_out;
    a.counter = (unsigned *)ws;
    a.partial = (float *)((char *)ws + 256);
    a.T = T;
    a.H = H;
    a.E = E;
    a.k = k;
    a.nseg = (H + 1023) / 1024;
    a.gating = gating;
    a.renorm = renormalize ? 1 : 0;
    a.shared_gate = shared_gate;
    a.shared_scale = shared_scale;
    if (shared_gate) {
        const moe_status st = cuda_status(launch_shared_gate(hidden, T, H, shared_gate, shared_scale, stream));
        if (st != MOE_OK) return st;
    }
    return cuda_status(launch_route(a, rtype, stream));
}

size_t moe_ffn_workspace_bytes(int T, int k, const moe_pool *pool, const moe_pool *shared) {
    if (T < 0 || k < 1 || !pool) return 0;
    return ffn_ws_layout(T, k, pool->H, pool->I, shared ? shared->I : 0).total;
}

moe_status moe_expert_ffn(const void *xq, int T, const int32_t *ids, const float *weights, int k,
                          const moe_pool *pool, const moe_pool *shared, const float *shared_scale, float *y,
                          void *ws, size_t ws_bytes, cudaStream_t stream) {
    const moe_status v = moe::ffn_check_args(xq, T, ids, weights, k, pool, shared, shared_scale, y);
    if (v != MOE_OK || T == 0) return v;
    const FfnWs L = ffn_ws_layout(T, k, pool->H, pool->I, shared ? shared->I : 0);
    if (!ws || ws_bytes < L.total || !aligned16(ws)) return MOE_ERR_WORKSPACE;
    char *w = (char *)ws;
    FfnArgs a;
    a.xq = (const uint8_t *)xq;
    a.ids = ids;
    a.weights = weights;
    a.experts = pool->experts;
    a.shared = shared ? shared->experts : nullptr;
    a.shared_scale = shared_scale;
    a.y = y;
    a.status = (unsigned *)(w + L.status);
    a.counters = (unsigned *)(w + L.counters);
    a.h_r = (float *)(w + L.h_r);
    a.h_s = (float *)(w + L.h_s);
    a.hq_r = (uint8_t *)(w + L.hq_r);
    a.hq_s = (uint8_t *)(w + L.hq_s);
    a.T = T;
    a.k = k;
    a.H = pool->H;
    a.I = pool->I;
    a.Is = shared ? shared->I : 0;
    a.E = pool->E;
    a.qtype = pool->qtype;
    a.sqtype = shared ? shared->qtype : pool->qtype;
    return cuda_status(launch_ffn(a, stream));
}

moe_status moe_sum_partials(const float *parts, int R, size_t n, float *y, cudaStream_t stream) {
    if (R < 1 || R > MOE_MAX_RANKS || n % 4) return MOE_ERR_INVALID_ARG;
    if (n == 0) return MOE_OK;
    if (!parts || !y || !aligned16(parts) || !aligned16(y)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_sum_partials(parts, R, n, y, stream));
}

moe_status moe_add_rmsnorm(const void *x, const void *residual, const float *weight, float eps, int T, int n,
                           moe_dtype dtype, void *residual_out, void *y, moe_dtype ydtype, void *xq, void *x8,
                           float *x8_scale, cudaStream_t stream) {
    if (T < 0 || T > MOE_MAX_ROWS || !dtype_ok(dtype) || !dtype_ok(ydtype)) return MOE_ERR_INVALID_ARG;
    if (!(eps > 0.f) || isinf(eps)) return MOE_ERR_INVALID_ARG;
    if (n < 16 || n > MOE_MAX_NORM_WIDTH || n % 16 || (xq && !act_block(n))) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if ((x8 == nullptr) != (x8_scale == nullptr)) return MOE_ERR_INVALID_ARG;
    if (!residual_out && !y && !xq && !x8) return MOE_ERR_INVALID_ARG;
    if (!x || !weight) return MOE_ERR_INVALID_ARG;
    for (const void *p : {x, residual, (const void *)weight, (const void *)residual_out, (const void *)y,
                          (const void *)xq, (const void *)x8})
        if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
    if (!aligned4(x8_scale)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_norm(x, residual, weight, eps, T, n, dtype, residual_out, y, ydtype, (uint8_t *)xq,
                                   (uint8_t *)x8, x8_scale, stream));
}

size_t moe_expert_order_workspace_bytes(int T, int k, int E) {
    if (T <= 0 || k < 1 || E < 1) return 0;
    return order_ws_bytes(T, k, E);
}

moe_status moe_expert_order(const int32_t *ids, int T, int k, int E, int32_t *counts, int32_t *offsets,
                            int32_t *rows, int32_t *pos, void *ws, size_t ws_bytes, cudaStream_t stream) {
    if (T < 0 || T > MOE_MAX_ROWS || k < 1 || k > MOE_MAX_K || E < 1 || E > MOE_MAX_EXPERTS)
        return MOE_ERR_INVALID_ARG;
    if ((long long)T * k > MOE_MAX_PAIRS) return MOE_ERR_INVALID_ARG;
    if (!counts && !offsets && !rows && !pos) return T == 0 ? MOE_OK : MOE_ERR_INVALID_ARG;
    if (T > 0 && !ids) return MOE_ERR_INVALID_ARG;
    for (const void *p : {(const void *)ids, (const void *)counts, (const void *)offsets, (const void *)rows,
                          (const void *)pos})
        if (!aligned4(p)) return MOE_ERR_INVALID_ARG;
    const size_t need = moe_expert_order_workspace_bytes(T, k, E);
    if (need && (!ws || ws_bytes < need || !aligned16(ws))) return MOE_ERR_WORKSPACE;
    return cuda_status(launch_order(ids, T, k, E, counts, offsets, rows, pos, ws, stream));
}

size_t moe_balance_loss_workspace_bytes(int T, int E) {
    if (T < 0 || E < 1) return 0;
    return balance_ws_bytes();
}

moe_status moe_balance_loss(const void *logits, moe_dtype dtype, const int32_t *counts, const uint8_t *valid, int T,
                            int E, int k, moe_gating gating, float alpha, const float *grad_loss, float *loss,
                            void *dlogits, void *ws, size_t ws_bytes, cudaStream_t stream) {
    if (T < 0 || T > MOE_MAX_ROWS || E < 1 || E > MOE_MAX_EXPERTS || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
    if (k < 1 || k > E || k > MOE_MAX_K) return MOE_ERR_INVALID_ARG;
    if (gating != MOE_GATE_SOFTMAX && gating != MOE_GATE_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (!counts || !aligned4(counts) || !aligned4(grad_loss) || !aligned4(loss)) return MOE_ERR_INVALID_ARG;
    if (!loss && !dlogits) return T == 0 ? MOE_OK : MOE_ERR_INVALID_ARG;
    if (T > 0 && !logits) return MOE_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned16(dlogits)) return MOE_ERR_INVALID_ARG;
    if (!ws || ws_bytes < balance_ws_bytes() || !aligned16(ws)) return MOE_ERR_WORKSPACE;
    return cuda_status(launch_balance(logits, dtype, counts, valid, T, E, k, gating, alpha, grad_loss, loss, dlogits,
                                      ws, stream));
}

size_t moe_fp8_matmul_workspace_bytes(void) { return 256; }

moe_status moe_fp8_matmul(const void *x8, const float *x_scale, int X, const int32_t *rows, int M,
                          const int32_t *offsets, int G, const void *w, const float *w_scale, int N, int K,
                          void *y, moe_dtype ydtype, void *ws, size_t ws_bytes, cudaStream_t stream) {
    if (X < 0 || X > MOE_MAX_ROWS || M < 0 || M > MOE_MAX_ROWS || G < 1 || G > MOE_MAX_EXPERTS)
        return MOE_ERR_INVALID_ARG;
    if (N < 1 || N > (1 << 20) || (long long)G * N > (1ll << 30) || !dtype_ok(ydtype)) return MOE_ERR_INVALID_ARG;
    if (K < 16 || K > (1 << 20) || K % 16) return MOE_ERR_UNSUPPORTED;
    if ((long long)X * K > (1ll << 36)) return MOE_ERR_INVALID_ARG;
    if (!offsets && G != 1) return MOE_ERR_INVALID_ARG;
    if (M == 0) return MOE_OK;
    if (X == 0 || (!rows && X < M)) return MOE_ERR_INVALID_ARG;
    if (!x8 || !x_scale || !w || !w_scale || !y) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x8) || !aligned16(w) || !aligned16(y)) return MOE_ERR_INVALID_ARG;
    if (!aligned4(x_scale) || !aligned4(w_scale) || !aligned4(rows) || !aligned4(offsets)) return MOE_ERR_INVALID_ARG;
    if (!ws || ws_bytes < moe_fp8_matmul_workspace_bytes() || !aligned16(ws)) return MOE_ERR_WORKSPACE;
    return cuda_status(launch_fp8(x8, x_scale, X, rows, M, offsets, G, w, w_scale, N, K, y, ydtype, (unsigned *)ws,
                                  stream));
}

moe_status moe_topk(const void *logits, moe_dtype dtype, const uint8_t *valid, int T, int E, int k, moe_gating gating,
                    int renormalize, int32_t *ids, float *weights, cudaStream_t stream) {
    if (!topk_ok(T, E, k, dtype, gating)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!logits || !aligned16(logits) || !ids || !aligned4(ids) || !aligned4(weights)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_topk(logits, dtype, valid, T, E, k, gating, renormalize, ids, weights, stream));
}

moe_status moe_topk_grad(const void *logits, moe_dtype dtype, const int32_t *ids, const float *dweights, int T, int E,
                         int k, moe_gating gating, int renormalize, const void *addend, void *dlogits,
                         cudaStream_t stream) {
    if (!topk_ok(T, E, k, dtype, gating)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!logits || !ids || !dweights || !dlogits) return MOE_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned16(addend) || !aligned16(dlogits)) return MOE_ERR_INVALID_ARG;
    if (!aligned4(ids) || !aligned4(dweights)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_topk_grad(logits, dtype, ids, dweights, T, E, k, gating, renormalize, addend, dlogits,
                                        stream));
}

moe_status moe_dispatch_rows(const void *x, moe_dtype dtype, const int32_t *pos, int T, int k, int n, int M, void *xs,
                             cudaStream_t stream) {
    if (!rows_ok(T, k, n, M) || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
    if (T == 0 || M == 0) return MOE_OK;
    if (!x || !pos || !xs || !aligned16(x) || !aligned4(pos) || !aligned16(xs)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_dispatch_rows(x, dtype, pos, T, k, n, M, xs, stream));
}

moe_status moe_combine_rows(const void *o, moe_dtype dtype, const int32_t *pos, const float *weights, int T, int k,
                            int n, int M, const void *addend, void *y, moe_dtype ydtype, cudaStream_t stream) {
    if (!rows_ok(T, k, n, M) || !dtype_ok(dtype) || !dtype_ok(ydtype)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if ((!o && M > 0) || !pos || !y) return MOE_ERR_INVALID_ARG;
    if (!aligned16(o) || !aligned16(addend) || !aligned16(y)) return MOE_ERR_INVALID_ARG;
    if (!aligned4(pos) || !aligned4(weights)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_combine_rows(o, dtype, pos, weights, T, k, n, M, addend, y, ydtype, stream));
}

moe_status moe_combine_grad(const void *dy, moe_dtype ydtype, const int32_t *pos, const float *weights, int T, int k,
                            int n, int M, const void *o, moe_dtype dtype, void *d_o, float *dweights,
                            cudaStream_t stream) {
    if (!rows_ok(T, k, n, M) || !dtype_ok(dtype) || !dtype_ok(ydtype)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!d_o && !dweights) return M == 0 ? MOE_OK : MOE_ERR_INVALID_ARG;
    if (!dy || !pos || (dweights && !o && M > 0)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(o) || !aligned16(d_o)) return MOE_ERR_INVALID_ARG;
    if (!aligned4(pos) || !aligned4(weights) || !aligned4(dweights)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_combine_grad(dy, ydtype, pos, weights, T, k, n, M, o, dtype, d_o, dweights, stream));
}

size_t moe_matmul_workspace_bytes(void) { return 256; }

moe_status moe_matmul(const void *x, int X, const int32_t *rows, int M, const int32_t *offsets, int G, const void *w,
                      int transposed, const float *bias, moe_act act, const void *residual, void *z, int N, int K,
                      void *y, moe_dtype ydtype, void *ws, size_t ws_bytes, cudaStream_t stream) {
    if (X < 0 || X > MOE_MAX_ROWS || M < 0 || M > MOE_MAX_ROWS || G < 1 || G > MOE_MAX_EXPERTS)
        return MOE_ERR_INVALID_ARG;
    if (act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU_GRAD || !dtype_ok(ydtype)) return MOE_ERR_INVALID_ARG;
    if (N < 1 || N > (1 << 20) || (long long)G * N > (1ll << 30)) return MOE_ERR_INVALID_ARG;
    if (K < 8 || K > (1 << 20) || K % 8 || (transposed && N % 8)) return MOE_ERR_UNSUPPORTED;
    if (act == MOE_ACT_SWIGLU && (transposed || N % 16)) return MOE_ERR_UNSUPPORTED;
    if ((long long)X * K > (1ll << 35)) return MOE_ERR_INVALID_ARG;
    if (!offsets && G != 1) return MOE_ERR_INVALID_ARG;
    const bool grad = act >= MOE_ACT_SILU_GRAD;
    if (grad ? bias || residual : act == MOE_ACT_NONE && z != nullptr) return MOE_ERR_INVALID_ARG;
    if (M == 0) return MOE_OK;
    if (X == 0 || (!rows && X < M)) return MOE_ERR_INVALID_ARG;
    if (!x || !w || !y || (grad && !z)) return MOE_ERR_INVALID_ARG;
    for (const void *p : {x, w, residual, (const void *)z, (const void *)y})
        if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
    if (!aligned4(bias) || !aligned4(rows) || !aligned4(offsets)) return MOE_ERR_INVALID_ARG;
    if (!ws || ws_bytes < moe_matmul_workspace_bytes() || !aligned16(ws)) return MOE_ERR_WORKSPACE;
    MatmulArgs a = {};
    a.x = (const __nv_bfloat16 *)x;
    a.w = (const __nv_bfloat16 *)w;
    a.bias = bias;
    a.rows = rows;
    a.offsets = offsets;
    a.residual = residual;
    a.z = z;
    a.y = y;
    a.status = (unsigned *)ws;
    a.X = X;
    a.M = M;
    a.G = G;
    a.N = N;
    a.K = K;
    a.act = act;
    a.transposed = transposed != 0;
    a.ybf16 = ydtype == MOE_DT_BF16;
    return cuda_status(launch_matmul(a, stream));
}

moe_status moe_debug_hold_fp8_matmul(int hold, long long cycles) {
    if (hold < 0 || hold > 2 || cycles < 0) return MOE_ERR_INVALID_ARG;
    hold_fp8(hold, cycles);
    return MOE_OK;
}

moe_status moe_debug_hold_matmul(int hold, long long cycles) {
    if (hold < 0 || hold > 2 || cycles < 0) return MOE_ERR_INVALID_ARG;
    hold_matmul(hold, cycles);
    return MOE_OK;
}

moe_status moe_read_device_status(void *ws, int clear, uint32_t *flags, cudaStream_t stream) {
    if (!ws || !flags) return MOE_ERR_INVALID_ARG;
    uint32_t v = 0;
    if (cudaMemcpyAsync(&v, ws, sizeof v, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return MOE_ERR_CUDA;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return MOE_ERR_CUDA;
    if (clear && v) {
        if (cudaMemsetAsync(ws, 0, sizeof v, stream) != cudaSuccess) return MOE_ERR_CUDA;
        if (cudaStreamSynchronize(stream) != cudaSuccess) return MOE_ERR_CUDA;
    }
    *flags = v;
    return v ? MOE_ERR_DEVICE_STATUS : MOE_OK;
}

moe_status moe_debug_row_dots(const void *packed, moe_qtype qtype, int rows, int cols, int row, const void *xq,
                              int32_t *isums, cudaStream_t stream) {
    if (!packed || !xq || !isums) return MOE_ERR_INVALID_ARG;
    if (packed_bytes(qtype, rows, cols) == 0) return MOE_ERR_UNSUPPORTED;
    if (row < 0 || row >= rows) return MOE_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(packed)) return MOE_ERR_INVALID_ARG;
    if (qtype != MOE_MXFP4 && act_block(cols) != 256) return MOE_ERR_UNSUPPORTED;
    return cuda_status(launch_row_dots((const uint8_t *)packed, qtype, cols, row, (const uint8_t *)xq, isums,
                                       stream));
}

const char *moe_status_str(moe_status s) {
    switch (s) {
        case MOE_OK: return "ok";
        case MOE_ERR_INVALID_ARG: return "invalid argument";
        case MOE_ERR_UNSUPPORTED: return "unsupported format or shape";
        case MOE_ERR_WORKSPACE: return "workspace missing or too small";
        case MOE_ERR_CUDA: return "CUDA error";
        case MOE_ERR_DEVICE_STATUS: return "device reported a data error";
        case MOE_ERR_TIMEOUT: return "device wait timed out";
    }
    return "unknown status";
}

}  // extern "C"
