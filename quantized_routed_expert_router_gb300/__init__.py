"""Python binding of the GB300 quantized routed-expert MoE FFN library.

Argument marshalling only: every step of the path runs in the CUDA library
``_moe.so`` (C ABI, ``include/moe.h``); this module passes tensor addresses,
sizes and the current CUDA stream through ctypes (the calls around the experts:
through ``_calls.so``, a compiled binding of the same ABI).  PyTorch supplies device
memory and streams.  Importing works without a GPU; the library must have
been built (``_build.build()``) - there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _build

F32, Q8_0, Q4_K, Q2_K, MXFP4, Q6_K, Q3_K = 0, 1, 2, 3, 4, 5, 6
SOFTMAX, SIGMOID = 0, 1
DEV_BAD_ID, DEV_DUP_ID = 0x1, 0x2
MAX_TOKENS, MAX_K, MAX_EXPERTS = 16, 32, 1024

EXPORTS = ["moe_act_block", "moe_q8_row_bytes", "moe_packed_bytes", "moe_pack_weights", "moe_quantize_q8K",
           "moe_route", "moe_route_workspace_bytes", "moe_expert_ffn", "moe_ffn_workspace_bytes",
           "moe_read_device_status", "moe_debug_row_dots", "moe_status_str", "moe_expert_ffn_noalloc",
           "moe_layer_forward", "moe_layer_workspace_bytes", "moe_sum_partials", "moe_debug_set_exchange_wait",
           "moe_add_rmsnorm", "moe_expert_order", "moe_expert_order_workspace_bytes", "moe_balance_loss",
           "moe_balance_loss_workspace_bytes", "moe_fp8_matmul", "moe_fp8_matmul_workspace_bytes",
           "moe_debug_hold_fp8_matmul", "moe_topk", "moe_topk_grad", "moe_dispatch_rows", "moe_combine_rows",
           "moe_combine_grad", "moe_matmul", "moe_matmul_workspace_bytes",
           "moe_debug_hold_matmul"]
LAYER_OVERLAP_PREVIOUS = 0x1
DEV_TIMEOUT, DEV_BAD_ROW = 0x4, 0x8
DT_F32, DT_BF16 = 0, 1
ACT_NONE, ACT_SILU, ACT_GELU, ACT_SWIGLU, ACT_SILU_GRAD, ACT_GELU_GRAD, ACT_SWIGLU_GRAD = range(7)
FP8_GROUP = 128          # values that share a scale of an e4m3 row

_P = ctypes.c_void_p
_lib_handle = None


class MoeError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call}: {status_str(status)} (status {status})")


class _Expert(ctypes.Structure):
    _fields_ = [("gate", _P), ("up", _P), ("down", _P), ("b_gate", _P), ("b_up", _P), ("b_down", _P)]


class _Pool(ctypes.Structure):
    _fields_ = [("qtype", ctypes.c_int), ("H", ctypes.c_int), ("I", ctypes.c_int), ("E", ctypes.c_int),
                ("experts", _P)]


def library_path() -> str:
    return _build.SO


def lib():
    """The loaded C library.  Raises if it has not been built."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(_build.SO):
            raise RuntimeError(f"CUDA library not built: {_build.SO} is missing (run __graft_entry__.build())")
        L = ctypes.CDLL(_build.SO)
        i, sz = ctypes.c_int, ctypes.c_size_t
        L.moe_act_block.restype = i
        L.moe_act_block.argtypes = [i]
        L.moe_q8_row_bytes.restype = sz
        L.moe_q8_row_bytes.argtypes = [i]
        L.moe_packed_bytes.restype = sz
        L.moe_packed_bytes.argtypes = [i, i, i]
        L.moe_pack_weights.restype = i
        L.moe_pack_weights.argtypes = [_P, i, i, i, _P, _P]
        L.moe_quantize_q8K.restype = i
        L.moe_quantize_q8K.argtypes = [_P, i, i, _P, _P]
        L.moe_route.restype = i
        L.moe_route.argtypes = [_P, _P, i, i, _P, i, i, _P, i, i, i, _P, _P, _P, _P, _P, _P, sz, _P]
        L.moe_route_workspace_bytes.restype = sz
        L.moe_route_workspace_bytes.argtypes = [i, i, i]
        L.moe_expert_ffn.restype = i
        L.moe_expert_ffn.argtypes = [_P, i, _P, _P, i, ctypes.POINTER(_Pool), ctypes.POINTER(_Pool), _P, _P, _P, sz,
                                     _P]
        L.moe_expert_ffn_noalloc.restype = i
        L.moe_expert_ffn_noalloc.argtypes = [_P, i, _P, _P, i, ctypes.POINTER(_Pool), ctypes.POINTER(_Pool), _P, _P,
                                             _P]
        L.moe_layer_forward.restype = i
        L.moe_layer_forward.argtypes = [_P, i, _P, i, _P, i, i, i, ctypes.POINTER(_Pool), ctypes.POINTER(_Pool),
                                        _P, _P, _P, _P, _P, _P, _P, sz, ctypes.c_uint, _P]
        L.moe_layer_workspace_bytes.restype = sz
        L.moe_layer_workspace_bytes.argtypes = [i, i, ctypes.POINTER(_Pool), ctypes.POINTER(_Pool)]
        L.moe_ffn_workspace_bytes.restype = sz
        L.moe_ffn_workspace_bytes.argtypes = [i, i, ctypes.POINTER(_Pool), ctypes.POINTER(_Pool)]
        L.moe_read_device_status.restype = i
        L.moe_read_device_status.argtypes = [_P, i, ctypes.POINTER(ctypes.c_uint32), _P]
        L.moe_debug_row_dots.restype = i
        L.moe_debug_row_dots.argtypes = [_P, i, i, i, i, _P, _P, _P]
        L.moe_sum_partials.restype = i
        L.moe_sum_partials.argtypes = [_P, i, sz, _P, _P]
        f = ctypes.c_float
        L.moe_add_rmsnorm.restype = i
        L.moe_add_rmsnorm.argtypes = [_P, _P, _P, f, i, i, i, _P, _P, i, _P, _P, _P, _P]
        L.moe_expert_order.restype = i
        L.moe_expert_order.argtypes = [_P, i, i, i, _P, _P, _P, _P, _P, sz, _P]
        L.moe_expert_order_workspace_bytes.restype = sz
        L.moe_expert_order_workspace_bytes.argtypes = [i, i, i]
        L.moe_balance_loss.restype = i
        L.moe_balance_loss.argtypes = [_P, i, _P, _P, i, i, i, i, f, _P, _P, _P, _P, sz, _P]
        L.moe_balance_loss_workspace_bytes.restype = sz
        L.moe_balance_loss_workspace_bytes.argtypes = [i, i]
        L.moe_fp8_matmul.restype = i
        L.moe_fp8_matmul.argtypes = [_P, _P, i, _P, i, _P, i, _P, _P, i, i, _P, i, _P, sz, _P]
        L.moe_fp8_matmul_workspace_bytes.restype = sz
        L.moe_fp8_matmul_workspace_bytes.argtypes = []
        L.moe_topk.restype = i
        L.moe_topk.argtypes = [_P, i, _P, i, i, i, i, i, _P, _P, _P]
        L.moe_topk_grad.restype = i
        L.moe_topk_grad.argtypes = [_P, i, _P, _P, i, i, i, i, i, _P, _P, _P]
        L.moe_dispatch_rows.restype = i
        L.moe_dispatch_rows.argtypes = [_P, i, _P, i, i, i, i, _P, _P]
        L.moe_combine_rows.restype = i
        L.moe_combine_rows.argtypes = [_P, i, _P, _P, i, i, i, i, _P, _P, i, _P]
        L.moe_combine_grad.restype = i
        L.moe_combine_grad.argtypes = [_P, i, _P, _P, i, i, i, i, _P, i, _P, _P, _P]
        L.moe_matmul.restype = i
        L.moe_matmul.argtypes = [_P, i, _P, i, _P, i, _P, i, _P, i, _P, _P, i, i, _P, i, _P, sz, _P]
        L.moe_matmul_workspace_bytes.restype = sz
        L.moe_matmul_workspace_bytes.argtypes = []
        L.moe_debug_set_exchange_wait.restype = i
        L.moe_debug_set_exchange_wait.argtypes = [ctypes.c_longlong]
        L.moe_debug_hold_fp8_matmul.restype = i
        L.moe_debug_hold_fp8_matmul.argtypes = [i, ctypes.c_longlong]
        L.moe_debug_hold_matmul.restype = i
        L.moe_debug_hold_matmul.argtypes = [i, ctypes.c_longlong]
        L.moe_status_str.restype = ctypes.c_char_p
        L.moe_status_str.argtypes = [i]
        _lib_handle = L
    return _lib_handle


def status_str(s: int) -> str:
    return lib().moe_status_str(s).decode()


def _check(s: int, call: str):
    if s != 0:
        raise MoeError(s, call)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# ------------------------------------------------------------------ sizes

def moe_act_block(n: int) -> int:
    return lib().moe_act_block(n)


def moe_q8_row_bytes(n: int) -> int:
    return lib().moe_q8_row_bytes(n)


def moe_packed_bytes(qtype: int, rows: int, cols: int) -> int:
    return lib().moe_packed_bytes(qtype, rows, cols)


# ------------------------------------------------------------------ calls

def moe_pack_weights(blocks: torch.Tensor, qtype: int, rows: int, cols: int, packed: torch.Tensor, stream=None):
    _check(lib().moe_pack_weights(_ptr(blocks), qtype, rows, cols, _ptr(packed), _stream(stream)),
           "moe_pack_weights")


def moe_quantize_q8K(x: torch.Tensor, xq: torch.Tensor, stream=None):
    T, n = x.shape
    _check(lib().moe_quantize_q8K(_ptr(x), T, n, _ptr(xq), _stream(stream)), "moe_quantize_q8K")


def moe_route_workspace_bytes(T: int, E: int, H: int) -> int:
    return lib().moe_route_workspace_bytes(T, E, H)


def moe_route(hidden, xq, w_router, rtype: int, E: int, router_bias, k: int, gating: int, renormalize: bool,
              ids, weights, logits_out, ws, T: int | None = None, H: int | None = None, stream=None,
              shared_gate=None, shared_scale=None):
    if T is None or H is None:
        T, H = hidden.shape
    _check(lib().moe_route(_ptr(hidden), _ptr(xq), T, H, _ptr(w_router), rtype, E, _ptr(router_bias), k, gating,
                           int(bool(renormalize)), _ptr(ids), _ptr(weights), _ptr(logits_out), _ptr(shared_gate),
                           _ptr(shared_scale), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "moe_route")


class ExpertPool:
    """A moe_pool: packed expert matrices plus the device pointer table.

    entries: list of dicts with packed 'gate', 'up', 'down' tensors (or None
    for "not mine") and optional 'b_gate', 'b_up', 'b_down' fp32 tensors.
    A fused gate_up tensor (GGUF files may store gate and up as one [2I][H]
    matrix, gate rows first) packed as one matrix is given as 'gate_up': its
    first moe_packed_bytes(qtype, I, H) bytes are the gate, the rest the up
    projection (packed tiles of 32 rows are contiguous)."""

    def __init__(self, qtype: int, H: int, I: int, entries: list, device=None):
        self.qtype, self.H, self.I, self.E = qtype, H, I, len(entries)
        self._keep = []
        rows = []
        for en in entries:
            if en is not None and en.get("gate_up") is not None:
                if en.get("gate") is not None or en.get("up") is not None:
                    raise ValueError("give either 'gate_up' or 'gate' and 'up'")
                half = moe_packed_bytes(qtype, I, H)
                gu = en["gate_up"]
                if half == 0 or gu.numel() * gu.element_size() != 2 * half:
                    raise ValueError(f"'gate_up' must hold 2 x {half} packed bytes")
                flat = gu.reshape(-1).view(torch.uint8)
                en = dict(en, gate=flat[:half], up=flat[half:])
                del en["gate_up"]
            if en is None or en.get("gate") is None:
                rows.append([0] * 6)
                continue
            vals = [en.get(n) for n in ("gate", "up", "down", "b_gate", "b_up", "b_down")]
            self._keep.extend(v for v in vals if v is not None)
            rows.append([0 if v is None else v.data_ptr() for v in vals])
        device = device or (self._keep[0].device if self._keep else torch.device("cuda"))
        self.table = torch.tensor(rows, dtype=torch.int64).reshape(-1, 6).to(device)
        self.c = _Pool(qtype, H, I, self.E, self.table.data_ptr())


def moe_ffn_workspace_bytes(T: int, k: int, pool: ExpertPool, shared: ExpertPool | None) -> int:
    return lib().moe_ffn_workspace_bytes(T, k, ctypes.byref(pool.c),
                                         ctypes.byref(shared.c) if shared is not None else None)


def moe_expert_ffn(xq, T: int, ids, weights, k: int, pool: ExpertPool, shared: ExpertPool | None, y, ws,
                   stream=None, shared_scale=None):
    _check(lib().moe_expert_ffn(_ptr(xq), T, _ptr(ids), _ptr(weights), k, ctypes.byref(pool.c),
                                ctypes.byref(shared.c) if shared is not None else None, _ptr(shared_scale), _ptr(y),
                                _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)), "moe_expert_ffn")


def moe_expert_ffn_noalloc(xq, T: int, ids, weights, k: int, pool: ExpertPool, shared: ExpertPool | None, y,
                           stream=None, shared_scale=None):
    """moe_expert_ffn with the library's fixed device scratch (no workspace, no allocation)."""
    _check(lib().moe_expert_ffn_noalloc(_ptr(xq), T, _ptr(ids), _ptr(weights), k, ctypes.byref(pool.c),
                                        ctypes.byref(shared.c) if shared is not None else None,
                                        _ptr(shared_scale), _ptr(y), _stream(stream)), "moe_expert_ffn_noalloc")


def moe_layer_workspace_bytes(T: int, k: int, pool: ExpertPool, shared: ExpertPool | None) -> int:
    return lib().moe_layer_workspace_bytes(T, k, ctypes.byref(pool.c),
                                           ctypes.byref(shared.c) if shared is not None else None)


def moe_layer_forward(hidden, w_router, rtype: int, router_bias, k: int, gating: int, renormalize: bool,
                      pool: ExpertPool, shared: ExpertPool | None, y, ws, ids_out=None, weights_out=None,
                      logits_out=None, xq_out=None, flags: int = 0, T: int | None = None, stream=None,
                      shared_gate=None):
    T = hidden.shape[0] if T is None else T
    _check(lib().moe_layer_forward(_ptr(hidden), T, _ptr(w_router), rtype, _ptr(router_bias), k, gating,
                                   int(bool(renormalize)), ctypes.byref(pool.c),
                                   ctypes.byref(shared.c) if shared is not None else None, _ptr(shared_gate),
                                   _ptr(y),
                                   _ptr(ids_out), _ptr(weights_out), _ptr(logits_out), _ptr(xq_out), _ptr(ws),
                                   ws.numel() * ws.element_size(), flags, _stream(stream)), "moe_layer_forward")


def moe_sum_partials(parts, y, stream=None):
    """y = the partial outputs parts [R, ...] summed in rank order (expert parallelism)."""
    R = parts.shape[0]
    n = y.numel()
    if parts.numel() != R * n:
        raise ValueError("parts must hold R partials of y's size")
    _check(lib().moe_sum_partials(_ptr(parts), R, n, _ptr(y), _stream(stream)), "moe_sum_partials")


# --------------------------------------------------- around the experts
#
# These calls check shapes, types, layouts and devices of their tensors (ValueError, csrc/binding.cpp) and run on
# the device that holds them, on its current stream unless one is given.

_bound = None


def _native():
    """The compiled binding of the calls below.  Raises if it has not been built, or for another torch or Python."""
    global _bound
    if _bound is None:
        lib()
        from . import _calls
        have, want = _calls.built_for, _build.calls_stamp()
        if have != want:
            raise RuntimeError(f"{_build.CALLS_SO} is built for {have}, this is {want}: run __graft_entry__.build()")
        _bound = _calls
    return _bound


def moe_add_rmsnorm(x, residual, weight, eps: float, residual_out=None, y=None, xq=None, x8=None, x8_scale=None,
                    stream=None):
    """s = x + residual (None: s = x), v = s / sqrt(mean(s^2) + eps) * weight, row by row.

    x, residual, residual_out (s; may be x or residual): [T, n] fp32 or bf16.  y (v): [T, n] fp32 or bf16.
    xq: q8 records of v (device_bytes(T * moe_q8_row_bytes(n))).  x8, x8_scale: e4m3 [T, n] and its fp32
    scales [T, ceil(n / 128)].  Give the outputs that are wanted."""
    s = (_bound or _native()).add_rmsnorm(x, residual, weight, eps, residual_out, y, xq, x8, x8_scale, stream)
    if s:
        raise MoeError(s, "moe_add_rmsnorm")


def moe_expert_order_workspace_bytes(T: int, k: int, E: int) -> int:
    return lib().moe_expert_order_workspace_bytes(T, k, E)


def moe_expert_order(ids, E: int, ws=None, counts=None, offsets=None, rows=None, pos=None, stream=None):
    """The (token, slot) pairs of ids [T, k] sorted by expert: counts [E], offsets [E + 1], the token of each
    sorted place rows [T * k] (-1 past the last) and the sorted place of each pair pos [T, k] (-1: takes no
    part, its id is not in [0, E)).  All int32; give the outputs that are wanted."""
    s = (_bound or _native()).expert_order(ids, E, ws, counts, offsets, rows, pos, stream)
    if s:
        raise MoeError(s, "moe_expert_order")


def moe_balance_loss_workspace_bytes(T: int, E: int) -> int:
    return lib().moe_balance_loss_workspace_bytes(T, E)


def moe_balance_loss(logits, counts, k: int, gating: int, alpha: float, ws, loss=None, dlogits=None, valid=None,
                     grad_loss=None, stream=None):
    """The balance loss alpha * sum_e (E c_e / N)(mean p_e) of logits [T, E] (fp32 or bf16) and counts [E]
    (moe_expert_order) into loss [1], and grad_loss [1] times its gradient into dlogits [T, E]; either may be
    None.  valid: uint8 or bool [T], 0 for padded tokens."""
    s = (_bound or _native()).balance_loss(logits, counts, k, gating, alpha, ws, loss, dlogits, valid, grad_loss, stream)
    if s:
        raise MoeError(s, "moe_balance_loss")


def moe_fp8_matmul_workspace_bytes() -> int:
    return lib().moe_fp8_matmul_workspace_bytes()


def moe_fp8_matmul(x8, x_scale, w, w_scale, y, ws, offsets=None, rows=None, stream=None):
    """y = x8 @ w.T with the scales of both, dense or grouped by expert.

    x8 [X, K] e4m3, x_scale [X, ceil(K/128)] fp32; w [N, K] or [G, N, K] e4m3, w_scale [ceil(N/128),
    ceil(K/128)] or [G, ...] fp32; y [M, N] fp32 or bf16.  offsets int32 [G + 1]: the places of y of each
    group (moe_expert_order); rows int32 [M]: the row of x8 of each place (None: the place itself).  e4m3
    tensors are torch.float8_e4m3fn or uint8."""
    s = (_bound or _native()).fp8_matmul(x8, x_scale, w, w_scale, y, ws, offsets, rows, stream)
    if s:
        raise MoeError(s, "moe_fp8_matmul")


def moe_topk(logits, gating: int, renormalize: bool, ids, weights=None, valid=None, stream=None):
    """The k experts of each token, the largest logits first, and their gating weights, as moe_route chooses and weighs
    them, for any number of tokens: logits [T, E] fp32 or bf16 -> ids int32 [T, k], weights fp32 [T, k].
    valid: uint8 or bool [T], 0 for padded tokens (ids -1, weights 0)."""
    s = (_bound or _native()).topk(logits, gating, renormalize, ids, weights, valid, stream)
    if s:
        raise MoeError(s, "moe_topk")


def moe_topk_grad(logits, ids, dweights, gating: int, renormalize: bool, dlogits, addend=None, stream=None):
    """dlogits = addend (None: 0) + the gradient of moe_topk's weights, from dweights [T, k], with the choice held
    fixed.  logits, addend, dlogits: [T, E] of one type; dlogits may be either of the others."""
    s = (_bound or _native()).topk_grad(logits, ids, dweights, gating, renormalize, dlogits, addend, stream)
    if s:
        raise MoeError(s, "moe_topk_grad")


def moe_dispatch_rows(x, pos, xs, stream=None):
    """xs[pos[t, s]] = x[t]: token rows [T, n] to their places [M, n] in the order by expert (moe_expert_order's
    pos [T, k]; -1: takes no part).  Its gradient is moe_combine_rows without weights."""
    s = (_bound or _native()).dispatch_rows(x, pos, xs, stream)
    if s:
        raise MoeError(s, "moe_dispatch_rows")


def moe_combine_rows(o, pos, y, weights=None, addend=None, stream=None):
    """y[t] = addend[t] + sum_s weights[t, s] o[pos[t, s]] (None: 0 and 1), added in fp32 in the order of the slots.
    o [M, n], y [T, n], addend [T, n] of y's type (may be y), weights fp32 [T, k]."""
    s = (_bound or _native()).combine_rows(o, pos, y, weights, addend, stream)
    if s:
        raise MoeError(s, "moe_combine_rows")


def moe_combine_grad(dy, pos, weights=None, o=None, do=None, dweights=None, stream=None):
    """The gradient of moe_combine_rows: do[pos[t, s]] = weights[t, s] dy[t] and dweights[t, s] = <o[pos[t, s]], dy[t]>;
    either may be None, and o without dweights.  do may be o."""
    s = (_bound or _native()).combine_grad(dy, pos, weights, o, do, dweights, stream)
    if s:
        raise MoeError(s, "moe_combine_grad")


def moe_matmul_workspace_bytes() -> int:
    return lib().moe_matmul_workspace_bytes()


def moe_matmul(x, w, y, ws, act: int = ACT_NONE, bias=None, residual=None, z=None, offsets=None, rows=None,
               transposed: bool = False, stream=None):
    """y = act(x @ w.T + bias) + residual, dense or grouped by expert; with an ACT_*_GRAD y = (x @ w.T) act'(z).

    x [X, K] bf16; w [N, K] or [G, N, K] bf16 (transposed: [K, N], [G, K, N]); y [M, N] fp32 or bf16; bias fp32
    [N] or [G, N]; residual [M, N] of y's type (may be y).  ACT_SWIGLU: w and bias have 2 N rows, gate then up.
    z of y's type: what the activation takes, out ([M, N], ACT_SWIGLU [M, 2 N]); the gradients' input.
    ACT_SWIGLU_GRAD: y is [M, 2 N].  offsets int32 [G + 1]: the places of y of each group (moe_expert_order);
    rows int32 [M]: the row of x of each place (None: the place itself)."""
    s = (_bound or _native()).matmul(x, w, y, ws, act, bias, residual, z, offsets, rows, transposed, stream)
    if s:
        raise MoeError(s, "moe_matmul")


def moe_debug_set_exchange_wait(cycles: int):
    """Test hook: bound on a layer launch's waits for other blocks' words (0: default)."""
    _check(lib().moe_debug_set_exchange_wait(int(cycles)), "moe_debug_set_exchange_wait")


def moe_debug_hold_fp8_matmul(hold: int, cycles: int = 0):
    """Test hook: 1 or 2 makes the waits of moe_fp8_matmul's tiles run out after `cycles` (0: default); 0 is off."""
    _check(lib().moe_debug_hold_fp8_matmul(int(hold), int(cycles)), "moe_debug_hold_fp8_matmul")


def moe_debug_hold_matmul(hold: int, cycles: int = 0):
    """Test hook: 1 or 2 makes the waits of moe_matmul run out after `cycles` (0: default); 0 is off."""
    _check(lib().moe_debug_hold_matmul(int(hold), int(cycles)), "moe_debug_hold_matmul")


def moe_read_device_status(ws, clear: bool = True, stream=None) -> int:
    flags = ctypes.c_uint32(0)
    s = lib().moe_read_device_status(_ptr(ws), int(clear), ctypes.byref(flags), _stream(stream))
    if s not in (0, 5):
        raise MoeError(s, "moe_read_device_status")
    return flags.value


def moe_debug_row_dots(packed, qtype: int, rows: int, cols: int, row: int, xq, isums, stream=None):
    _check(lib().moe_debug_row_dots(_ptr(packed), qtype, rows, cols, row, _ptr(xq), _ptr(isums),
                                    _stream(stream)), "moe_debug_row_dots")


# ----------------------------------------------------------- conveniences

def device_bytes(n: int, device="cuda") -> torch.Tensor:
    """A 256-byte aligned uint8 device buffer (torch's allocator aligns to 512)."""
    return torch.empty(max(int(n), 16), dtype=torch.uint8, device=device)


def pack(blocks: torch.Tensor, qtype: int, rows: int, cols: int, stream=None) -> torch.Tensor:
    """Pack one GGUF-style block matrix (device uint8) into a new device buffer."""
    out = device_bytes(moe_packed_bytes(qtype, rows, cols), blocks.device)
    moe_pack_weights(blocks, qtype, rows, cols, out, stream)
    return out


def quantize(x: torch.Tensor, stream=None) -> torch.Tensor:
    T, n = x.shape
    xq = device_bytes(T * moe_q8_row_bytes(n), x.device)
    moe_quantize_q8K(x, xq, stream)
    return xq


def unpack_q8(xq: torch.Tensor, T: int, n: int):
    """Split q8 records (host or device uint8) into (d [T, n/B], q [T, n], bsum [T, n/16]) tensors."""
    B = moe_act_block(n)
    rb = moe_q8_row_bytes(n)
    a = ((4 * (n // B)) + 15) & ~15
    r = xq[: T * rb].reshape(T, rb)
    d = r[:, : 4 * (n // B)].contiguous().view(torch.float32)
    q = r[:, a: a + n].contiguous().view(torch.int8)
    bs = r[:, a + n: a + n + 2 * (n // 16)].contiguous().view(torch.int16)
    return d, q, bs
