"""Host-side checks of the calls around the experts: limits, types, buffers and workspaces are refused before
anything is launched.  Stand-in addresses, so only where no GPU is visible (as in test_abi.py)."""
import ctypes

import pytest

import quantized_routed_expert_router_gb300 as moe
from test_abi import host_only

INVALID, UNSUP, WS = 1, 2, 3
P = 1 << 20                       # a stand-in device address, 16-byte aligned
S = ctypes.c_void_p(0)


def test_sizes():
    assert moe.moe_expert_order_workspace_bytes(512, 8, 256) == 0            # few pairs need none
    assert moe.moe_expert_order_workspace_bytes(65536, 8, 256) % (256 * 2) == 0
    assert moe.moe_expert_order_workspace_bytes(65536, 8, 256) > 0
    assert moe.moe_expert_order_workspace_bytes(0, 8, 256) == 0
    assert moe.moe_expert_order_workspace_bytes(1, 0, 256) == 0
    assert moe.moe_balance_loss_workspace_bytes(1, 1) > 0 and moe.moe_balance_loss_workspace_bytes(-1, 8) == 0
    assert moe.moe_fp8_matmul_workspace_bytes() % 16 == 0


@host_only
@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(T=(1 << 24) + 1), INVALID), (dict(n=0), UNSUP), (dict(n=24), UNSUP),
    (dict(n=16400), UNSUP), (dict(dtype=2), INVALID), (dict(ydtype=-1), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(x=P + 8), INVALID), (dict(r=P + 4), INVALID), (dict(y=P + 8), INVALID),
    (dict(x8=P), INVALID), (dict(sc=P), INVALID), (dict(x8=P + 8, sc=P), INVALID), (dict(x8=P, sc=P + 2), INVALID),
    (dict(xq=P, n=48), UNSUP), (dict(xq=P + 8), INVALID), (dict(y=None), INVALID), (dict(T=0, x=None), 0),
    (dict(T=0, y=None), 0)])
def test_norm_refusals(change, status):
    a = dict(x=P, r=P, w=P, eps=1e-6, T=4, n=64, dtype=0, out=None, y=P, ydtype=0, xq=None, x8=None, sc=None)
    a.update(change)
    assert moe.lib().moe_add_rmsnorm(a["x"], a["r"], a["w"], a["eps"], a["T"], a["n"], a["dtype"], a["out"], a["y"],
                                     a["ydtype"], a["xq"], a["x8"], a["sc"], S) == status


@host_only
@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(k=33), INVALID), (dict(E=0), INVALID), (dict(E=1025), INVALID),
    (dict(T=(1 << 22) // 8 + 1), INVALID), (dict(ids=None), INVALID), (dict(ids=P + 2), INVALID),
    (dict(counts=P + 1), INVALID), (dict(counts=None), INVALID), (dict(T=0, counts=None), 0), (dict(T=10000, ws=None), WS),
    (dict(T=10000, size=8 * 2 * 10 - 1), WS), (dict(T=10000, ws=P + 4), WS)])
def test_order_refusals(change, status):
    a = dict(ids=P, T=4, k=8, E=8, counts=P, ws=P, size=1 << 20)
    a.update(change)
    assert moe.lib().moe_expert_order(a["ids"], a["T"], a["k"], a["E"], a["counts"], None, None, None, a["ws"],
                                      a["size"], S) == status


@host_only
@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(E=1025), INVALID), (dict(k=0), INVALID), (dict(k=9), INVALID),
    (dict(dtype=2), INVALID), (dict(gating=2), INVALID), (dict(counts=None), INVALID), (dict(counts=P + 2), INVALID),
    (dict(logits=None), INVALID), (dict(logits=P + 4), INVALID), (dict(d=P + 4), INVALID), (dict(loss=None), INVALID),
    (dict(T=0, loss=None), 0),
    (dict(loss=P + 1), INVALID), (dict(gl=P + 1), INVALID), (dict(ws=None), WS), (dict(size=100), WS),
    (dict(ws=P + 8), WS)])
def test_balance_refusals(change, status):
    a = dict(logits=P, dtype=0, counts=P, T=4, E=8, k=2, gating=0, gl=None, loss=P, d=None, ws=P, size=1 << 20)
    a.update(change)
    assert moe.lib().moe_balance_loss(a["logits"], a["dtype"], a["counts"], None, a["T"], a["E"], a["k"], a["gating"],
                                      0.01, a["gl"], a["loss"], a["d"], a["ws"], a["size"], S) == status


@host_only
@pytest.mark.parametrize("change,status", [
    (dict(X=-1), INVALID), (dict(M=-1), INVALID), (dict(M=(1 << 24) + 1), INVALID), (dict(G=0), INVALID),
    (dict(G=1025), INVALID), (dict(N=0), INVALID), (dict(N=(1 << 20) + 1), INVALID), (dict(G=1024, N=1 << 20, offs=P), 0),
    (dict(G=1024, N=(1 << 20), M=4, offs=None), INVALID), (dict(K=0), UNSUP), (dict(K=24), UNSUP),
    (dict(K=(1 << 20) + 16), UNSUP), (dict(X=1 << 17, K=1 << 20), INVALID), (dict(yd=3), INVALID), (dict(G=2), INVALID), (dict(X=0), INVALID),
    (dict(X=3), INVALID), (dict(x=None), INVALID), (dict(xs=None), INVALID), (dict(w=None), INVALID),
    (dict(wsc=None), INVALID), (dict(y=None), INVALID), (dict(x=P + 8), INVALID), (dict(w=P + 8), INVALID),
    (dict(y=P + 8), INVALID), (dict(xs=P + 2), INVALID), (dict(wsc=P + 2), INVALID), (dict(rows=P + 1), INVALID),
    (dict(offs=P + 1), INVALID), (dict(ws=None), WS), (dict(size=16), WS), (dict(ws=P + 4), WS),
    (dict(M=0, x=None), 0)])
def test_matmul_refusals(change, status):
    a = dict(x=P, xs=P, X=4, rows=None, M=4, offs=None, G=1, w=P, wsc=P, N=64, K=64, y=P, yd=0, ws=P, size=1 << 20)
    a.update(change)
    if status == 0 and a["M"]:
        a["M"] = 0                # in range: shown by the no-op, nothing is launched
    assert moe.lib().moe_fp8_matmul(a["x"], a["xs"], a["X"], a["rows"], a["M"], a["offs"], a["G"], a["w"], a["wsc"],
                                    a["N"], a["K"], a["y"], a["yd"], a["ws"], a["size"], S) == status


def test_the_binding_checks_tensors_before_the_call():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_add_rmsnorm(x, None, torch.ones(64), 1e-6, y=torch.zeros(2, 64))
    with pytest.raises(ValueError, match="weight"):
        moe.moe_add_rmsnorm(x, None, torch.ones(32), 1e-6, y=torch.zeros(2, 64))
    with pytest.raises(ValueError, match="ids"):
        moe.moe_expert_order(torch.zeros(2, 4, dtype=torch.int64), 8, counts=torch.zeros(8, dtype=torch.int32))
    with pytest.raises(ValueError, match="counts"):
        moe.moe_balance_loss(x, torch.zeros(63, dtype=torch.int32), 2, moe.SOFTMAX, 0.1, torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="x_scale"):
        moe.moe_fp8_matmul(x.to(torch.float8_e4m3fn), torch.zeros(2, 2), torch.zeros(8, 64, dtype=torch.float8_e4m3fn),
                           torch.zeros(1, 1), torch.zeros(2, 8), torch.zeros(256, dtype=torch.uint8))


def test_the_binding_refuses_what_is_no_tensor_or_number():
    torch = pytest.importorskip("torch")
    x, w, y = torch.zeros(2, 64), torch.ones(64), torch.zeros(2, 64)
    with pytest.raises(ValueError, match="x: want a tensor"):
        moe.moe_add_rmsnorm([1.0], None, w, 1e-6, y=y)
    with pytest.raises(ValueError, match="y: want a tensor or None"):
        moe.moe_add_rmsnorm(x, None, w, 1e-6, y=3)
    with pytest.raises(TypeError):
        moe.moe_add_rmsnorm(x, None, w, "small", y=y)
    ids = torch.zeros(2, 4, dtype=torch.int32)
    for E in (2 ** 40, 2 ** 70):
        with pytest.raises((ValueError, OverflowError)):
            moe.moe_expert_order(ids, E)
    with pytest.raises(TypeError):
        moe.moe_expert_order(ids, None)
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_add_rmsnorm(x, None, w, 1e-6, y=torch.zeros(64, 2).t())
    with pytest.raises(TypeError, match="arguments"):
        moe._native().add_rmsnorm(x)
    with pytest.raises(ValueError, match="w: want"):
        moe.moe_fp8_matmul(x.to(torch.float8_e4m3fn), torch.zeros(2, 1), torch.zeros(8), torch.zeros(1, 1), y,
                           torch.zeros(256, dtype=torch.uint8))
