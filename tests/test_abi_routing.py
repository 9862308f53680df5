"""Host-side checks of the top-k gating, the expert rows and the products with an epilogue: limits, types, buffers and
workspaces are refused before anything is launched.  Stand-in addresses, so only where no GPU is visible."""
import ctypes

import pytest

import quantized_routed_expert_router_gb300 as moe
from test_abi import host_only

INVALID, UNSUP, WS = 1, 2, 3
P = 1 << 20                       # a stand-in device address, 16-byte aligned
S = ctypes.c_void_p(0)
MANY = (1 << 24) + 1


@host_only
@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(T=MANY), INVALID), (dict(E=0), INVALID), (dict(E=1025), INVALID), (dict(k=0), INVALID),
    (dict(k=9), INVALID), (dict(E=64, k=33), INVALID), (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID),
    (dict(gating=2), INVALID), (dict(logits=None), INVALID), (dict(logits=P + 8), INVALID), (dict(ids=None), INVALID),
    (dict(ids=P + 2), INVALID), (dict(w=P + 1), INVALID), (dict(T=0, logits=None, ids=None), 0)])
def test_topk_refusals(change, status):
    a = dict(logits=P, dtype=0, T=4, E=8, k=2, gating=0, ids=P, w=P)
    a.update(change)
    assert moe.lib().moe_topk(a["logits"], a["dtype"], None, a["T"], a["E"], a["k"], a["gating"], 1, a["ids"], a["w"],
                              S) == status


@host_only
@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(E=1025), INVALID), (dict(k=9), INVALID), (dict(dtype=2), INVALID),
    (dict(gating=-1), INVALID), (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(dw=None), INVALID),
    (dict(d=None), INVALID), (dict(logits=P + 4), INVALID), (dict(add=P + 8), INVALID), (dict(d=P + 2), INVALID),
    (dict(ids=P + 2), INVALID), (dict(dw=P + 1), INVALID), (dict(T=0, d=None), 0)])
def test_topk_grad_refusals(change, status):
    a = dict(logits=P, dtype=0, ids=P, dw=P, T=4, E=8, k=2, gating=0, add=None, d=P)
    a.update(change)
    assert moe.lib().moe_topk_grad(a["logits"], a["dtype"], a["ids"], a["dw"], a["T"], a["E"], a["k"], a["gating"], 1,
                                   a["add"], a["d"], S) == status


ROW_LIMITS = [(dict(T=-1), INVALID), (dict(T=MANY), INVALID), (dict(k=0), INVALID), (dict(k=33), INVALID),
              (dict(T=(1 << 22) // 2 + 1), INVALID), (dict(n=0), INVALID), (dict(n=65537), INVALID), (dict(M=-1), INVALID),
              (dict(M=MANY), INVALID), (dict(M=1 << 24, n=8192), INVALID), (dict(T=1 << 21, n=65536), INVALID),
              (dict(dtype=2), INVALID), (dict(pos=None), INVALID), (dict(pos=P + 2), INVALID)]


@host_only
@pytest.mark.parametrize("change,status", ROW_LIMITS + [
    (dict(x=None), INVALID), (dict(xs=None), INVALID), (dict(x=P + 8), INVALID), (dict(xs=P + 4), INVALID),
    (dict(T=0, x=None), 0), (dict(M=0, xs=None), 0)])
def test_dispatch_refusals(change, status):
    a = dict(x=P, dtype=0, pos=P, T=4, k=2, n=64, M=8, xs=P)
    a.update(change)
    assert moe.lib().moe_dispatch_rows(a["x"], a["dtype"], a["pos"], a["T"], a["k"], a["n"], a["M"], a["xs"], S) == status


@host_only
@pytest.mark.parametrize("change,status", ROW_LIMITS + [
    (dict(yd=2), INVALID), (dict(o=None), INVALID), (dict(y=None), INVALID), (dict(o=P + 8), INVALID),
    (dict(y=P + 8), INVALID), (dict(add=P + 8), INVALID), (dict(w=P + 2), INVALID), (dict(T=0, o=None, y=None), 0)])
def test_combine_refusals(change, status):
    a = dict(o=P, dtype=0, pos=P, w=None, T=4, k=2, n=64, M=8, add=None, y=P, yd=0)
    a.update(change)
    assert moe.lib().moe_combine_rows(a["o"], a["dtype"], a["pos"], a["w"], a["T"], a["k"], a["n"], a["M"], a["add"],
                                      a["y"], a["yd"], S) == status


@host_only
@pytest.mark.parametrize("change,status", ROW_LIMITS + [
    (dict(yd=2), INVALID), (dict(dy=None), INVALID), (dict(o=None), INVALID), (dict(d=None, dw=None), INVALID),
    (dict(dy=P + 4), INVALID), (dict(o=P + 4), INVALID), (dict(d=P + 4), INVALID), (dict(dw=P + 2), INVALID),
    (dict(w=P + 2), INVALID), (dict(T=0, dy=None), 0)])
def test_combine_grad_refusals(change, status):
    a = dict(dy=P, yd=0, pos=P, w=None, T=4, k=2, n=64, M=8, o=P, dtype=0, d=P, dw=P)
    a.update(change)
    assert moe.lib().moe_combine_grad(a["dy"], a["yd"], a["pos"], a["w"], a["T"], a["k"], a["n"], a["M"], a["o"],
                                      a["dtype"], a["d"], a["dw"], S) == status


@host_only
@pytest.mark.parametrize("change,status", [
    (dict(X=-1), INVALID), (dict(X=MANY), INVALID), (dict(M=-1), INVALID), (dict(M=MANY), INVALID), (dict(G=0), INVALID),
    (dict(G=1025), INVALID), (dict(N=0), INVALID), (dict(N=(1 << 20) + 1), INVALID), (dict(K=0), UNSUP), (dict(K=12), UNSUP),
    (dict(K=(1 << 20) + 8), UNSUP), (dict(X=1 << 17, K=1 << 20), INVALID), (dict(X=(1 << 15) + 1, K=1 << 20), INVALID), (dict(G=1024, N=(1 << 20) + 0, offs=None), INVALID),
    (dict(yd=2), INVALID), (dict(act=-1), INVALID), (dict(act=7), INVALID), (dict(G=2), INVALID), (dict(X=0), INVALID),
    (dict(X=3), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
    (dict(x=P + 8), INVALID), (dict(w=P + 8), INVALID), (dict(y=P + 8), INVALID), (dict(act=1, z=P + 8), INVALID),
    (dict(res=P + 8), INVALID), (dict(bias=P + 2), INVALID), (dict(rows=P + 1), INVALID), (dict(offs=P + 1), INVALID),
    (dict(z=P), INVALID), (dict(act=4), INVALID), (dict(act=4, z=P, bias=P), INVALID), (dict(act=6, z=P, res=P), INVALID),
    (dict(tr=1, N=60), UNSUP), (dict(act=3, N=56), UNSUP), (dict(act=3, tr=1), UNSUP), (dict(ws=None), WS),
    (dict(size=16), WS), (dict(ws=P + 4), WS), (dict(M=0, x=None), 0)])
def test_product_refusals(change, status):
    a = dict(x=P, X=4, rows=None, M=4, offs=None, G=1, w=P, tr=0, bias=None, act=0, res=None, z=None, N=64, K=64, y=P, yd=0,
             ws=P, size=1 << 20)
    a.update(change)
    assert moe.lib().moe_matmul(a["x"], a["X"], a["rows"], a["M"], a["offs"], a["G"], a["w"], a["tr"], a["bias"],
                                a["act"], a["res"], a["z"], a["N"], a["K"], a["y"], a["yd"], a["ws"], a["size"],
                                S) == status


def test_workspace_size():
    assert moe.moe_matmul_workspace_bytes() % 16 == 0 and moe.moe_matmul_workspace_bytes() > 0


def test_the_binding_checks_tensors_before_the_call():
    torch = pytest.importorskip("torch")
    i32, bf16 = torch.int32, torch.bfloat16
    l, ids, w = torch.zeros(2, 8), torch.zeros(2, 2, dtype=i32), torch.zeros(2, 2)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_topk(l, moe.SOFTMAX, True, ids, w)
    with pytest.raises(ValueError, match="weights"):
        moe.moe_topk(l, moe.SOFTMAX, True, ids, w[:, :1].contiguous())
    with pytest.raises(ValueError, match="ids"):
        moe.moe_topk(l, moe.SOFTMAX, True, ids.long(), w)
    with pytest.raises(ValueError, match="ids"):
        moe.moe_topk(l, moe.SOFTMAX, True, None, w)
    with pytest.raises(ValueError, match="addend"):
        moe.moe_topk_grad(l, ids, w, moe.SOFTMAX, True, l.clone(), addend=l.to(bf16))
    x, pos = torch.zeros(2, 16), torch.zeros(2, 2, dtype=i32)
    with pytest.raises(ValueError, match="xs"):
        moe.moe_dispatch_rows(x, pos, torch.zeros(4, 16, dtype=bf16))
    with pytest.raises(ValueError, match="pos"):
        moe.moe_dispatch_rows(x, torch.zeros(3, 2, dtype=i32), torch.zeros(4, 16))
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_dispatch_rows(torch.zeros(16, 2).t(), pos, torch.zeros(4, 16))
    with pytest.raises(ValueError, match="addend"):
        moe.moe_combine_rows(torch.zeros(4, 16), pos, x.to(bf16), addend=x)
    with pytest.raises(ValueError, match="y"):
        moe.moe_combine_rows(torch.zeros(4, 16), pos, torch.zeros(3, 16))
    with pytest.raises(ValueError, match="do"):
        moe.moe_combine_grad(x, pos, dweights=w)
    with pytest.raises(ValueError, match="do"):
        moe.moe_combine_grad(x, pos, o=torch.zeros(4, 16), do=torch.zeros(4, 16, dtype=bf16))
    ws, xb = torch.zeros(256, dtype=torch.uint8), torch.zeros(4, 16, dtype=bf16)
    wb, y = torch.zeros(8, 16, dtype=bf16), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="x: want"):
        moe.moe_matmul(xb.float(), wb, y, ws)
    with pytest.raises(ValueError, match="w: want"):
        moe.moe_matmul(xb, wb[0], y, ws)
    with pytest.raises(ValueError, match="w: want"):
        moe.moe_matmul(xb, wb, y, ws, transposed=True)
    with pytest.raises(ValueError, match="y: want"):
        moe.moe_matmul(xb, wb, y, ws, act=moe.ACT_SWIGLU)
    with pytest.raises(ValueError, match="bias"):
        moe.moe_matmul(xb, wb, y, ws, bias=torch.zeros(1, 8))
    with pytest.raises(ValueError, match="residual"):
        moe.moe_matmul(xb, wb, y, ws, residual=y.to(bf16))
    with pytest.raises(ValueError, match="z: want"):
        moe.moe_matmul(xb, wb, y, ws, act=moe.ACT_SILU, z=torch.zeros(4, 16))
    with pytest.raises(ValueError, match="gate rows"):
        moe.moe_matmul(xb, wb[:7].contiguous(), y, ws, act=moe.ACT_SWIGLU)
