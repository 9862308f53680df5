"""Routing, rows and products in a run, as a training step of a routed layer whose experts are held fixed makes it:
logits -> top-k -> order -> gate and up product with the gated activation -> down product -> combine, and back to the
rows and the logits; against 64-bit autograd of the whole layer.

Each value that goes from call to call in bf16 is rounded by 2^-8 of itself, four in a row on either way (h, o; do, dz,
dxs), and the sums of rounded values keep the relative size of their roundings where these are independent.  The check is of
the whole tensors' relative distance: each of n <= 5 roundings in turn adds at most 2^-8 of the tensor's norm times the
layer's gain for it, taken as 2 (silu's slope of 1.1 and gate times up, each with its own rounding), so 5 * 2 * 2^-8.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("quantized_routed_expert_router_gb300")

DEV = "cuda"
BF16 = torch.bfloat16


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 64, 32), (16, 16, 4, 512, 288), (300, 32, 4, 576, 288)])
@pytest.mark.parametrize("gating", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("graph", [False, True])
def test_step(T, E, k, H, I, gating, graph):
    g = torch.Generator(device=DEV).manual_seed(T + E)
    rand = lambda *s, scale=1.0: scale * torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    new = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731
    i32, P = torch.int32, T * k
    x, logits, dy = rand(T, H).to(BF16), rand(T, E), rand(T, H)
    wgu, wd = rand(E, 2 * I, H, scale=H ** -0.5).to(BF16), rand(E, H, I, scale=I ** -0.5).to(BF16)
    bgu, bd = rand(E, 2 * I, scale=0.2), rand(E, H, scale=0.2)
    residual, pad = rand(T, H), T // 5
    valid = torch.ones(T, dtype=torch.uint8, device=DEV)
    valid[T - pad:] = 0
    ids, w, pos, rows = new(T, k, dtype=i32), new(T, k, dtype=torch.float32), new(T, k, dtype=i32), new(P, dtype=i32)
    counts, offs = new(E, dtype=i32), new(E + 1, dtype=i32)
    ows = new(max(16, moe.moe_expert_order_workspace_bytes(T, k, E)), dtype=torch.uint8)
    bws = new(moe.moe_balance_loss_workspace_bytes(T, E), dtype=torch.uint8)
    mws = new(moe.moe_matmul_workspace_bytes(), dtype=torch.uint8)
    z, h, o, y = new(P, 2 * I), new(P, I), new(P, H), new(T, H, dtype=torch.float32)
    do, dz, dxs, dx = new(P, H), new(P, 2 * I), new(P, H), new(T, H, dtype=torch.float32)
    dw, dlogits, loss = new(T, k, dtype=torch.float32), new(T, E, dtype=torch.float32), new(1, dtype=torch.float32)

    def step():
        moe.moe_topk(logits, gating, True, ids, w, valid=valid)
        moe.moe_expert_order(ids, E, ows, counts=counts, offsets=offs, rows=rows, pos=pos)
        moe.moe_matmul(x, wgu, h, mws, act=moe.ACT_SWIGLU, bias=bgu, z=z, offsets=offs, rows=rows)
        moe.moe_matmul(h, wd, o, mws, bias=bd, offsets=offs)
        moe.moe_combine_rows(o, pos, y, weights=w, addend=residual)
        moe.moe_combine_grad(dy, pos, weights=w, o=o, do=do, dweights=dw)
        moe.moe_matmul(do, wd, dz, mws, act=moe.ACT_SWIGLU_GRAD, z=z, offsets=offs, transposed=True)
        moe.moe_matmul(dz, wgu, dxs, mws, offsets=offs, transposed=True)
        moe.moe_combine_rows(dxs, pos, dx)
        moe.moe_balance_loss(logits, counts, k, gating, 0.01, bws, loss=loss, dlogits=dlogits, valid=valid)
        moe.moe_topk_grad(logits, ids, dw, gating, True, dlogits, addend=dlogits)

    step()
    if graph:
        torch.cuda.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            step()
        for t in (x, logits, dy):
            t.copy_(rand(*t.shape))
        cg.replay()
    assert moe.moe_read_device_status(mws) == 0

    xl, ll = x.double().requires_grad_(True), logits.double().requires_grad_(True)
    log = torch.log_softmax(ll, 1) if gating == moe.SOFTMAX else torch.nn.functional.logsigmoid(ll)
    live = valid.bool()
    top = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids[live].long(), top[live]) and bool((ids[~live] == -1).all())
    c = torch.gather(log, 1, top)
    wl = torch.exp(c - torch.logsumexp(c, 1, keepdim=True))
    out = residual.double()
    for s in range(k):
        e = top[:, s]
        v = torch.einsum("th,tih->ti", xl, wgu.double()[e]) + bgu.double()[e]
        hh = torch.nn.functional.silu(v[:, :I]) * v[:, I:]
        oo = torch.einsum("ti,thi->th", hh, wd.double()[e]) + bd.double()[e]
        out = out + torch.where(live[:, None], wl[:, s:s + 1] * oo, torch.zeros_like(oo))
    p = torch.softmax(log, 1)
    n = int(live.sum()) * k
    f = torch.bincount(top[live].reshape(-1), minlength=E).double() * E / n
    bal = 0.01 * k / n * (p[live] * f).sum()
    gx, gl = torch.autograd.grad((out * dy.double()).sum() + bal, (xl, ll))

    def near(a, b, what):
        d = float((a.double() - b).norm() / b.norm())
        assert d <= 10 * 2.0 ** -8, (what, d)

    near(y, out.detach(), "y")
    near(dx, gx, "dx")
    near(dlogits, gl, "dlogits")
    assert bool((dx[~live] == 0).all()) and bool((dlogits[~live] == 0).all())
    assert abs(float(loss) - float(bal)) <= 1e-5 * float(bal)
