"""From hidden states to the experts' rows for any number of tokens, as README.md's first run of calls has it with a router
in bf16: norm -> router's product -> top-k -> order -> rows.

The normed state is bf16 (2^-8 of itself at most); logits are computed from it as it is stored, so they are held to the
bound that moe.h states for fp32 results, 1e-6 in the norm.  What follows is decided on the logits as they are."""
import pytest
import torch

from test_gpu_topk import order, weights_of

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("quantized_routed_expert_router_gb300")

DEV = "cuda"
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


@pytest.mark.parametrize("T,H,E,k", [(1, 256, 16, 2), (17, 2048, 128, 8), (40, 512, 60, 4), (1000, 2880, 32, 4)])
def test_routing_of_any_number_of_tokens(T, H, E, k):
    g = torch.Generator(device=DEV).manual_seed(T)
    new = lambda *s, dtype: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731
    x = torch.randn(T, H, generator=g, device=DEV).to(BF16)
    residual = torch.randn(T, H, generator=g, device=DEV).to(BF16)
    norm_w = 1 + 0.1 * torch.randn(H, generator=g, device=DEV)
    w_r = (H ** -0.5 * torch.randn(E, H, generator=g, device=DEV)).to(BF16)
    hidden, logits = new(T, H, dtype=BF16), new(T, E, dtype=F32)
    ids, weights, pos = new(T, k, dtype=I32), new(T, k, dtype=F32), new(T, k, dtype=I32)
    offsets, rows, xs = new(E + 1, dtype=I32), new(T * k, dtype=I32), new(T * k, H, dtype=BF16)
    ws_m = new(moe.moe_matmul_workspace_bytes(), dtype=torch.uint8)
    ws_o = new(max(16, moe.moe_expert_order_workspace_bytes(T, k, E)), dtype=torch.uint8)
    s = x.double() + residual.double()
    moe.moe_add_rmsnorm(x, residual, norm_w, 1e-6, residual_out=residual, y=hidden)
    moe.moe_matmul(hidden, w_r, logits, ws_m)
    moe.moe_topk(logits, moe.SOFTMAX, True, ids, weights)
    moe.moe_expert_order(ids, E, ws_o, offsets=offsets, rows=rows, pos=pos)
    moe.moe_dispatch_rows(hidden, pos, xs)
    assert moe.moe_read_device_status(ws_m) == 0
    want = s * torch.rsqrt((s * s).mean(1, keepdim=True) + 1e-6) * norm_w.double()
    # the statistics are fp32's: far below the rounding
    assert bool(((hidden.double() - want).abs() <= want.abs() * 2.0 ** -8 * 1.01 + 1e-30).all())
    want = hidden.double() @ w_r.double().t()
    assert float((logits.double() - want).norm() / want.norm()) <= 1e-6
    top = order(logits, k)
    assert torch.equal(ids.long(), top)
    ww, rel = weights_of(logits, top, moe.SOFTMAX, True)[:2]
    assert bool(((weights.double() - ww).abs() <= rel * ww).all())
    assert int(offsets[E]) == T * k and torch.equal(xs, hidden[rows.long()])
    assert torch.equal(xs[pos.long().view(-1)], hidden.repeat_interleave(k, 0))
