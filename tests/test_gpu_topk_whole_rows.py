"""moe_topk's softmax over all experts, many rows a launch, on rows that are masked, tied or not finite.

Ids have to be equal, and to those of calls of a few rows.  Weights by test_gpu_topk's tolerance; a NaN or +inf in a row
makes all its weights NaN, and a slot without an expert has 0."""
import pytest
import torch

from test_gpu_topk import DEV, MANY, TINY, awkward, order, weights_of

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("quantized_routed_expert_router_gb300")


@pytest.mark.parametrize("E,k", [(256, 8), (256, 5), (128, 8), (60, 6), (32, 8), (512, 8), (400, 3), (144, 8), (512, 12)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("padded", [False, True])
def test_awkward_rows(E, k, dtype, padded):
    l = awkward(MANY, E, dtype)
    valid = None
    if padded:
        valid = torch.rand(MANY, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV) < 0.8
    ids = torch.full((MANY, k), 7, dtype=torch.int32, device=DEV)
    w = torch.full((MANY, k), 7.0, device=DEV)
    moe.moe_topk(l, moe.SOFTMAX, False, ids, w, valid=valid)
    want = order(l, k)
    if padded:
        want = torch.where(valid[:, None], want, -1)
    assert torch.equal(ids.long(), want)
    few = torch.empty_like(ids)
    for t in range(0, MANY, 1000):
        to = min(t + 1000, MANY)
        moe.moe_topk(l[t:to], moe.SOFTMAX, False, few[t:to], valid=valid[t:to] if padded else None)
    assert torch.equal(few, ids)
    live = want >= 0
    odd = (torch.isnan(l) | (l == float("inf"))).any(1, keepdim=True)
    assert bool((w[~live] == 0).all())
    assert bool(torch.isnan(w[live & odd]).all()) and not bool(torch.isnan(w[~(live & odd)]).any())
    ww, rel = weights_of(l, want, moe.SOFTMAX, False)[:2]
    off = (w.double() - ww).abs() <= rel * ww + TINY
    assert bool(off[live & ~odd].all())
