"""The balance loss over millions of rows, compared with the definition in 64 bits.

All rows are alike and the router has collapsed: the sum over the rows then adds one number again and again, whose
roundings share a sign, so a plain fp32 sum of thousands of rows is off by hundreds of u (u = 2^-24).

Tolerance, in u of sum_e p |d|, for 8 experts, one value a lane: exp is off by 4 and by |l - m| through its argument, a
row's sums add 2 values a lane and take 5 steps, for the sum of p and for that of p d; the inverse and the product are
1 each, d is 4; a warp's rows are added with each rounding carried over to the next: 2, and 1 to join the two.  The
loss itself is rounded once and its factor is alpha's and the counts' in double: 2 of the loss.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("quantized_routed_expert_router_gb300")

U = 2.0 ** -24
DEV = "cuda"


@pytest.mark.parametrize("top", [2.0, 2.5, 2.75, 3.5, 4.5, 5.0])
@pytest.mark.parametrize("gating", ["softmax", "sigmoid"])
def test_loss_of_many_equal_rows(top, gating):
    T, E, k, alpha = 1 << 24, 8, 1, 0.01
    row = torch.zeros(E)
    row[2] = top if gating == "softmax" else top - 6.0       # (all below 0: the largest logit is factored out)
    if gating == "sigmoid":
        row[row == 0] = -6.0
    counts = torch.zeros(E, dtype=torch.int32, device=DEV)
    counts[2] = T * k
    logits = row.to(DEV).expand(T, E).contiguous()
    loss = torch.full((1,), 7.0, device=DEV)
    ws = torch.zeros(moe.moe_balance_loss_workspace_bytes(T, E), dtype=torch.uint8, device=DEV)
    moe.moe_balance_loss(logits, counts, k, moe.SOFTMAX if gating == "softmax" else moe.SIGMOID, alpha, ws, loss=loss)
    l = row.double()
    p = torch.softmax(l if gating == "softmax" else torch.nn.functional.logsigmoid(l), 0)
    d = counts.cpu().double() * E / (T * k) - 1
    q, spread, far = float((p * d).sum()), float((p * d.abs()).sum()), float((l.max() - l).max())
    want = alpha * k / (T * k) * T * (1 + q)
    # (sigmoid: a second exp and a reciprocal a value, 4 + 1 + 2 more)
    each = 2 * (4 + far + 7 + (7 if gating == "sigmoid" else 0)) + 2 + 4 + 3
    tol = alpha * spread * each * U + 2 * U * abs(want)
    assert abs(float(loss) - want) <= tol, ((float(loss) - want) / (alpha * spread * U), each)
