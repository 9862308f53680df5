"""A row of moe_add_rmsnorm has the same bits in a batch of any size.

Rows are laid out over a block in three ways, by the number of rows and their width; the sums of squares are added in
one order in all of them.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("quantized_routed_expert_router_gb300")

DEV = "cuda"


def outputs(x, r, w, eps=1e-6):
    T, n = x.shape
    o = dict(residual_out=torch.empty_like(x), y=torch.empty(T, n, device=DEV),
             x8=torch.empty(T, n, dtype=torch.uint8, device=DEV), x8_scale=torch.empty(T, -(-n // 128), device=DEV))
    if n % 32 == 0:
        o["xq"] = torch.zeros(T * moe.moe_q8_row_bytes(n), dtype=torch.uint8, device=DEV)
    moe.moe_add_rmsnorm(x, r, w, eps, **o)
    if n % 32 == 0:
        o["xq"] = o["xq"].view(T, -1)
    return o


# widths of one chunk of 256 to 64, whole and ragged; batches on both sides of a row an SM
@pytest.mark.parametrize("n", [256, 2880, 4096, 4112, 5120, 7168, 8192, 8208, 10000, 16384])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_row_does_not_see_how_many_there_are(n, dtype):
    g = torch.Generator(device=DEV).manual_seed(n)
    T = 700
    x = torch.randn(T, n, generator=g, device=DEV)
    x[:, n // 5] *= 40
    x, r = x.to(dtype), torch.randn(T, n, generator=g, device=DEV).to(dtype)
    w = torch.rand(n, generator=g, device=DEV) + 0.5
    want = outputs(x, r, w)
    for a, b in ((0, 1), (5, 21), (100, 240), (3, 403)):
        got = outputs(x[a:b].contiguous(), r[a:b].contiguous(), w)
        for name, v in got.items():
            assert torch.equal(v, want[name][a:b]), (name, a, b)
