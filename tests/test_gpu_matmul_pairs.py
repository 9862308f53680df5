"""moe_matmul on tiles that two blocks share: gathered rows and rows in order, many launches one behind the other.

A value that one block took before the other had it there would differ from launch to launch; equal calls give equal bits."""
import pytest
import torch

from test_gpu_matmul import check, finished, product, rand, sorted_rows, workspace

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("quantized_routed_expert_router_gb300")

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16

# group sizes, N, K: many places a group (tiles of 256) and about a hundred (of 128), several tiles a block, ragged
GROUPS = [((700, 900, 3, 1300, 0, 641), 2064, 1544), ((97, 0, 120, 101, 85, 97, 110, 64) * 4, 1040, 1160)]


@pytest.mark.parametrize("counts,N,K", GROUPS)
@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_launches_give_equal_bits(counts, N, K, gathered, dtype):
    M = sum(counts)
    g = torch.Generator(device=DEV).manual_seed(M + K)
    x, w = rand(M, K, g=g), rand(len(counts), N, K, g=g, scale=K ** -0.5)
    offs, rows = sorted_rows(counts, M, g)
    st, y = workspace(), torch.empty(M, N, dtype=dtype, device=DEV)
    moe.moe_matmul(x, w, y, st, offsets=offs, rows=rows if gathered else None)
    for e, c in enumerate(counts):
        p, q = int(offs[e]), int(offs[e + 1])
        if c:
            check(y[p:q], *finished(moe.ACT_NONE, *product(x[rows[p:q].long()] if gathered else x[p:q], w[e])))
    # other rows in between: what a stage held before is not what it is to hold
    x2, other = rand(M, K, g=g, scale=3.0), torch.empty_like(y)
    same, again = torch.ones((), dtype=torch.bool, device=DEV), torch.empty_like(y)
    for _ in range(100):
        moe.moe_matmul(x2, w, other, st, offsets=offs, rows=rows if gathered else None)
        moe.moe_matmul(x, w, again, st, offsets=offs, rows=rows if gathered else None)
        same &= (again == y).all()
    assert bool(same) and moe.moe_read_device_status(st) == 0
