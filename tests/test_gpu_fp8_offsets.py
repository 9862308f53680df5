"""moe_fp8_matmul with offsets that fall: groups overlap, the call is flagged and writes nothing but the rows of y."""
import pytest
import torch

from test_gpu_fp8_matmul import check, definition, matrices, states, workspace

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("quantized_routed_expert_router_gb300")

DEV = "cuda"


# groups that take all rows in turn with groups that take none: G / 2 times the tiles of rising offsets.  All groups have
# one matrix, so whichever is last in a row leaves the same.
@pytest.mark.parametrize("G,M", [(1024, 700), (64, 2000), (1024, 12)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_offsets_that_fall_over_and_over(G, M, dtype):
    N, K = 136, 272
    g = torch.Generator(device=DEV).manual_seed(G + M)
    x, xs = states(M, K, g)
    w, ws = matrices(1, N, K, g)
    offs = torch.zeros(G + 1, dtype=torch.int32, device=DEV)
    offs[1::2] = M
    room, st = torch.full((M + 2, N), 7.0, dtype=dtype, device=DEV), workspace()
    y = room[1:M + 1]
    moe.moe_fp8_matmul(x, xs, w.expand(G, N, K).contiguous(), ws.expand(G, *ws.shape[1:]).contiguous(), y, st, offsets=offs)
    assert moe.moe_read_device_status(st) == moe.DEV_BAD_ROW
    assert bool((room[0] == 7.0).all()) and bool((room[M + 1] == 7.0).all())
    check(y, *definition(x, xs, w[0], ws[0]), K)
