"""The bounded waits of moe_matmul, made to run out on purpose without any fault.

A test hook gives the barriers of a launch one arrival more than will ever come, at a stage's copies (1) or at its
products (2), and a short bound.  The waits run out, the launch records MOE_DEV_TIMEOUT, stores nothing and returns with
the context intact.  With the hook off and the workspace zero-filled the next call is correct.
"""
import pytest
import torch

from test_gpu_matmul import check, product, rand, sorted_rows, workspace

moe = pytest.importorskip("quantized_routed_expert_router_gb300")

DEV = "cuda"

# few places (transposed: by tiles) and many, whole depth and in parts, one block a tile and two, more depth than the ring and less
SIZES = [(33, 272, 4096), (40, 7168, 200), (100, 400, 4096), (600, 1000, 4096), (100, 4000, 1024), (2500, 1040, 400), (4000, 2048, 1024)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hold", [1, 2])
def test_waits_run_out_then_recovery(M, N, K, gathered, dtype, hold):
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    x, w = rand(M, K, g=g), rand(2, N, K, g=g, scale=K ** -0.5)
    st, kw = workspace(), {}
    if gathered:
        offs, rows = sorted_rows((M // 3, M - M // 3), M, g)
        kw = dict(offsets=offs, rows=rows)
    else:
        w = w[0]
    y = torch.full((M, N), 7.0, dtype=dtype, device=DEV)
    torch.cuda.synchronize()
    try:
        moe.moe_debug_hold_matmul(hold, 1 << 17)
        moe.moe_matmul(x, w, y, st, **kw)
        torch.cuda.synchronize()
    finally:
        moe.moe_debug_hold_matmul(0)
    assert moe.moe_read_device_status(st, clear=False) == moe.DEV_TIMEOUT
    assert bool((y == 7.0).all())
    st.zero_()
    moe.moe_matmul(x, w, y, st, **kw)
    assert moe.moe_read_device_status(st) == 0
    if gathered:
        for e in range(2):
            a, b = int(offs[e]), int(offs[e + 1])
            check(y[a:b], *product(x[rows[a:b].long()], w[e]))
    else:
        check(y, *product(x, w))


@pytest.mark.gpu
def test_few_rows_wait_for_nothing_unless_transposed():
    g = torch.Generator(device=DEV).manual_seed(3)
    x, w = rand(16, 1024, g=g), rand(136, 1024, g=g, scale=1024 ** -0.5)
    y, st = torch.full((16, 136), 7.0, device=DEV), workspace()
    try:
        moe.moe_debug_hold_matmul(1, 1 << 17)
        moe.moe_matmul(x, w, y, st)
        torch.cuda.synchronize()
        check(y, *product(x, w))
        assert moe.moe_read_device_status(st) == 0
        y.fill_(7.0)
        moe.moe_matmul(x, w.t().contiguous(), y, st, transposed=True)
        torch.cuda.synchronize()
    finally:
        moe.moe_debug_hold_matmul(0)
    assert moe.moe_read_device_status(st) == moe.DEV_TIMEOUT and bool((y == 7.0).all())


def test_the_hook_refuses_what_it_does_not_know():
    for hold, cycles in ((-1, 0), (3, 0), (1, -1)):
        with pytest.raises(moe.MoeError):
            moe.moe_debug_hold_matmul(hold, cycles)
    moe.moe_debug_hold_matmul(0)
