"""The bounded waits of moe_fp8_matmul's tiles, made to run out on purpose without any fault.

A test hook gives the barriers of a launch one arrival more than will ever come, at a stage's copies (1) or at its
products (2), and a short bound.  The waits run out, the launch records MOE_DEV_TIMEOUT, stores nothing and returns with
the context intact.  With the hook off and the workspace zero-filled the next call is correct.
"""
import pytest
import torch

from test_gpu_fp8_matmul import check, definition, matrices, sorted_rows, states, workspace

moe = pytest.importorskip("quantized_routed_expert_router_gb300")

DEV = "cuda"

# depth in parts with more blocks than stages and with fewer; tiles of 128 and of 192 columns, rows of y on a 16-byte
# boundary and off it, few and many blocks of depth
SIZES = [(200, 512, 8192), (64, 512, 4096), (2500, 400, 400), (2500, 403, 2000), (4000, 2048, 1024), (4000, 2051, 1024)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("hold", [1, 2])
def test_waits_run_out_then_recovery(M, N, K, gathered, hold):
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    x, xs = states(M, K, g)
    w, ws = matrices(2, N, K, g)
    st, kw = workspace(), {}
    if gathered:
        offs, rows = sorted_rows((M // 3, M - M // 3), M, g)
        kw = dict(offsets=offs, rows=rows)
    else:
        w, ws = w[0], ws[0]
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    try:
        moe.moe_debug_hold_fp8_matmul(hold, 1 << 17)
        moe.moe_fp8_matmul(x, xs, w, ws, y, st, **kw)
        torch.cuda.synchronize()
    finally:
        moe.moe_debug_hold_fp8_matmul(0)
    assert moe.moe_read_device_status(st, clear=False) == moe.DEV_TIMEOUT
    assert bool((y == 7.0).all())
    st.zero_()
    moe.moe_fp8_matmul(x, xs, w, ws, y, st, **kw)
    assert moe.moe_read_device_status(st) == 0
    if gathered:
        for e in range(2):
            a, b = int(offs[e]), int(offs[e + 1])
            r = rows[a:b].long()
            check(y[a:b], *definition(x[r], xs[r], w[e], ws[e]), K)
    else:
        check(y, *definition(x, xs, w, ws), K)


@pytest.mark.gpu
def test_few_rows_wait_for_nothing():
    g = torch.Generator(device=DEV).manual_seed(3)
    x, xs = states(16, 1024, g)
    w, ws = matrices(1, 136, 1024, g)
    y, st = torch.empty(16, 136, device=DEV), workspace()
    try:
        moe.moe_debug_hold_fp8_matmul(1, 1 << 17)
        moe.moe_fp8_matmul(x, xs, w[0], ws[0], y, st)
        torch.cuda.synchronize()
    finally:
        moe.moe_debug_hold_fp8_matmul(0)
    check(y, *definition(x, xs, w[0], ws[0]), 1024)
    assert moe.moe_read_device_status(st) == 0


def test_the_hook_refuses_what_it_does_not_know():
    for hold, cycles in ((-1, 0), (3, 0), (1, -1)):
        with pytest.raises(moe.MoeError):
            moe.moe_debug_hold_fp8_matmul(hold, cycles)
    moe.moe_debug_hold_fp8_matmul(0)
