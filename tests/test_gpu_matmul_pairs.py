"""moe_matmul on tiles that two blocks share: gathered rows and rows in order, many launches one behind the other.

A value that one block took before the other had it there would differ from launch to launch; equal calls give equal bits."""
import pytest
import torch

from test_gpu_matmul import GRADS, check, finished, product, rand, run_dense, sorted_rows, workspace

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


# more tiles than pairs of blocks, so that a block takes several, and more depth than two running sums; ragged in M, N and K
LARGE = [(4100, 1552, 1608), (4100, 1552, 264), (1000, 1536, 4096)]


@pytest.mark.parametrize("M,N,K", LARGE)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", range(7))
@pytest.mark.parametrize("more", [False, True])
def test_epilogues(M, N, K, dtype, act, more):
    """Every activation with everything that may go with it, as on small tiles."""
    grad = act in GRADS
    run_dense(M, N, K, act, dtype, transposed=grad and not more, bias=more and not grad,
              residual="in place" if more and not grad else None if grad else "own",
              keep=("in place" if more else True) if grad else more and act != moe.ACT_NONE)


@pytest.mark.parametrize("N", [1543, 1545, 1552])
@pytest.mark.parametrize("act", [moe.ACT_NONE, moe.ACT_SILU, moe.ACT_GELU_GRAD])
def test_rows_that_start_anywhere(N, act):
    """Rows of fp32 results off 16-byte boundaries, their residual and z too."""
    run_dense(3000, N, 1992, act, F32, residual="in place" if act not in GRADS else None, bias=act not in GRADS,
              keep="in place" if act in GRADS else act != moe.ACT_NONE, seed=N)


@pytest.mark.parametrize("counts,N,K", GROUPS)
@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", range(7))
def test_groups(counts, N, K, gathered, dtype, act):
    """With a residual, or z, in place; transposed where the gradient is taken and nothing is gathered."""
    grad, total = act in GRADS, sum(counts)
    g = torch.Generator(device=DEV).manual_seed(total + act)
    x = rand(500 if gathered else total, K, g=g)
    offs, rows = sorted_rows(counts, x.shape[0], g)
    rows = torch.cat([rows, rows.new_full((3,), -1)]) if gathered else None
    if not gathered:
        x = torch.cat([x, x.new_full((3, K), float("nan"))])
    G, wide = len(counts), 2 * N if act == moe.ACT_SWIGLU else N
    w = rand(G, wide, K, g=g, scale=1.5 * K ** -0.5)
    for e, c in enumerate(counts):
        if c == 0:
            w[e] = float("nan")
    transposed = grad and not gathered
    b = None if grad else 0.5 * torch.randn(G, wide, generator=g, device=DEV)
    y = torch.randn(total + 3, 2 * N if act == moe.ACT_SWIGLU_GRAD else N, generator=g, device=DEV).to(dtype)
    start, z, r = y.clone(), None, None
    if grad:
        z = y
    else:
        r = y
        if act != moe.ACT_NONE:
            z = torch.full((total + 3, wide), 7.0, dtype=dtype, device=DEV)
    st = workspace()
    moe.moe_matmul(x, w.transpose(1, 2).contiguous() if transposed else w, y, st, act=act, bias=b, residual=r, z=z,
                   offsets=offs, rows=rows, transposed=transposed)
    for e, c in enumerate(counts):
        p, q = int(offs[e]), int(offs[e + 1])
        if c:
            v, tol = product(x[rows[p:q].long()] if gathered else x[p:q], w[e], None if b is None else b[e])
            check(y[p:q], *finished(act, v, tol, start[p:q] if grad else None, None if grad else start[p:q]))
            if z is not None and not grad:
                check(z[p:q], v, tol)
    assert torch.equal(y[total:], start[total:])
    if z is not None and not grad:
        assert bool((z[total:] == 7.0).all())
    assert moe.moe_read_device_status(st) == 0


@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hold", [1, 2])
def test_waits_over_many_groups_run_out_then_recovery(gathered, dtype, hold):
    """Tiles of 128 places that two blocks share: a barrier that never completes ends the call with a status."""
    counts, N, K = GROUPS[1]
    M = sum(counts)
    g = torch.Generator(device=DEV).manual_seed(11)
    x, w = rand(M, K, g=g), rand(len(counts), N, K, g=g, scale=K ** -0.5)
    offs, rows = sorted_rows(counts, M, g)
    rows = rows if gathered else None
    y, st = torch.full((M, N), 7.0, dtype=dtype, device=DEV), workspace()
    torch.cuda.synchronize()
    try:
        moe.moe_debug_hold_matmul(hold, 1 << 17)
        moe.moe_matmul(x, w, y, st, offsets=offs, rows=rows)
        torch.cuda.synchronize()
    finally:
        moe.moe_debug_hold_matmul(0)
    assert moe.moe_read_device_status(st, clear=False) == moe.DEV_TIMEOUT
    assert bool((y == 7.0).all())
    st.zero_()
    moe.moe_matmul(x, w, y, st, offsets=offs, rows=rows)
    assert moe.moe_read_device_status(st) == 0
    for e, c in enumerate(counts):
        p, q = int(offs[e]), int(offs[e + 1])
        if c:
            check(y[p:q], *product(x[rows[p:q].long()] if gathered else x[p:q], w[e]))
