"""moe_matmul against the definition in 64 bits.

Tolerance.  Products of two bf16 values are exact in fp32.  An instruction of the tensor cores adds 16 of them to the
running sum, 17 addends held to 24 bits below the largest: each loses at most 2^-23 of it, and no addend is larger than
the running sum before or after or the sum of magnitudes of the 16.  Running sums are differences of the depth's prefix
sums P (a split depth starts anew), so over the K / 16 instructions v is off by
17 * 2^-23 * (2 * ceil(K / 16) * max|P| + mag), mag the sum of all magnitudes, and by 8 roundings more for the parts and
the bias.  An activation multiplies that by its largest slope (silu 1.1, gelu 1.13; its own arithmetic: 16 units of 2^-24),
y is rounded to its type (bf16 2^-8).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("quantized_routed_expert_router_gb300")

DEV = "cuda"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8 * 1.01}
GATED = (moe.ACT_SWIGLU, moe.ACT_SWIGLU_GRAD)
GRADS = (moe.ACT_SILU_GRAD, moe.ACT_GELU_GRAD, moe.ACT_SWIGLU_GRAD)


def product(x, w, bias=None):
    """x [M, K] by w [N, K] in 64 bits, and what a fp32 sum may be off by"""
    x, w = x.double(), w.double()
    M, K = x.shape
    v = torch.zeros(M, w.shape[0], dtype=torch.float64, device=DEV)
    top = torch.zeros_like(v)
    for k in range(0, K, 16):
        v += x[:, k:k + 16] @ w[:, k:k + 16].t()
        top = torch.maximum(top, v.abs())
    mag = x.abs() @ w.abs().t()
    tol = 17 * 2.0 ** -23 * (2 * -(-K // 16) * top + mag)
    if bias is not None:
        v = v + bias.double()
    return v, tol + 8 * U * (v.abs() + top)


def slope(act, z):
    z = z.double().requires_grad_(True)
    f = torch.nn.functional.silu if act == moe.ACT_SILU_GRAD else torch.nn.functional.gelu
    return torch.autograd.grad(f(z).sum(), z)[0]


def finished(act, v, tol, z=None, residual=None):
    """y and its tolerance before the rounding to its type"""
    f = torch.nn.functional
    N = v.shape[1] // 2
    if act == moe.ACT_NONE:
        y = v
    elif act in (moe.ACT_SILU, moe.ACT_GELU):
        y = f.silu(v) if act == moe.ACT_SILU else f.gelu(v)
        tol = 1.13 * tol + 16 * U * v.abs()
    elif act == moe.ACT_SWIGLU:
        g, u, tg, tu = v[:, :N], v[:, N:], tol[:, :N], tol[:, N:]
        y = f.silu(g) * u
        tol = 1.1 * tg * (u.abs() + tu) + f.silu(g).abs() * tu + 20 * U * g.abs() * u.abs()
    elif act == moe.ACT_SWIGLU_GRAD:
        n = v.shape[1]
        g, u = z[:, :n].double(), z[:, n:].double()
        s, d = f.silu(g), slope(moe.ACT_SILU_GRAD, z[:, :n])
        y = torch.cat([v * u * d, v * s], 1)
        # silu' is a sum of terms up to 1 + |g|
        tol = torch.cat([tol * u.abs() * 1.1 + v.abs() * u.abs() * (1 + g.abs()) * 20 * U,
                         tol * s.abs() + v.abs() * g.abs() * 20 * U], 1)
    else:
        d = slope(act, z)
        y = v * d
        tol = tol * 1.13 + v.abs() * (1 + z.double().abs()) * 20 * U
    if residual is not None:
        y = y + residual.double()
        tol = tol + U * (y.abs() + residual.double().abs())
    return y, tol


def check(y, want, tol):
    err = (y.double() - want).abs() - (tol + want.abs() * HALF[y.dtype] + 2.0 ** -126)
    assert bool((err <= 0).all()), (float(err.max()), float((y.double() - want).norm() / want.norm()))


def workspace():
    return torch.zeros(moe.moe_matmul_workspace_bytes(), dtype=torch.uint8, device=DEV)


def rand(*shape, g, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device=DEV)).to(BF16)


def run_dense(M, N, K, act, dtype, transposed=False, bias=False, residual=None, keep=False, seed=0):
    g = torch.Generator(device=DEV).manual_seed(M + 3 * N + K + act + seed)
    x = rand(M, K, g=g)
    wide = 2 * N if act == moe.ACT_SWIGLU else N
    w = rand(wide, K, g=g, scale=1.5 * K ** -0.5)
    b = 0.5 * torch.randn(wide, generator=g, device=DEV) if bias else None
    yn = 2 * N if act == moe.ACT_SWIGLU_GRAD else N
    room = torch.full((M * yn + 32,), 7.0, dtype=dtype, device=DEV)       # nothing is written on either side
    y = room[16:16 + M * yn].view(M, yn)
    r = None
    if residual:
        r = torch.randn(M, N, generator=g, device=DEV).to(dtype)
        if residual == "in place":
            y.copy_(r)
            r_in = y
        else:
            r_in = r
    z = z_in = None
    if act in GRADS:
        z = torch.randn(M, 2 * N if act in GATED else N, generator=g, device=DEV).mul(1.5).to(dtype)
        z_in = z
        if keep == "in place":
            y.copy_(z)
            z_in = y
    elif keep:
        z_in = torch.full((M, wide), 7.0, dtype=dtype, device=DEV)
    st = workspace()
    moe.moe_matmul(x, w.t().contiguous() if transposed else w, y, st, act=act, bias=b, residual=r_in if residual else None,
                   z=z_in, transposed=transposed)
    v, tol = product(x, w, b)
    check(y, *finished(act, v, tol, z, r))
    if keep and act not in GRADS:
        check(z_in, v, tol)
    assert bool((room[:16] == 7.0).all()) and bool((room[16 + M * yn:] == 7.0).all())
    assert moe.moe_read_device_status(st) == 0


# one row to many; widths and depths around tiles of 16, 64, 128 and 256; depths that are split and that are not
DENSE = [(1, 1, 8), (1, 16, 64), (1, 2048, 4096), (2, 7, 72), (3, 136, 4096), (5, 24, 40), (8, 200, 4112), (15, 2051, 1008),
         (16, 7168, 512), (17, 100, 1040), (31, 129, 136), (33, 130, 64), (40, 136, 8192), (64, 512, 1024), (65, 1000, 72),
         (100, 333, 2048), (127, 257, 272), (128, 128, 128), (129, 384, 640), (200, 1026, 4096), (255, 60, 24),
         (257, 300, 336), (300, 2880, 2880), (333, 4000, 256), (513, 129, 4000), (600, 1030, 4096), (400, 512, 8192), (1000, 1536, 4096), (2048, 2560, 272),
         (2500, 2051, 400), (4100, 1000, 1168)]


@pytest.mark.parametrize("M,N,K", DENSE)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_dense(M, N, K, dtype):
    run_dense(M, N, K, moe.ACT_NONE, dtype)


# every activation with everything that may go with it, at one row, few rows, a split depth, whole tiles, ragged ones
SHAPES = [(1, 48, 264), (4, 512, 2048), (21, 144, 4096), (130, 272, 200), (300, 2880, 288), (700, 528, 2056), (1100, 400, 136)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", range(7))
@pytest.mark.parametrize("more", [False, True])
def test_epilogues(M, N, K, dtype, act, more):
    grad = act in GRADS
    run_dense(M, N, K, act, dtype, transposed=grad and not more, bias=more and not grad,
              residual="in place" if more and not grad else None,
              keep=("in place" if more else True) if grad else more and act != moe.ACT_NONE)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", [moe.ACT_NONE, moe.ACT_SWIGLU])
def test_residual_and_bias_apart(M, N, K, act):
    run_dense(M, N, K, act, BF16, residual="own", seed=1)
    run_dense(M, N, K, act, F32, bias=True, seed=2)


@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (1, 4096, 1000), (3, 72, 200), (16, 1000, 2880), (20, 136, 4000),
                                   (100, 264, 72), (129, 1032, 8), (300, 512, 1160), (1000, 2880, 2880), (2500, 520, 400)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_transposed(M, N, K, dtype):
    run_dense(M, N, K, moe.ACT_NONE, dtype, transposed=True, bias=True)


def sorted_rows(counts, X, g):
    """offsets and random rows for these group sizes"""
    offs = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device=DEV)
    rows = torch.randint(0, X, (int(offs[-1]),), generator=g, device=DEV, dtype=torch.int32)
    return offs, rows


GROUPED = [((0, 9, 0, 4, 3), 320, 4112), ((0,) * 70 + (16,), 96, 208), ((1,), 16, 64), ((0, 3, 0, 1, 0), 112, 272),
           ((1, 1, 2, 1, 3), 256, 1024), ((128, 129, 0, 127), 384, 528), ((5, 0, 300, 1, 0, 0, 77, 260), 1008, 1040),
           ((700, 900, 0, 1300), 2064, 400), ((0,) * 40 + (2,), 144, 2048), (tuple(range(1, 60)), 272, 384),
           ((40, 33, 31, 64, 20, 0, 1), 512, 200), ((17,) * 30, 48, 72), ((256, 257, 1, 255), 144, 328)]


@pytest.mark.parametrize("counts,N,K", GROUPED)
@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("act", [moe.ACT_NONE, moe.ACT_SWIGLU, moe.ACT_SWIGLU_GRAD])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_grouped(counts, N, K, gathered, act, dtype):
    """Rows of no group, behind the last one, are NaN where they are read from and stay as they were where they are
    written to."""
    grad, total = act == moe.ACT_SWIGLU_GRAD, sum(counts)
    g = torch.Generator(device=DEV).manual_seed(len(counts) + N + K)
    x = rand(50 if gathered else total + 5, K, g=g)
    offs, rows = sorted_rows(counts, x.shape[0], g)
    if gathered:
        rows = torch.cat([rows, rows.new_full((5,), -1)])
    else:
        x[total:] = float("nan")
        rows = None
    G, wide = len(counts), 2 * N if act == moe.ACT_SWIGLU else N
    w = rand(G, wide, K, g=g, scale=1.5 * K ** -0.5)
    for e, c in enumerate(counts):
        if c == 0:
            w[e] = float("nan")                                 # matrices of no rows are not taken
    b = None if grad else 0.5 * torch.randn(G, wide, generator=g, device=DEV)
    yn = 2 * N if grad else N
    y = torch.full((total + 5, yn), 7.0, dtype=dtype, device=DEV)
    z = torch.randn(total + 5, 2 * N, generator=g, device=DEV).to(dtype) if grad else None
    if act == moe.ACT_SWIGLU:
        z = torch.full((total + 5, wide), 7.0, dtype=dtype, device=DEV)
    st = workspace()
    moe.moe_matmul(x, w.transpose(1, 2).contiguous() if grad else w, y, st, act=act, bias=b, z=z, offsets=offs, rows=rows,
                   transposed=grad)
    for e, c in enumerate(counts):
        p, q = int(offs[e]), int(offs[e + 1])
        if c:
            v, tol = product(x[rows[p:q].long()] if gathered else x[p:q], w[e], None if b is None else b[e])
            check(y[p:q], *finished(act, v, tol, z[p:q] if grad else None))
            if act == moe.ACT_SWIGLU:
                check(z[p:q], v, tol)
    assert bool((y[total:] == 7.0).all())
    if act == moe.ACT_SWIGLU:
        assert bool((z[total:] == 7.0).all())
    assert moe.moe_read_device_status(st) == 0


@pytest.mark.parametrize("M,N,K", [(3, 32, 72), (16, 144, 1032), (200, 528, 72), (1000, 1040, 136)])
@pytest.mark.parametrize("transposed", [False, True])
def test_values_past_the_ends_do_not_matter(M, N, K, transposed):
    """A NaN or infinity in one group's rows or matrix shows in that group's results alone, and in the rows and columns
    that it belongs to; depths, widths and groups end inside tiles."""
    g = torch.Generator(device=DEV).manual_seed(5)
    counts = (M // 3, M - M // 3 - 1, 1)
    offs, _ = sorted_rows(counts, 1, g)
    x, w = rand(M, K, g=g), rand(3, N, K, g=g, scale=K ** -0.5)

    def call(x, w):
        y, st = torch.empty(M, N, device=DEV), workspace()
        moe.moe_matmul(x, w.transpose(1, 2).contiguous() if transposed else w, y, st, offsets=offs, transposed=transposed)
        assert moe.moe_read_device_status(st) == 0
        return y

    clean = call(x, w)
    p, q = int(offs[1]), int(offs[2])
    for bad in (float("nan"), float("inf")):
        w2 = w.clone()
        w2[1] = bad
        y = call(x, w2)
        assert torch.equal(y[:p], clean[:p]) and torch.equal(y[q:], clean[q:])
        assert not bool(torch.isfinite(y[p:q]).any())
        w2 = w.clone()
        w2[0, N - 1, K - 1] = w2[2, 0, 0] = bad
        y = call(x, w2)
        assert torch.equal(y[:p, :N - 1], clean[:p, :N - 1]) and torch.equal(y[p:q], clean[p:q])
        assert torch.equal(y[q:, 1:], clean[q:, 1:]) and not bool(torch.isfinite(y[:p, N - 1]).any())
        x2 = x.clone()
        x2[p] = bad
        y = call(x2, w)
        keep = torch.arange(M, device=DEV) != p
        assert torch.equal(y[keep], clean[keep]) and not bool(torch.isfinite(y[p]).any())


def test_bad_rows_and_offsets_are_reported_and_not_followed():
    g = torch.Generator(device=DEV).manual_seed(6)
    for M, N, K in ((4, 64, 128), (300, 272, 200)):
        x, w = rand(10, K, g=g), rand(2, N, K, g=g)
        w[1, 0, 0] = float("inf")
        offs = torch.tensor([0, M // 2, M], dtype=torch.int32, device=DEV)
        rows = torch.randint(0, 10, (M,), generator=g, device=DEV, dtype=torch.int32)
        rows[1], rows[M - 1] = 10, -5
        r, b = torch.randn(M, N, generator=g, device=DEV), torch.randn(2, N, generator=g, device=DEV)
        y, st = torch.full((M, N), 7.0, device=DEV), workspace()
        moe.moe_matmul(x, w, y, st, offsets=offs, rows=rows, residual=r, bias=b)
        assert moe.moe_read_device_status(st) == moe.DEV_BAD_ROW
        for i, e in ((1, 0), (M - 1, 1)):                              # the product of such a row is 0
            want = b[e].double() + r[i].double()
            assert bool(((y[i].double() - want).abs() <= 2 * U * (want.abs() + b[e].abs())).all())
        ok = torch.ones(M // 2, dtype=torch.bool, device=DEV)
        ok[1] = False
        v, tol = product(x[rows[:M // 2][ok].long()], w[0], b[0])
        check(y[:M // 2][ok], *finished(moe.ACT_NONE, v, tol, residual=r[:M // 2][ok]))
        rows.clamp_(0, 9)
        for bad in ([0, M + 7, M], [-3, M // 2, M], [0, M, M // 2]):
            guard = torch.full((M + 64, N), 7.0, device=DEV)
            moe.moe_matmul(x, w, guard[:M], st, offsets=torch.tensor(bad, dtype=torch.int32, device=DEV), rows=rows)
            assert moe.moe_read_device_status(st) == moe.DEV_BAD_ROW
            assert bool((guard[M:] == 7.0).all())


def test_no_rows():
    g = torch.Generator(device=DEV).manual_seed(7)
    x, w, st = rand(4, 64, g=g), rand(3, 32, 64, g=g), workspace()
    y = torch.empty(0, 32, device=DEV)
    moe.moe_matmul(x, w, y, st, offsets=torch.zeros(4, dtype=torch.int32, device=DEV))
    y = torch.full((4, 32), 7.0, device=DEV)
    moe.moe_matmul(x, w, y, st, offsets=torch.zeros(4, dtype=torch.int32, device=DEV))     # every group empty
    moe.moe_matmul(x, w, y, st, offsets=torch.full((4,), 4, dtype=torch.int32, device=DEV))
    assert bool((y == 7.0).all()) and moe.moe_read_device_status(st) == 0


def test_equal_calls_give_equal_bits_on_streams_and_in_graphs():
    """Two captured graphs that share a workspace, replayed on two streams at once, and an eager call."""
    g = torch.Generator(device=DEV).manual_seed(8)
    st = workspace()
    for M, N, K in ((5, 512, 2048), (40, 144, 8192), (900, 1040, 272)):
        x, w = rand(M, K, g=g), rand(2 * N, K, g=g, scale=K ** -0.5)
        y = [torch.zeros(M, N, dtype=BF16, device=DEV) for _ in range(3)]
        moe.moe_matmul(x, w, y[2], st, act=moe.ACT_SWIGLU)
        torch.cuda.synchronize()
        graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
        for i in range(2):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[i]):
                moe.moe_matmul(x, w, y[i], st, act=moe.ACT_SWIGLU)
        torch.cuda.synchronize()
        for _ in range(3):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(y[0], y[2]) and torch.equal(y[1], y[2])
    assert moe.moe_read_device_status(st) == 0


def test_operands_past_32_bit_offsets():
    g = torch.Generator(device=DEV).manual_seed(9)
    K, N, M = 4096, 8192, (1 << 31) // 8192 + 77
    X = (1 << 31) // K + 5
    x = torch.zeros(X, K, dtype=BF16, device=DEV)
    x[-3:] = rand(3, K, g=g)
    w = rand(N, K, g=g, scale=K ** -0.5)
    rows = torch.zeros(M, dtype=torch.int32, device=DEV)
    rows[-3:] = torch.arange(X - 3, X, dtype=torch.int32, device=DEV)
    y, st = torch.full((M, N), 7.0, dtype=BF16, device=DEV), workspace()
    moe.moe_matmul(x, w, y, st, rows=rows, offsets=torch.tensor([0, M], dtype=torch.int32, device=DEV))
    check(y[-3:], *product(x[-3:], w))
    assert bool((y[:-3] == 0).all()) and moe.moe_read_device_status(st) == 0
    # many matrices: the last ones start past 2^31 values
    G = 80
    w = torch.zeros(G, N, K, dtype=BF16, device=DEV)
    w[-1] = rand(N, K, g=g, scale=K ** -0.5)
    offs = torch.zeros(G + 1, dtype=torch.int32, device=DEV)
    offs[-1] = 3
    for transposed in (False, True):
        y = torch.empty(3, N, device=DEV)
        wt = w.view(G, K, N) if transposed else w
        moe.moe_matmul(x[-3:], wt, y, st, offsets=offs, transposed=transposed)
        check(y, *product(x[-3:], wt[-1].t() if transposed else wt[-1]))
