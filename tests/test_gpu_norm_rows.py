"""moe_add_rmsnorm against the definition in 64 bits.

Tolerances count roundings (u = 2^-24, half a step of fp32).  s = x + residual is one rounding.  The sum of
squares adds at most 32 squares a lane and two butterflies of 5 steps, each square carries 3 u (two from s, one
of its own), the mean 2 u, eps 1 u: 48 u at most, all terms being positive; the square root halves that and adds
1 u, the division 1 u, the two products 1 u each and s its own 1 u: v is off by at most 29 u of itself.  The
rounding of an output in bf16 adds 2^-8 of it, one in e4m3 2^-4 of the code (2^-10 below the smallest normal
code, whose step is 2^-9); scales are v's error and one division.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("quantized_routed_expert_router_gb300")

U = 2.0 ** -24
V_TOL = 29 * U
DEV = "cuda"


def make(T, n, dtype, seed, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, n, generator=g)
    x[:, n // 3] *= 30.0                       # an outlier channel
    if T > 1:
        x[T // 2] *= 1e-3                      # a quiet row
    r = torch.randn(T, n, generator=g) * 2 if residual else None
    w = 1 + 0.3 * torch.randn(n, generator=g)
    cast = lambda t: None if t is None else t.to(dtype).to(DEV)  # noqa: E731
    return cast(x), cast(r), w.to(DEV)


def definition(x, r, w, eps):
    s = x.double() if r is None else x.double() + r.double()
    return s, s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * w.double()


def groups(v):
    T, n = v.shape
    kb = -(-n // 128)
    pad = torch.zeros(T, kb * 128, dtype=v.dtype, device=v.device)
    pad[:, :n] = v
    return pad.reshape(T, kb, 128)


def check_rows8(x8, scale, v):
    T, n = v.shape
    amax = groups(v).abs().amax(2)
    want = amax / 448
    assert bool(((scale.double() - want).abs() <= (V_TOL + U) * want).all())
    q = (groups(v) * torch.where(amax > 0, 448 / amax, 0)[:, :, None]).reshape(T, -1)[:, :n]
    got = x8.view(torch.float8_e4m3fn).float().double()
    # the code's rounding, then v's and the inverse's error moved through it
    tol = torch.clamp(q.abs() * 2.0 ** -4, min=2.0 ** -10) + q.abs() * (2 * V_TOL + 3 * U)
    assert bool(((got - q).abs() <= tol).all()), float(((got - q).abs() - tol).max())


# widths: one chunk and less, ragged groups, odd chunk counts, the widest; tokens on both sides of the
# rule that lays out few and many rows
@pytest.mark.parametrize("T,n", [(1, 16), (3, 32), (5, 112), (1, 128), (2, 144), (7, 256), (1, 2880), (33, 2880),
                                 (1, 4096), (300, 528), (1, 7168), (200, 7168), (153, 2048), (1, 8208), (160, 8208),
                                 (2, 16384), (200, 16384), (400, 4112)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_against_the_definition(T, n, dtype):
    x, r, w = make(T, n, dtype, 7 * T + n)
    s64, v64 = definition(x, r, w, 1e-6)
    out, y = torch.empty_like(x), torch.empty_like(x)
    x8 = torch.empty(T, n, dtype=torch.float8_e4m3fn, device=DEV)
    sc = torch.empty(T, -(-n // 128), device=DEV)
    moe.moe_add_rmsnorm(x, r, w, 1e-6, residual_out=out, y=y, x8=x8, x8_scale=sc)
    assert torch.equal(out, (x.float() + r.float()).to(dtype))
    round_y = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    assert bool(((y.double() - v64).abs() <= (V_TOL + round_y * (1 + V_TOL)) * v64.abs() + 1e-37).all())
    check_rows8(x8, sc, v64)


@pytest.mark.parametrize("T,n", [(1, 2048), (16, 4096), (5, 2880), (300, 2880), (1, 7168), (200, 96)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_q8_records_are_those_of_the_quantiser(T, n, dtype):
    x, r, w = make(T, n, dtype, T + n)
    y = torch.empty(T, n, device=DEV)
    size = T * moe.moe_q8_row_bytes(n)
    xq = torch.zeros(size, dtype=torch.uint8, device=DEV)
    moe.moe_add_rmsnorm(x, r, w, 1e-5, y=y, xq=xq)
    want = torch.zeros(size, dtype=torch.uint8, device=DEV)
    moe.moe_quantize_q8K(y, want)
    assert torch.equal(xq, want)


def test_without_residual_and_single_outputs():
    x, _, w = make(4, 400, torch.bfloat16, 3)
    _, v64 = definition(x, None, w, 1e-6)
    y = torch.empty(4, 400, device=DEV)          # bf16 in, fp32 out: what an fp32 router reads
    moe.moe_add_rmsnorm(x, None, w, 1e-6, y=y)
    assert bool(((y.double() - v64).abs() <= V_TOL * v64.abs() + 1e-37).all())
    yb = torch.empty(4, 400, dtype=torch.bfloat16, device=DEV)
    moe.moe_add_rmsnorm(x.float(), None, w, 1e-6, y=yb)
    assert torch.equal(yb, y.to(torch.bfloat16))
    x8 = torch.empty(4, 400, dtype=torch.uint8, device=DEV)
    sc = torch.empty(4, 4, device=DEV)
    moe.moe_add_rmsnorm(x, None, w, 1e-6, x8=x8, x8_scale=sc)
    check_rows8(x8, sc, v64)
    out = torch.empty_like(x)
    moe.moe_add_rmsnorm(x, x, w, 1e-6, residual_out=out)
    assert torch.equal(out, (x.float() * 2).to(x.dtype))


@pytest.mark.parametrize("which", ["x", "residual"])
def test_residual_out_in_place(which):
    x, r, w = make(170, 2880, torch.bfloat16, 11)
    want = torch.empty_like(x)
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    moe.moe_add_rmsnorm(x, r, w, 1e-6, residual_out=want, y=y)
    moe.moe_add_rmsnorm(x, r, w, 1e-6, residual_out=x if which == "x" else r, y=y2)
    assert torch.equal(x if which == "x" else r, want) and torch.equal(y, y2)


def test_zero_rows_tiny_groups_and_equal_magnitudes():
    n = 384
    x = torch.zeros(4, n, device=DEV)
    x[1, :128] = 1e-30                    # v is about 1e-27 / sqrt(eps): far above the floor, far below 1
    x[2, 200] = 5.0                       # one value: its group holds +-448, the others nothing
    x[3] = -2.0
    w = torch.ones(n, device=DEV)
    w[300:] = 1e-38                       # a group of v below the floor of the scale
    x8 = torch.empty(4, n, dtype=torch.float8_e4m3fn, device=DEV)
    sc = torch.empty(4, 3, device=DEV)
    y = torch.empty_like(x)
    moe.moe_add_rmsnorm(x, None, w, 1e-6, y=y, x8=x8, x8_scale=sc)
    c = x8.float()
    assert bool((c[0] == 0).all()) and bool((sc[0] == 0).all()) and bool((y[0] == 0).all())
    assert bool((c[1, :128] == 448).all()) and float(sc[1, 1]) == 0.0
    assert float(c[2, 200]) == 448 and int((c[2] != 0).sum()) == 1
    assert bool((c[3, :256] == -448).all())
    assert float(sc[3, 2]) > 0 and bool((c[3, 256:300] == -448).all()) and bool((c[3, 300:] == 0).all())
    w[256:] = 1e-38
    moe.moe_add_rmsnorm(x, None, w, 1e-6, x8=x8, x8_scale=sc)
    assert float(sc[3, 2]) == 0.0 and bool((x8.float()[3, 256:] == 0).all())
    assert bool(torch.isfinite(x8.float()).all())


def test_rows_do_not_depend_on_their_neighbours_and_none_are_written_beyond():
    x, r, w = make(9, 2880, torch.float32, 5)
    y = torch.full((12, 2880), 7.0, device=DEV)
    moe.moe_add_rmsnorm(x, r, w, 1e-6, y=y[:9])
    assert bool((y[9:] == 7.0).all())
    one = torch.empty(1, 2880, device=DEV)
    moe.moe_add_rmsnorm(x[4:5], r[4:5], w, 1e-6, y=one)
    assert torch.equal(one[0], y[4])
    moe.moe_add_rmsnorm(x[:0], r[:0], w, 1e-6, y=y[:0])       # no rows: a no-op


def test_captured_and_on_another_stream():
    x, r, w = make(20, 4096, torch.bfloat16, 6)
    y, want = torch.empty_like(x), torch.empty_like(x)
    moe.moe_add_rmsnorm(x, r, w, 1e-6, y=want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_add_rmsnorm(x, r, w, 1e-6, y=y, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_add_rmsnorm(x, r, w, 1e-6, y=y)
    x.copy_(x * 2)
    moe.moe_add_rmsnorm(x, r, w, 1e-6, y=want)
    y.zero_()
    g.replay()
    assert torch.equal(y, want)


def test_a_stream_is_a_stream():
    x, r, w = make(2, 64, torch.float32, 1)
    y = torch.full_like(x, 7.0)
    with pytest.raises(AttributeError):
        moe.moe_add_rmsnorm(x, r, w, 1e-6, y=y, stream=5)
    assert bool((y == 7.0).all())


def test_refusals_leave_outputs_alone():
    x, r, w = make(2, 64, torch.float32, 1)
    y = torch.full_like(x, 7.0)
    with pytest.raises(moe.MoeError):
        moe.moe_add_rmsnorm(x, r, w, 1e-6)                                   # no output
    with pytest.raises(moe.MoeError):
        moe.moe_add_rmsnorm(x, r, w, -1.0, y=y)
    with pytest.raises(moe.MoeError):
        moe.moe_add_rmsnorm(x, r, w, 1e-6, y=y, x8=torch.empty(2, 64, dtype=torch.uint8, device=DEV))
    with pytest.raises(moe.MoeError):                                        # 8-byte aligned rows
        moe.moe_add_rmsnorm(torch.zeros(130, device=DEV)[2:].view(2, 64), r, w, 1e-6, y=y)
    for bad in (dict(y=y.half()), dict(y=y[:1]), dict(y=y.cpu()), dict(y=torch.empty(64, 2, device=DEV).t())):
        with pytest.raises(ValueError):
            moe.moe_add_rmsnorm(x, r, w, 1e-6, **bad)
    with pytest.raises(ValueError):
        moe.moe_add_rmsnorm(x, r.bfloat16(), w, 1e-6, y=y)
    assert bool((y == 7.0).all())


@pytest.mark.parametrize("n", [16, 400, 7168])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_keep_nan(n, bad):
    """a NaN in x (a NaN or infinity once normed) shows in y and in the e4m3 row's scale and codes; other rows stay"""
    x, r, w = make(5, n, torch.float32, 3)
    out = [torch.empty(5, n, device=DEV), torch.empty(5, n, dtype=torch.uint8, device=DEV),
           torch.empty(5, -(-n // 128), device=DEV)]
    moe.moe_add_rmsnorm(x, r, w, 1e-6, y=out[0], x8=out[1], x8_scale=out[2])
    want = [o.clone() for o in out]
    x[3, n // 2] = bad
    moe.moe_add_rmsnorm(x, r, w, 1e-6, y=out[0], x8=out[1], x8_scale=out[2])
    keep = [0, 1, 2, 4]
    assert all(torch.equal(o[keep], v[keep]) for o, v in zip(out, want))
    # an infinity makes the others 0 and itself NaN
    g = n // 2 // 128
    assert bool(torch.isnan(out[0][3, n // 2])) and bool(torch.isnan(out[2][3, g]))
    assert bool(((out[1][3, 128 * g:128 * g + 128] & 0x7F) == 0x7F).all())
    if bad != bad:
        assert bool(torch.isnan(out[0][3]).all()) and bool(torch.isnan(out[2][3]).all())


def test_rows_beyond_32_bits():
    T, n = 140000, 16384
    x = torch.empty(T, n, dtype=torch.bfloat16, device=DEV).normal_()
    w = torch.rand(n, device=DEV) + 0.5
    y, x8 = torch.empty_like(x), torch.empty(T, n, dtype=torch.uint8, device=DEV)
    scale = torch.empty(T, n // 128, device=DEV)
    moe.moe_add_rmsnorm(x, None, w, 1e-6, y=y, x8=x8, x8_scale=scale)
    for a in (slice(0, 3), slice(T // 2, T // 2 + 3), slice(T - 3, T)):
        _, v = definition(x[a], None, w, 1e-6)
        assert bool(((y[a].double() - v).abs() <= v.abs() * (2.0 ** -8 * 1.01 + V_TOL)).all())
        check_rows8(x8[a], scale[a], v)
