"""moe_dispatch_rows, moe_combine_rows and moe_combine_grad against the definition in 64 bits.

Tolerances, u = 2^-24: rows that move are equal bit for bit.  A sum over the slots is a chain of fused additions, each
off by u of the sum of magnitudes.  A row of the gradient is one product (u); its dot with another row is a sum of at
most 8 ceil(n / 1024) additions in turn and 12 more.  What is stored in bf16 is rounded by 2^-8 of itself.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("quantized_routed_expert_router_gb300")

DEV = "cuda"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
TINY = 2.0 ** -126
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8 * 1.01}


def places(T, k, E, g, drop=0.0):
    """pos and how many places it fills"""
    ids = torch.rand(T, E, generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32).contiguous()
    if drop:
        ids[torch.rand(T, k, generator=g, device=DEV) < drop] = -1
    pos, offs = torch.empty_like(ids), torch.empty(E + 1, dtype=torch.int32, device=DEV)
    size = moe.moe_expert_order_workspace_bytes(T, k, E)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV) if size else None
    moe.moe_expert_order(ids, E, ws, offsets=offs, pos=pos)
    return pos, int(offs[E])


SIZES = [(1, 1, 1, 1), (1, 8, 16, 4096), (16, 8, 128, 4096), (3, 2, 4, 7), (5, 3, 8, 130), (7, 4, 8, 2880), (33, 9, 16, 136),
         (6, 32, 40, 264), (257, 4, 32, 1024), (64, 1, 3, 7168), (10, 6, 64, 1001), (9, 7, 16, 1026), (2, 2, 4, 65536),
         (1000, 5, 8, 72), (4, 17, 20, 2050)]


@pytest.mark.parametrize("T,k,E,n", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_dispatch(T, k, E, n, dtype):
    g = torch.Generator(device=DEV).manual_seed(T + k + n)
    pos, live = places(T, k, E, g, 0.2 if T > 2 else 0.0)
    x = torch.randn(T, n, generator=g, device=DEV).to(dtype)
    x[0, 0] = float("nan")
    xs = torch.full((T * k + 3, n), 7.0, dtype=dtype, device=DEV)
    moe.moe_dispatch_rows(x, pos, xs)
    want = torch.full_like(xs, 7.0)
    token = torch.arange(T, device=DEV)[:, None].expand(T, k)
    want[pos[pos >= 0].long()] = x[token[pos >= 0]]
    raw = torch.int32 if dtype == F32 else torch.int16
    assert torch.equal(xs.view(raw), want.view(raw)) and bool((xs[live:] == 7.0).all())


def combined(o, pos, w, add):
    """y and the sum of magnitudes"""
    live = (pos >= 0) & (pos < o.shape[0])
    at = pos.long().clamp(0, max(o.shape[0] - 1, 0))
    w = (w.double() if w is not None else torch.ones(pos.shape, dtype=torch.float64, device=DEV))
    y = add.double() if add is not None else torch.zeros(pos.shape[0], o.shape[1], dtype=torch.float64, device=DEV)
    mag = y.abs()
    for s in range(pos.shape[1]):
        term = torch.where(live[:, s:s + 1], w[:, s:s + 1] * o[at[:, s]].double(), torch.zeros_like(y))
        y, mag = y + term, mag + term.abs()
    return y, mag


@pytest.mark.parametrize("T,k,E,n", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ydtype", [F32, BF16])
@pytest.mark.parametrize("form", ["weights and addend", "plain", "in place"])
def test_combine(T, k, E, n, dtype, ydtype, form):
    g = torch.Generator(device=DEV).manual_seed(T + k + n)
    pos, live = places(T, k, E, g, 0.2 if T > 2 else 0.0)
    o = torch.randn(T * k, n, generator=g, device=DEV).to(dtype)
    o[live:] = float("nan")                                          # rows of no pair are not read
    w = torch.randn(T, k, generator=g, device=DEV) if form != "plain" else None
    if w is not None:
        w[pos < 0] = float("nan")
    add = torch.randn(T, n, generator=g, device=DEV).to(ydtype) if form != "plain" else None
    want, mag = combined(o, pos, w, add)
    y = add if form == "in place" else torch.full((T, n), 7.0, dtype=ydtype, device=DEV)
    moe.moe_combine_rows(o, pos, y, weights=w, addend=add)
    err = (y.double() - want).abs() - (mag * (k * U * 1.01) + want.abs() * HALF[ydtype])
    assert bool((err <= 0).all()), float(err.max())


@pytest.mark.parametrize("T,k,E,n", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ydtype", [F32, BF16])
@pytest.mark.parametrize("form", ["both", "rows", "dots", "in place", "without weights"])
def test_combine_grad(T, k, E, n, dtype, ydtype, form):
    g = torch.Generator(device=DEV).manual_seed(T + k + n)
    pos, live = places(T, k, E, g, 0.2 if T > 2 else 0.0)
    M = T * k + 2
    o = torch.randn(M, n, generator=g, device=DEV).to(dtype)
    o[live:] = 7.0
    before = o.clone()
    w = torch.randn(T, k, generator=g, device=DEV) if form != "without weights" else None
    dy = torch.randn(T, n, generator=g, device=DEV).to(ydtype)
    do = {"dots": None, "in place": o}.get(form, torch.full((M, n), 7.0, dtype=dtype, device=DEV))
    dw = torch.full((T, k), 7.0, device=DEV) if form != "rows" else None
    moe.moe_combine_grad(dy, pos, weights=w, o=o if form != "rows" else None, do=do, dweights=dw)
    at, token = pos.long(), torch.arange(T, device=DEV)[:, None].expand(T, k)
    on = at >= 0
    if do is not None:
        want = torch.full((M, n), 7.0, dtype=torch.float64, device=DEV)
        scale = w.double()[on][:, None] if w is not None else 1.0
        want[at[on]] = scale * dy.double()[token[on]]
        err = (do.double() - want).abs() - want.abs() * (U * 1.01 + HALF[dtype])
        assert bool((err <= 0).all()), float(err.max())
        assert bool((do[live:] == 7.0).all())
    if dw is not None:
        a, b = before.double()[at.clamp(min=0)], dy.double()[token]
        want = torch.where(on, (a * b).sum(2), torch.zeros(T, k, dtype=torch.float64, device=DEV))
        tol = (a * b).abs().sum(2) * (8 * -(-n // 1024) + 12) * U
        assert bool(((dw.double() - want).abs() <= tol).all())
        assert (dw[~on] == 0).all()


def test_places_outside_are_not_followed():
    g = torch.Generator(device=DEV).manual_seed(4)
    T, k, n, M = 12, 3, 96, 20
    pos = torch.randperm(M + 16, generator=g, device=DEV)[:T * k].to(torch.int32).reshape(T, k).contiguous()
    pos[0, 0], pos[1, 1], pos[2, 2] = -2147483648, 2147483647, M
    guard = torch.full((M + 40, n), 7.0, device=DEV)
    xs = guard[:M]
    x = torch.randn(T, n, generator=g, device=DEV)
    moe.moe_dispatch_rows(x, pos, xs)
    on = (pos >= 0) & (pos < M)
    want = torch.full((M, n), 7.0, device=DEV)
    want[pos[on].long()] = x[torch.arange(T, device=DEV)[:, None].expand(T, k)[on]]
    assert torch.equal(xs, want) and bool((guard[M:] == 7.0).all())
    o = torch.randn(M, n, generator=g, device=DEV)
    y = torch.empty(T, n, device=DEV)
    moe.moe_combine_rows(o, pos, y)
    full, mag = combined(o, pos, None, None)
    assert bool(((y.double() - full).abs() <= mag * k * U * 1.01 + TINY).all())
    do, dw = guard[:M].clone(), torch.full((T, k), 7.0, device=DEV)
    moe.moe_combine_grad(x, pos, o=o, do=do, dweights=dw)
    assert torch.equal(do, want) and (dw[~on] == 0).all()


def test_tokens_without_experts_and_no_rows_at_all():
    n = 40
    pos = torch.full((5, 3), -1, dtype=torch.int32, device=DEV)
    add = torch.randn(5, n, device=DEV)
    for M in (0, 4):
        o = torch.full((M, n), float("nan"), device=DEV)
        y = torch.empty(5, n, device=DEV)
        moe.moe_combine_rows(o, pos, y, addend=add)
        assert torch.equal(y, add)
        moe.moe_combine_rows(o, pos, y)
        assert bool((y == 0).all())
        dw = torch.full((5, 3), 7.0, device=DEV)
        moe.moe_combine_grad(add, pos, o=o, do=o, dweights=dw)
        assert bool((dw == 0).all())
        moe.moe_dispatch_rows(add, pos, o)
    none = torch.empty(0, 3, dtype=torch.int32, device=DEV)
    o = torch.full((4, n), 7.0, device=DEV)
    empty = torch.empty(0, n, device=DEV)
    moe.moe_dispatch_rows(empty, none, o)
    moe.moe_combine_rows(o, none, empty)
    moe.moe_combine_grad(empty, none, o=o, do=o, dweights=torch.empty(0, 3, device=DEV))
    assert bool((o == 7.0).all())


def test_gradient_against_differences():
    """sum(dy * y) is linear in o and in the weights: a whole step gives the gradient but for roundings.  y is off by
    (k + 1) u of the magnitudes on either side; the dot with dy in 64 bits adds nothing."""
    g = torch.Generator(device=DEV).manual_seed(9)
    T, k, E, n = 6, 3, 8, 48
    pos, live = places(T, k, E, g)
    o, w = torch.randn(T * k, n, generator=g, device=DEV), torch.randn(T, k, generator=g, device=DEV)
    dy = torch.randn(T, n, generator=g, device=DEV)
    do, dw = torch.empty_like(o), torch.empty_like(w)
    moe.moe_combine_grad(dy, pos, weights=w, o=o, do=do, dweights=dw)

    def value(o, w):
        y = torch.empty(T, n, device=DEV)
        moe.moe_combine_rows(o, pos, y, weights=w)
        return float((y.double() * dy.double()).sum()), float((combined(o, pos, w, None)[1] * dy.double().abs()).sum())

    base, mag = value(o, w)
    for t, s in ((0, 0), (3, 2), (5, 1)):
        moved = w.clone()
        moved[t, s] += 1.0
        up, mag2 = value(o, moved)
        step = float(moved[t, s].double() - w[t, s].double())
        assert abs((up - base) / step - float(dw[t, s])) <= (mag + mag2) * (k + 40) * U / step
        j = 7 * t + s
        moved = o.clone()
        moved[int(pos[t, s]), j] += 1.0
        up, mag2 = value(moved, w)
        step = float(moved[int(pos[t, s]), j].double() - o[int(pos[t, s]), j].double())
        assert abs((up - base) / step - float(do[int(pos[t, s]), j])) <= (mag + mag2) * (k + 40) * U / step


def test_dispatch_and_combine_are_each_others_gradient():
    """<dispatch(x), r> = <x, combine(r)>, exactly in whole numbers"""
    g = torch.Generator(device=DEV).manual_seed(10)
    T, k, E, n = 50, 4, 16, 100
    pos, live = places(T, k, E, g, 0.1)
    x = torch.randint(-4, 5, (T, n), generator=g, device=DEV).float()
    r = torch.randint(-4, 5, (T * k, n), generator=g, device=DEV).float()
    xs, y = torch.zeros(T * k, n, device=DEV), torch.empty(T, n, device=DEV)
    moe.moe_dispatch_rows(x, pos, xs)
    moe.moe_combine_rows(r, pos, y)
    assert float((xs * r).sum()) == float((x * y).sum())


def test_rows_past_32_bit_offsets():
    n, T, k = 65536, 3, 2
    M = (1 << 31) // n + 8
    o = torch.zeros(M, n, dtype=BF16, device=DEV)
    pos = torch.tensor([[0, M - 1], [M - 2, 5], [M - 3, -1]], dtype=torch.int32, device=DEV)
    x = torch.randint(-8, 9, (T, n), device=DEV).to(BF16)
    moe.moe_dispatch_rows(x, pos, o)
    assert torch.equal(o[M - 1], x[0]) and torch.equal(o[M - 2], x[1]) and torch.equal(o[M - 3], x[2])
    assert bool((o[6:M - 3] == 0).all())
    y, dw = torch.empty(T, n, device=DEV), torch.empty(T, k, device=DEV)
    moe.moe_combine_rows(o, pos, y)
    assert torch.equal(y, x.float() * torch.tensor([[2.0], [2.0], [1.0]], device=DEV))
    moe.moe_combine_grad(x, pos, o=o, dweights=dw)
    # whole numbers: the sums stay below 2^24
    want = (x.double() ** 2).sum(1)
    assert dw[0].tolist() == [float(want[0])] * 2 and float(dw[2, 0]) == float(want[2]) and float(dw[2, 1]) == 0.0


def test_replayed_graph_and_other_stream():
    g = torch.Generator(device=DEV).manual_seed(12)
    T, k, E, n = 40, 4, 16, 264
    pos, live = places(T, k, E, g)
    x, w = torch.randn(T, n, generator=g, device=DEV), torch.rand(T, k, generator=g, device=DEV)
    xs, y, do, dw = (torch.zeros(T * k, n, device=DEV), torch.zeros(T, n, device=DEV),
                     torch.zeros(T * k, n, device=DEV), torch.zeros(T, k, device=DEV))

    def step():
        moe.moe_dispatch_rows(x, pos, xs)
        moe.moe_combine_rows(xs, pos, y, weights=w)
        moe.moe_combine_grad(y, pos, weights=w, o=xs, do=do, dweights=dw)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(torch.randn(T, n, generator=g, device=DEV))
    graph.replay()
    got = [t.clone() for t in (xs, y, do, dw)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, (xs, y, do, dw)):
        assert torch.equal(a, b)
