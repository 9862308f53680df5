"""moe_topk and moe_topk_grad against the definition in 64 bits.

Ids have to be equal.  Tolerances, u = 2^-24, x = a logit less its row's largest: expf is off by 2 units in the last
place (4 u) and its argument by |x| u; sigma by 12 u and, with the row's largest factored out, |x| u more; a sum over
the slots adds 5 u (five additions in turn) and what its terms are off by, a division u.  A sum over all experts takes
the machine's exp, (4 + 1.3 |x|) u, and at most 37 additions in turn.  So a weight is off by at most
(64 + |x| + 1.3 mean|x|) u of itself with the mean taken under the row's probabilities.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("quantized_routed_expert_router_gb300")

DEV = "cuda"
U = 2.0 ** -24
TINY = 2.0 ** -125


def order(l, k):
    """Ids of the k largest: NaN above all, ties to the lower index, -1 where only -inf is left."""
    key = torch.where(torch.isnan(l), torch.full_like(l, float("inf")), l.double().clamp(max=1e300))
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    return torch.where(torch.gather(key, 1, ids) == -float("inf"), torch.full_like(ids, -1), ids)


def weights_of(l, ids, gating, renormalize):
    """Weights in 64 bits and what they may be off by, relative to themselves."""
    l = l.double()
    log = torch.log_softmax(l, 1) if gating == moe.SOFTMAX else torch.nn.functional.logsigmoid(l)
    log = torch.where(l == -float("inf"), l, log)
    p = torch.exp(log - log.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    x = (l - l.amax(1, keepdim=True)).abs()
    mean = torch.where(p > 0, p * x, torch.zeros_like(p)).sum(1, keepdim=True)
    live = ids >= 0
    at = ids.clamp(min=0)
    c = torch.where(live, torch.gather(log, 1, at), torch.full_like(log[:, :1], -float("inf")))
    w = torch.exp(c - torch.logsumexp(c, 1, keepdim=True) if renormalize else c)
    w = torch.where(live, w, torch.zeros_like(w))
    rel = (64 + torch.where(live, torch.gather(x, 1, at), torch.zeros_like(w)) + 1.3 * mean) * U
    return w, rel, p, x, mean


def logits(T, E, g, dtype, spread=1.5):
    return (spread * torch.randn(T, E, generator=g, device=DEV)).to(dtype)


SIZES = [(1, 1, 1), (1, 8, 8), (3, 7, 2), (16, 128, 8), (5, 33, 5), (4, 64, 1), (9, 65, 4), (17, 100, 32), (7, 130, 9),
         (33, 256, 8), (21, 260, 8), (6, 512, 6), (5, 513, 7), (11, 1024, 32), (4, 1021, 3), (4099, 60, 4), (2050, 32, 8),
         (37, 48, 12), (37, 128, 16), (37, 256, 16), (37, 256, 20), (4099, 128, 8), (4099, 256, 8), (2051, 64, 6)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("gating", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_choice_and_weights(T, E, k, gating, renormalize, dtype):
    g = torch.Generator(device=DEV).manual_seed(T + E + k)
    l = logits(T, E, g, dtype)
    ids = torch.full((T, k), 7, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), 7.0, device=DEV)
    moe.moe_topk(l, gating, renormalize, ids, w)
    want = order(l, k)
    assert torch.equal(ids.long(), want)
    ww, rel = weights_of(l, want, gating, renormalize)[:2]
    assert bool(((w.double() - ww).abs() <= rel * ww + TINY).all())


def test_ties_take_the_lowest_index():
    l = torch.zeros(5, 300, device=DEV)
    l[1] = -0.0
    l[1, 250] = 0.0
    l[2, 100:] = 1.0
    l[3, ::7] = 2.0
    l[4] = torch.tensor([1.0, 0.5], device=DEV).repeat(150)
    for dtype in (torch.float32, torch.bfloat16):
        ids = torch.empty(5, 8, dtype=torch.int32, device=DEV)
        moe.moe_topk(l.to(dtype), moe.SOFTMAX, True, ids)
        assert torch.equal(ids.long(), order(l, 8))
        assert ids[1].tolist() == list(range(8))          # -0 is no smaller than 0


@pytest.mark.parametrize("gating", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("E", [12, 13])
def test_experts_that_may_not_be_taken(gating, renormalize, E):
    """-inf, down to rows with fewer experts than slots and with none; the type's lowest value counts as a number."""
    inf = float("inf")
    l = torch.randn(6, E, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    l[0, 3:] = -inf
    l[1] = -inf
    l[2, 1:] = torch.finfo(torch.float32).min
    l[3, :E - 1] = -inf
    l[4] = torch.finfo(torch.float32).min
    ids = torch.full((6, 4), 7, dtype=torch.int32, device=DEV)
    w = torch.full((6, 4), 7.0, device=DEV)
    moe.moe_topk(l, gating, renormalize, ids, w)
    want = order(l, 4)
    assert torch.equal(ids.long(), want)
    assert (ids[0] >= 0).sum() == 3 and (ids[1] == -1).all() and ids[3].tolist() == [E - 1, -1, -1, -1]
    assert (ids[2] >= 0).all() and ids[4].tolist() == [0, 1, 2, 3]
    ok = [0, 1, 2, 3, 5]      # (row 4's sigmas are 0 in 64 bits too)
    ww, rel = weights_of(l[ok], want[ok], gating, renormalize)[:2]
    ww = torch.nan_to_num(ww)
    assert bool(((w[ok].double() - ww).abs() <= rel.nan_to_num(1e-5, 1e-5, 1e-5).clamp(max=1e-5) * ww + TINY).all())
    assert (w[1] == 0).all()


def test_far_sigmoids_keep_their_ratios():
    """Rows whose sigmas all vanish in 32 bits."""
    l = torch.tensor([[-200.0, -201.0, -203.0, -204.0], [-1000.0, -1000.5, -1002.0, -3000.0]], device=DEV)
    ids = torch.empty(2, 2, dtype=torch.int32, device=DEV)
    w = torch.empty(2, 2, device=DEV)
    moe.moe_topk(l, moe.SIGMOID, True, ids, w)
    want = torch.softmax(l.double()[:, :2], 1)     # sigma(l) = exp(l) there
    assert bool(((w.double() - want).abs() <= 66 * U * want).all())


@pytest.mark.parametrize("gating", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("renormalize", [True, False])
def test_a_nan_shows(gating, renormalize):
    l = torch.randn(4, 40, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2))
    l[1, 30] = float("nan")
    l[2, 5] = l[2, 6] = -float("nan")
    ids, w = torch.empty(4, 3, dtype=torch.int32, device=DEV), torch.empty(4, 3, device=DEV)
    moe.moe_topk(l, gating, renormalize, ids, w)
    assert torch.equal(ids.long(), order(l, 3))
    assert ids[1, 0] == 30 and ids[2, :2].tolist() == [5, 6]
    assert bool(torch.isnan(w[1, 0])) and bool(torch.isnan(w[2, :2]).all())
    assert not bool(torch.isnan(w[[0, 3]]).any())
    if renormalize or gating == moe.SOFTMAX:
        assert bool(torch.isnan(w[1]).all())


@pytest.mark.parametrize("dtype", [torch.uint8, torch.bool])
def test_padded_tokens(dtype):
    g = torch.Generator(device=DEV).manual_seed(3)
    l = logits(37, 50, g, torch.float32)
    valid = (torch.rand(37, generator=g, device=DEV) < 0.6).to(dtype)
    clean = l.clone()
    l[~valid.bool()] = float("nan")
    ids, w = torch.empty(37, 6, dtype=torch.int32, device=DEV), torch.empty(37, 6, device=DEV)
    moe.moe_topk(l, moe.SOFTMAX, True, ids, w, valid=valid)
    on = valid.bool()
    assert torch.equal(ids[on].long(), order(clean, 6)[on]) and (ids[~on] == -1).all() and (w[~on] == 0).all()


MANY = 40003      # rows enough that several share a warp


@pytest.mark.parametrize("E,k", [(8, 8), (12, 1), (60, 4), (64, 8), (100, 7), (128, 8), (132, 8), (256, 8), (256, 3),
                                 (256, 9), (61, 8), (260, 8), (512, 8), (512, 2), (388, 6), (512, 9)])
@pytest.mark.parametrize("gating", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_rows(E, k, gating, renormalize, dtype):
    l = logits(MANY, E, torch.Generator(device=DEV).manual_seed(E + k), dtype)
    ids = torch.full((MANY + 1, k), 7, dtype=torch.int32, device=DEV)
    w = torch.full((MANY + 1, k), 7.0, device=DEV)
    moe.moe_topk(l, gating, renormalize, ids[:MANY], w[:MANY])
    want = order(l, k)
    assert torch.equal(ids[:MANY].long(), want)
    ww, rel = weights_of(l, want, gating, renormalize)[:2]
    assert bool(((w[:MANY].double() - ww).abs() <= rel * ww + TINY).all())
    assert (ids[MANY] == 7).all() and (w[MANY] == 7).all()
    alone = torch.empty_like(ids)
    moe.moe_topk(l, gating, renormalize, alone[:MANY])
    assert torch.equal(alone[:MANY], ids[:MANY])


def awkward(T, E, dtype):
    """Rows of eleven kinds in turn, so that those of a warp differ; every kind meets every place in a warp."""
    g = torch.Generator(device=DEV).manual_seed(E)
    l = torch.randn(T, E, generator=g, device=DEV)
    inf, kind = float("inf"), torch.arange(T, device=DEV) % 11
    col = torch.arange(E, device=DEV)
    l[kind == 1] = 0.0
    l[kind == 2] = torch.where(col % 3 == 1, 0.0, -0.0)
    l[kind == 3] = torch.where(col >= 3, -inf, l[kind == 3])                     # fewer than the slots
    l[kind == 4] = -inf
    l[kind == 5] = torch.finfo(dtype).min
    l[kind == 6] = torch.where(col % 19 == 5, float("nan"), l[kind == 6])
    lane = torch.randint(0, 8, (T, 1), generator=g, device=DEV)
    crowd = (col // 4 % 8 == lane) | (col // 4 % 32 == lane)                      # the largest side by side
    l = torch.where((kind == 7)[:, None] & crowd, l + 20, l)
    l[kind == 8] = (1 + torch.randint(0, 40, (int((kind == 8).sum()), E), generator=g, device=DEV) * 2.0 ** -23)
    l[kind == 9] = torch.where(col % 50 == 3, inf, l[kind == 9])
    l[kind == 10] = torch.sort(l[kind == 10], dim=1).values
    return l.to(dtype)


@pytest.mark.parametrize("E,k", [(256, 8), (256, 5), (128, 8), (60, 6), (32, 8), (512, 8), (400, 3), (144, 8)])
@pytest.mark.parametrize("gating,renormalize", [(moe.SOFTMAX, True), (moe.SIGMOID, True), (moe.SIGMOID, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_awkward_rows(E, k, gating, renormalize, dtype):
    """As the definition has them, and as calls of a few rows do: the same weights to the bit."""
    l = awkward(MANY, E, dtype)
    valid = torch.rand(MANY, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV) < 0.8
    for on in (None, valid):
        ids = torch.full((MANY, k), 7, dtype=torch.int32, device=DEV)
        w = torch.full((MANY, k), 7.0, device=DEV)
        moe.moe_topk(l, gating, renormalize, ids, w, valid=on)
        want = order(l, k) if on is None else torch.where(on[:, None], order(l, k), -1)
        assert torch.equal(ids.long(), want)
        few, few_w = torch.empty_like(ids), torch.empty_like(w)
        for t in range(0, MANY, 1000):
            to = min(t + 1000, MANY)   # (1000 rows of any E start on 16 bytes)
            moe.moe_topk(l[t:to], gating, renormalize, few[t:to], few_w[t:to], valid=None if on is None else on[t:to])
        assert torch.equal(ids, few) and torch.equal(w.nan_to_num(nan=-1.0), few_w.nan_to_num(nan=-1.0))
        assert torch.equal(torch.isnan(w), torch.isnan(few_w))


def gradient(l, ids, d, gating, renormalize):
    """dlogits in 64 bits by autograd, without the tolerance."""
    l = l.double().requires_grad_(True)
    log = torch.log_softmax(l, 1) if gating == moe.SOFTMAX else torch.nn.functional.logsigmoid(l)
    live = ids >= 0
    c = torch.gather(log, 1, ids.clamp(min=0)).masked_fill(~live, -float("inf"))
    if renormalize:
        some = live.any(1, keepdim=True)
        c = torch.where(live & some, c - torch.logsumexp(torch.where(some, c, torch.zeros_like(c)), 1, keepdim=True), c)
    w = torch.where(live, torch.exp(c), torch.zeros_like(c))
    return torch.autograd.grad((w * torch.where(live, d.double(), torch.zeros_like(w))).sum(), l)[0]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("gating", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("addend", [None, "own", "in place"])
def test_gradient(T, E, k, gating, renormalize, dtype, addend):
    """With S = sum w |d| over the slots: dlogits is a product of a weight (rel), a slope (12 u) and d - sum w d, off by
    rel S + 8 u (|d| + S); over all experts p d - p sum w d likewise with p's tolerance.  Then one addition (u) and the
    rounding to the type.  The definition itself is computed in 64 bits through the logarithms of all E: what is 0 by the
    formula (experts not chosen) comes out as a difference of sums of up to E terms of w |d|, each off by 2^-53 of itself
    and their sum by E 2^-53 of S, on both sides: 2 (E + 8) 2^-53 S."""
    g = torch.Generator(device=DEV).manual_seed(T * 3 + E + k)
    l = logits(T, E, g, dtype)
    ids = order(l, k)
    if T > 4:
        ids[T - T // 4:] = -1                                        # padded tokens
        ids[0, k // 2:] = -1                                         # slots that take no part
        ids[1, 0] = E                                                # so does an id outside
    want_ids = torch.where(ids >= E, torch.full_like(ids, -1), ids)
    d = torch.randn(T, k, generator=g, device=DEV)
    d_in = torch.where(want_ids >= 0, d, torch.full_like(d, float("nan")))
    add = (0.3 * torch.randn(T, E, generator=g, device=DEV)).to(dtype) if addend else None
    out = add.clone() if addend == "in place" else torch.full_like(l, 7.0)
    moe.moe_topk_grad(l, ids.to(torch.int32), d_in, gating, renormalize, out,
                      addend=out if addend == "in place" else add)
    want = gradient(l, want_ids, d, gating, renormalize)
    w, rel, p, x, mean = weights_of(l, want_ids, gating, renormalize)
    live = (want_ids >= 0).double()
    S = (w * d.double().abs() * live).sum(1, keepdim=True)
    one = w * live * ((2 * rel + 40 * U) * (d.double().abs() + S))
    tol = torch.zeros_like(want).scatter_add_(1, want_ids.clamp(min=0), one)
    if gating == moe.SOFTMAX and not renormalize:
        tol = tol + p * S * (100 + 2.3 * x + 1.3 * mean) * U
    a = add.double() if addend else torch.zeros_like(want)
    tol = tol + 2 * (E + 8) * 2.0 ** -53 * S + U * (a.abs() + want.abs()) + TINY
    want = want + a
    if dtype == torch.bfloat16:
        tol = tol + want.abs() * 2.0 ** -8 * 1.01
    err = (out.double() - want).abs() - tol
    assert bool((err <= 0).all()), float(err.max())


def test_gradient_against_differences():
    """A central difference of moe_topk's own weights: step h = 2^-6, the third derivative of a weight in its logits is
    below 1, so the difference is off by h^2 / 6 sum|d| and by the weights' rounding, 70 u w |d| / h."""
    g = torch.Generator(device=DEV).manual_seed(5)
    T, E, k, h = 40, 24, 4, 2.0 ** -6
    for gating in (moe.SOFTMAX, moe.SIGMOID):
        for renormalize in (True, False):
            l = logits(T, E, g, torch.float32)
            top = order(l, k)
            l.scatter_add_(1, top, torch.full((T, k), 0.5, device=DEV))      # the choice holds while a logit moves by h
            ids, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
            moe.moe_topk(l, gating, renormalize, ids, w)
            d = torch.randn(T, k, generator=g, device=DEV)
            grad = torch.empty_like(l)
            moe.moe_topk_grad(l, ids, d, gating, renormalize, grad)
            bound = d.double().abs().sum(1) * (h * h / 6 + 70 * U / h)
            for e in range(0, E, 5):
                value = []
                for step in (h, -h):
                    moved = l.clone()
                    moved[:, e] += step
                    i2, w2 = torch.empty_like(ids), torch.empty_like(w)
                    moe.moe_topk(moved, gating, renormalize, i2, w2)
                    # by expert: two slots may have changed places
                    at = (i2[:, None, :] == ids[:, :, None]).double()
                    assert bool((at.sum(2) == 1).all())
                    value.append((at * w2.double()[:, None, :]).sum(2).mul(d.double()).sum(1))
                diff = (value[0] - value[1]) / (2 * h)
                assert bool(((grad[:, e].double() - diff).abs() <= bound).all())


def test_an_id_that_comes_twice_counts_as_two_slots():
    g = torch.Generator(device=DEV).manual_seed(6)
    l = logits(8, 20, g, torch.float32)
    ids = torch.tensor([[3, 3, 3, 9]] * 8, dtype=torch.int32, device=DEV)
    d = torch.randn(8, 4, generator=g, device=DEV)
    for gating in (moe.SOFTMAX, moe.SIGMOID):
        for renormalize in (True, False):
            out = torch.empty_like(l)
            moe.moe_topk_grad(l, ids, d, gating, renormalize, out)
            want = gradient(l, ids.long(), d, gating, renormalize)
            # weights of at most 1, slopes and differences of |d| sums: 4 slots of (2 * 80 + 40) u (|d| + S), S <= sum|d|
            tol = 4 * 200 * U * 2 * d.double().abs().sum(1, keepdim=True)
            assert bool(((out.double() - want).abs() <= tol).all())
            again = torch.empty_like(l)
            moe.moe_topk_grad(l, ids, d, gating, renormalize, again)
            assert torch.equal(out, again)


def test_masked_logits_have_no_gradient():
    inf = float("inf")
    l = torch.randn(3, 16, device=DEV, generator=torch.Generator(device=DEV).manual_seed(7))
    l[0, 2:] = -inf
    l[1] = -inf
    d = torch.ones(3, 4, device=DEV)
    for gating in (moe.SOFTMAX, moe.SIGMOID):
        for renormalize in (True, False):
            ids = torch.empty(3, 4, dtype=torch.int32, device=DEV)
            moe.moe_topk(l, gating, renormalize, ids)
            for given in (ids, torch.arange(4, dtype=torch.int32, device=DEV).repeat(3, 1)):
                out = torch.full_like(l, 7.0)
                moe.moe_topk_grad(l, given.contiguous(), d, gating, renormalize, out)
                assert bool(torch.isfinite(out).all())
                assert (out[0, 2:] == 0).all() and (out[1] == 0).all()


def test_logits_may_be_overwritten_and_streams_are_kept():
    g = torch.Generator(device=DEV).manual_seed(8)
    l = logits(300, 130, g, torch.float32)
    ids, w = torch.empty(300, 8, dtype=torch.int32, device=DEV), torch.empty(300, 8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_topk(l, moe.SOFTMAX, False, ids, w, stream=side)
    d = w * 0 + 1.5
    side.wait_stream(torch.cuda.current_stream())
    own = torch.empty_like(l)
    moe.moe_topk_grad(l, ids, d, moe.SOFTMAX, False, own, stream=side)
    over = l.clone()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_topk_grad(over, ids, d, moe.SOFTMAX, False, over, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(own, over)


def test_no_tokens():
    for E, k in ((8, 2), (1000, 32)):
        l = torch.empty(0, E, device=DEV)
        ids, w = torch.empty(0, k, dtype=torch.int32, device=DEV), torch.empty(0, k, device=DEV)
        moe.moe_topk(l, moe.SOFTMAX, True, ids, w)
        moe.moe_topk_grad(l, ids, w, moe.SOFTMAX, True, l)


def test_rows_past_32_bit_offsets():
    T, E = (1 << 31) // 1024 + 3, 1024
    l = torch.zeros(T, E, dtype=torch.bfloat16, device=DEV)
    l[-2, 1000] = 2.0
    l[-1, 1023] = 3.0
    ids = torch.empty(T, 1, dtype=torch.int32, device=DEV)
    moe.moe_topk(l, moe.SOFTMAX, True, ids)
    assert ids[-2:, 0].tolist() == [1000, 1023] and int(ids[:-2].sum()) == 0
    moe.moe_topk_grad(l, ids, torch.ones(T, 1, device=DEV), moe.SIGMOID, False, l)
    s = torch.sigmoid(torch.tensor([2.0, 3.0], dtype=torch.float64, device=DEV))
    want = s * (1 - s)
    assert bool(((l[[-2, -1], [1000, 1023]].double() - want).abs() <= want * (2.0 ** -8 * 1.01)).all())
    assert float(l[-1, 1022]) == 0.0 and float(l[0, 0]) == 0.25
