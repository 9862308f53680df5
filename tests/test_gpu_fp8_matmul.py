"""moe_fp8_matmul against the definition in 64 bits.

Tolerance: products of two e4m3 values are exact in fp32.  A block of 128 is summed by the tensor cores; every one
of its additions is taken to lose at most one unit of 24 bits (2^-23) of the sum of magnitudes, so a block is off by
128 * 2^-23 of it.  The scale is two roundings with the scaled addition and there is one addition a block and one a
part of the depth (8 at most): (blocks + 11) * 2^-24.  bf16 outputs are rounded by 2^-8 of themselves.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("quantized_routed_expert_router_gb300")

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


def matrices(G, N, K, g):
    w = (torch.randn(G, N, K, generator=g, device=DEV) * 100).clamp(-448, 448).to(E4M3)
    ws = torch.rand(G, -(-N // 128), -(-K // 128), generator=g, device=DEV) * 1e-4 + 1e-5
    return w, ws


def states(X, K, g):
    x = (torch.randn(X, K, generator=g, device=DEV) * 60).clamp(-448, 448).to(E4M3)
    xs = torch.rand(X, -(-K // 128), generator=g, device=DEV) * 0.02 + 1e-3
    return x, xs


def definition(x, xs, w, ws):
    """y and the sum of magnitudes, [rows, N]"""
    K, N = x.shape[1], w.shape[0]
    a = x.double() * xs.double().repeat_interleave(128, 1)[:, :K]
    b = w.double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return a @ b.t(), a.abs() @ b.abs().t()


def check(y, want, mag, K):
    tol = mag * (128 * 2.0 ** -23 + (-(-K // 128) + 11) * 2.0 ** -24)
    if y.dtype == torch.bfloat16:
        tol = tol + want.abs() * 2.0 ** -8 * 1.01
    err = (y.double() - want).abs() - tol
    assert bool((err <= 0).all()), (float(err.max()), float(((y.double() - want).norm() / want.norm())))


def workspace():
    return torch.zeros(moe.moe_fp8_matmul_workspace_bytes(), dtype=torch.uint8, device=DEV)


# one block of depth and less, ragged depth and width, every part count of a split depth, tiles of 128 and of 192
# columns; places around the tile's 128
DENSE = [(100, 333, 2048), (70, 1026, 4096), (40, 136, 8192), (21, 130, 1536), (5, 24, 48), (8, 200, 4112), (9, 1000, 336), (15, 2051, 1008), (1, 8, 16), (1, 1, 128), (2, 7, 144), (1, 128, 512), (16, 2048, 7168), (1, 7168, 2048), (3, 136, 4096),
         (17, 100, 1040), (64, 512, 1024), (127, 257, 272), (128, 128, 128), (129, 384, 640), (130, 1000, 2880),
         (300, 2880, 2880), (333, 4000, 256), (1000, 1536, 4096), (2048, 2560, 272), (2500, 2051, 400),
         (2560, 2304, 1168)]


@pytest.mark.parametrize("M,N,K", DENSE)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_dense(M, N, K, dtype):
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    x, xs = states(M, K, g)
    w, ws = matrices(1, N, K, g)
    y = torch.full((M + 1, N), 7.0, dtype=dtype, device=DEV)
    st = workspace()
    moe.moe_fp8_matmul(x, xs, w[0], ws[0], y[:M], st)
    check(y[:M], *definition(x, xs, w[0], ws[0]), K)
    assert bool((y[M] == 7.0).all()) and moe.moe_read_device_status(st) == 0


# rows of y that start off a 16-byte boundary: tiles of 128 columns, of 192, depth in parts, last tiles of 1 to 191 columns
@pytest.mark.parametrize("M,N,K", [(1000, 1283, 400), (1001, 1409, 272), (2500, 2052, 400), (2497, 2305, 272),
                                   (2500, 2111, 144), (200, 515, 1040)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_unaligned_rows(M, N, K, dtype):
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    x, xs = states(M, K, g)
    w, ws = matrices(1, N, K, g)
    room = torch.full((M * N + 16,), 7.0, dtype=dtype, device=DEV)
    y = room[8:8 + M * N].view(M, N)
    st = workspace()
    moe.moe_fp8_matmul(x, xs, w[0], ws[0], y, st)
    check(y, *definition(x, xs, w[0], ws[0]), K)
    assert bool((room[:8] == 7.0).all()) and bool((room[8 + M * N:] == 7.0).all())
    assert moe.moe_read_device_status(st) == 0


def sorted_rows(counts, X, g):
    """offsets and random rows for these group sizes"""
    offs = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device=DEV)
    rows = torch.randint(0, X, (int(offs[-1]),), generator=g, device=DEV, dtype=torch.int32)
    return offs, rows


GROUPED = [((0, 9, 0, 4, 3), 328, 4112), ((0,) * 70 + (16,), 100, 208), ((1,), 16, 64), ((0, 3, 0, 1, 0), 100, 272), ((1, 1, 2, 1, 3), 256, 1024), ((128, 129, 0, 127), 384, 528),
           ((5, 0, 300, 1, 0, 0, 77, 260), 1000, 1040), ((700, 900, 0, 1300), 2050, 400), ((0,) * 40 + (2,), 136, 2048),
           (tuple(range(1, 60)), 264, 384)]


@pytest.mark.parametrize("counts,N,K", GROUPED)
@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_grouped(counts, N, K, gathered, dtype):
    g = torch.Generator(device=DEV).manual_seed(len(counts) + N + K)
    total = sum(counts)
    x, xs = states(total if not gathered else 50, K, g)
    offs, rows = sorted_rows(counts, x.shape[0], g)
    w, ws = matrices(len(counts), N, K, g)
    # places behind the last group keep their values
    y = torch.full((total + 5, N), 7.0, dtype=dtype, device=DEV)
    st = workspace()
    if gathered:
        moe.moe_fp8_matmul(x, xs, w, ws, y, st, offsets=offs, rows=torch.cat([rows, rows.new_full((5,), -1)]))
    else:
        pad = torch.cat([x.view(torch.uint8), torch.full((5, K), 0x7F, dtype=torch.uint8, device=DEV)])   # NaN codes
        moe.moe_fp8_matmul(pad, torch.cat([xs, xs[:5] if total >= 5 else xs[:1].expand(5, -1)]), w, ws, y, st, offsets=offs)
    for e, c in enumerate(counts):
        a, b = int(offs[e]), int(offs[e + 1])
        if c:
            r = rows[a:b].long() if gathered else slice(a, b)
            check(y[a:b], *definition(x[r], xs[r], w[e], ws[e]), K)
    assert bool((y[total:] == 7.0).all()) and moe.moe_read_device_status(st) == 0


def test_rows_of_other_groups_and_columns_of_other_experts_do_not_leak():
    """a tile copies rows and columns past its group's: NaN codes there must stay there"""
    g = torch.Generator(device=DEV).manual_seed(5)
    for counts in ((70, 60, 70), (5, 3, 8)):
        leaks_nothing(counts, g)


def leaks_nothing(counts, g):
    a, b, n = counts[0], counts[0] + counts[1], sum(counts)
    x, xs = states(n, 384, g)
    w, ws = matrices(3, 200, 384, g)
    x.view(torch.uint8)[a:b] = 0x7F                    # the middle group
    w.view(torch.uint8)[1] = 0xFF
    offs = torch.tensor([0, a, b, n], dtype=torch.int32, device=DEV)
    y = torch.empty(n, 200, device=DEV)
    moe.moe_fp8_matmul(x, xs, w, ws, y, workspace(), offsets=offs)
    check(y[:a], *definition(x[:a], xs[:a], w[0], ws[0]), 384)
    check(y[b:], *definition(x[b:], xs[b:], w[2], ws[2]), 384)
    assert bool(torch.isnan(y[a:b]).all())


def test_dense_rows_gathered_and_repeated():
    g = torch.Generator(device=DEV).manual_seed(6)
    x, xs = states(10, 640, g)
    w, ws = matrices(1, 136, 640, g)
    rows = torch.tensor([9, 0, 0, 3, 3, 3, 9], dtype=torch.int32, device=DEV)
    y = torch.empty(7, 136, device=DEV)
    moe.moe_fp8_matmul(x, xs, w[0], ws[0], y, workspace(), rows=rows)
    check(y, *definition(x[rows.long()], xs[rows.long()], w[0], ws[0]), 640)
    assert torch.equal(y[1], y[2]) and torch.equal(y[0], y[6])


def test_indexes_out_of_range_with_few_rows():
    g = torch.Generator(device=DEV).manual_seed(17)
    x, xs = states(6, 400, g)
    w, ws = matrices(3, 136, 400, g)
    w.view(torch.uint8)[1, 5] = 0x7F                  # a NaN weight: a bad row is zero all the same
    rows = torch.tensor([0, 5, 6, 1, -1, 2, 3, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    offs = torch.tensor([0, 2, 6, 8], dtype=torch.int32, device=DEV)
    y, st = torch.full((8, 136), 7.0, device=DEV), workspace()
    moe.moe_fp8_matmul(x, xs, w, ws, y, st, offsets=offs, rows=rows)
    assert moe.moe_read_device_status(st) == moe.DEV_BAD_ROW
    for i in (2, 4, 7):
        assert bool((y[i] == 0).all())
    check(y[:2], *definition(x[rows[:2].long()], xs[rows[:2].long()], w[0], ws[0]), 400)
    check(y[6:7], *definition(x[3:4], xs[3:4], w[2], ws[2]), 400)
    for bad in ([-4, 2, 6, 8], [0, 2, 6, 1000], [0, 5, 3, 8], [9, 9, 9, 9], [-9, -9, -9, -9]):
        offs = torch.tensor(bad, dtype=torch.int32, device=DEV)
        y = torch.full((10, 136), 7.0, device=DEV)
        moe.moe_fp8_matmul(x, xs, w, ws, y[:8], st, offsets=offs, rows=rows.clamp(0, 5))
        assert moe.moe_read_device_status(st) == moe.DEV_BAD_ROW, bad
        assert bool((y[8:] == 7.0).all())


@pytest.mark.parametrize("N,K", [(264, 272), (2600, 272)])
def test_indexes_out_of_range_are_not_followed(N, K):
    g = torch.Generator(device=DEV).manual_seed(7)
    x, xs = states(20, K, g)
    w, ws = matrices(3, N, K, g)
    rows = torch.randint(0, 20, (60,), generator=g, device=DEV, dtype=torch.int32)
    rows[5], rows[30], rows[59] = -1, 20, 2 ** 31 - 1
    offs = torch.tensor([0, 20, 40, 60], dtype=torch.int32, device=DEV)
    y, st = torch.full((60, N), 7.0, device=DEV), workspace()
    moe.moe_fp8_matmul(x, xs, w, ws, y, st, offsets=offs, rows=rows)
    assert moe.moe_read_device_status(st) == moe.DEV_BAD_ROW
    good = (rows >= 0) & (rows < 20)
    assert bool((y[~good] == 0).all())
    for e in range(3):
        at = torch.arange(20 * e, 20 * e + 20, device=DEV)[good[20 * e:20 * e + 20]]
        check(y[at], *definition(x[rows[at].long()], xs[rows[at].long()], w[e], ws[e]), K)
    # offsets that leave [0, M] or fall: taken as the range's ends, flagged
    rows = rows.clamp(0, 19)
    for bad in ([-4, 20, 40, 60], [0, 20, 40, 1000], [0, 50, 40, 60]):
        offs = torch.tensor(bad, dtype=torch.int32, device=DEV)
        y = torch.full((62, N), 7.0, device=DEV)
        moe.moe_fp8_matmul(x, xs, w, ws, y[:60], st, offsets=offs, rows=rows)
        assert moe.moe_read_device_status(st) == moe.DEV_BAD_ROW, bad
        assert bool((y[60:] == 7.0).all())
        if bad[1] == 20:
            check(y[:20], *definition(x[rows[:20].long()], xs[rows[:20].long()], w[0], ws[0]), K)


def test_equal_calls_give_equal_bits_and_a_row_does_not_see_its_neighbours():
    g = torch.Generator(device=DEV).manual_seed(8)
    x, xs = states(40, 4096, g)
    w, ws = matrices(1, 520, 4096, g)
    y = [torch.empty(40, 520, device=DEV) for _ in range(3)]
    st = workspace()
    for i in range(2):
        moe.moe_fp8_matmul(x, xs, w[0], ws[0], y[i], st)
    assert torch.equal(y[0], y[1])
    x2, xs2 = x.clone(), xs.clone()
    x2[:11], xs2[12:] = x[29:40], xs2[12:] * 3
    moe.moe_fp8_matmul(x2, xs2, w[0], ws[0], y[2], st)
    assert torch.equal(y[2][11], y[0][11])


def test_captured_and_two_streams_with_one_workspace():
    g = torch.Generator(device=DEV).manual_seed(9)
    x, xs = states(300, 1024, g)
    w, ws = matrices(4, 640, 1024, g)
    offs, rows = sorted_rows((100, 0, 150, 50), 300, g)
    st = workspace()
    want, y1, y2 = (torch.empty(300, 640, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    moe.moe_fp8_matmul(x, xs, w, ws, want, st, offsets=offs, rows=rows)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        moe.moe_fp8_matmul(x, xs, w, ws, y1, st, offsets=offs, rows=rows, stream=a)
        moe.moe_fp8_matmul(x, xs, w, ws, y2, st, offsets=offs, rows=rows, stream=b)
    torch.cuda.synchronize()
    assert torch.equal(y1, want) and torch.equal(y2, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_fp8_matmul(x, xs, w, ws, y1, st, offsets=offs, rows=rows)
    rows.copy_(rows.flip(0))                       # other rows and group sizes through the same graph
    offs.copy_(torch.tensor([0, 0, 10, 290, 300], dtype=torch.int32))
    moe.moe_fp8_matmul(x, xs, w, ws, want, st, offsets=offs, rows=rows)
    y1.zero_()
    graph.replay()
    assert torch.equal(y1, want) and moe.moe_read_device_status(st) == 0


def test_no_rows_and_refusals():
    g = torch.Generator(device=DEV).manual_seed(10)
    x, xs = states(8, 256, g)
    w, ws = matrices(2, 64, 256, g)
    offs = torch.tensor([0, 3, 8], dtype=torch.int32, device=DEV)
    y, st = torch.full((8, 64), 7.0, device=DEV), workspace()
    moe.moe_fp8_matmul(x, xs, w, ws, y[:0], st, offsets=torch.zeros(3, dtype=torch.int32, device=DEV))
    moe.moe_fp8_matmul(x, xs, w, ws, y, st, offsets=torch.zeros(3, dtype=torch.int32, device=DEV))    # empty groups
    ok = dict(x8=x, x_scale=xs, w=w, w_scale=ws, y=y, ws=st, offsets=offs)
    for kw in (dict(ws=None), dict(ws=st[:100]), dict(ws=st[4:]), dict(offsets=None),
               dict(x8=x[:4], x_scale=xs[:4]),                                       # fewer rows than places
               dict(x8=x[:, :248].contiguous(), w=w[:, :, :248].contiguous()),       # depth no multiple of 16
               dict(x8=torch.zeros(8 * 256 + 8, dtype=torch.uint8, device=DEV)[8:].view(8, 256))):
        with pytest.raises(moe.MoeError):
            moe.moe_fp8_matmul(**{**ok, **kw})
    for kw in (dict(x8=x.float()), dict(x_scale=xs[:, :1]), dict(w=w[:, :, :128]), dict(w_scale=ws[:1]),
               dict(y=y.half()), dict(y=y[:, :32]), dict(offsets=offs.long()), dict(offsets=offs[:2]),
               dict(rows=torch.zeros(3, dtype=torch.int32, device=DEV)), dict(x_scale=xs.cpu())):
        with pytest.raises(ValueError):
            moe.moe_fp8_matmul(**{**ok, **kw})
    assert bool((y == 7.0).all()) and moe.moe_read_device_status(st) == 0


def test_prefill_of_a_layer():
    """norm -> 8-bit rows and the fp32 state -> router -> order -> grouped gate product; counts -> balance loss"""
    T, H, I, E, k = 100, 2048, 512, 32, 4
    g = torch.Generator(device=DEV).manual_seed(11)
    x, r = (torch.randn(T, H, generator=g, device=DEV) for _ in range(2))
    nw = torch.rand(H, generator=g, device=DEV) + 0.5
    router = torch.randn(E, H, generator=g, device=DEV) * 0.02
    gate, gs = matrices(E, I, H, g)
    out, y = torch.empty_like(x), torch.empty_like(x)
    x8 = torch.empty(T, H, dtype=E4M3, device=DEV)
    xs = torch.empty(T, H // 128, device=DEV)
    moe.moe_add_rmsnorm(x, r, nw, 1e-6, residual_out=out, y=y, x8=x8, x8_scale=xs)
    ids = torch.empty(T, k, dtype=torch.int32, device=DEV)
    wts, logits = torch.empty(T, k, device=DEV), torch.empty(T, E, device=DEV)
    wr = torch.zeros(moe.moe_route_workspace_bytes(16, E, H), dtype=torch.uint8, device=DEV)
    for a in range(0, T, 16):
        b = min(T, a + 16)
        moe.moe_route(y[a:b], None, router, moe.F32, E, None, k, moe.SOFTMAX, True, ids[a:b], wts[a:b], logits[a:b], wr)
    counts, offsets = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (E, E + 1))
    rows, pos = torch.empty(T * k, dtype=torch.int32, device=DEV), torch.empty(T, k, dtype=torch.int32, device=DEV)
    moe.moe_expert_order(ids, E, None, counts=counts, offsets=offsets, rows=rows, pos=pos)
    o, st = torch.empty(T * k, I, dtype=torch.bfloat16, device=DEV), workspace()
    moe.moe_fp8_matmul(x8, xs, gate, gs, o, st, offsets=offsets, rows=rows)
    loss, d = torch.empty(1, device=DEV), torch.empty_like(logits)
    wb = torch.zeros(moe.moe_balance_loss_workspace_bytes(T, E), dtype=torch.uint8, device=DEV)
    moe.moe_balance_loss(logits, counts, k, moe.SOFTMAX, 0.01, wb, loss=loss, dlogits=d)

    s = x.double() + r.double()
    v = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * nw.double()
    # a logit: fp32 dots of 2048 values, within 64 + 16 roundings of the magnitudes' sum; the choice by exact logits
    # is the kernel's wherever it is not that close
    l64 = v @ router.double().t()
    assert bool(((logits.double() - l64).abs() <= 120 * 2.0 ** -24 * (v.abs() @ router.double().abs().t())).all())
    assert torch.equal(counts.long(), torch.bincount(ids.reshape(-1).long(), minlength=E))
    for t in range(T):
        for s_ in range(k):
            e, i = int(ids[t, s_]), int(pos[t, s_])
            assert int(offsets[e]) <= i < int(offsets[e + 1]) and int(rows[i]) == t
    tt = torch.arange(T, device=DEV).repeat_interleave(k)
    for e in range(E):
        at = pos.reshape(-1)[ids.reshape(-1) == e].long()
        who = tt[ids.reshape(-1) == e]
        if at.numel():
            check(o[at], *definition(x8[who], xs[who], gate[e], gs[e]), H)
    # against the product of the unquantised state: each value is off by 2^-4 of itself or half the smallest step of
    # its group (2^-10 of the scale), so a dot by at most that of the magnitudes
    e, at = int(ids[7, 0]), int(pos[7, 0])
    wf = gate[e].double() * gs[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    off = v[7].abs() * 2.0 ** -4 * 1.001 + xs[7].double().repeat_interleave(128) * 2.0 ** -10
    want = wf @ v[7]
    bound = wf.abs() @ off + want.abs() * 2.0 ** -8 * 1.01 + (wf.abs() @ v[7].abs()) * 2e-5
    assert bool(((o[at].double() - want).abs() <= bound).all())
    p = torch.softmax(logits.double(), 1)
    f = counts.double() * E / (T * k)
    assert abs(float(loss) - 0.01 * float((f * p.mean(0)).sum())) <= 1e-6 * 0.01 * E
    assert moe.moe_read_device_status(st) == 0


def codes(*shape):
    """random finite codes, both signs, made in place (float values of such a size would not be small)"""
    c = torch.empty(shape, dtype=torch.uint8, device=DEV).random_(0, 0x70)
    c[..., ::3] += 0x80
    return c


@pytest.mark.parametrize("M", [12, 300])
def test_rows_beyond_32_bits(M):
    """x past 2^32 bytes, gathered: by the calls for few rows and by tiles"""
    X, K, N = 540000, 8192, 200
    torch.manual_seed(M)
    x, xs = codes(X, K), torch.rand(X, K // 128, device=DEV) * 0.02
    w, ws = matrices(1, N, K, torch.Generator(device=DEV).manual_seed(1))
    rows = torch.randint(X - 2000, X, (M,), device=DEV, dtype=torch.int32)
    rows[0], rows[1] = X - 1, 0
    y, st = torch.empty(M, N, device=DEV), workspace()
    moe.moe_fp8_matmul(x, xs, w[0], ws[0], y, st, rows=rows)
    r = rows.long()
    check(y, *definition(x[r].view(E4M3), xs[r], w[0], ws[0]), K)
    assert moe.moe_read_device_status(st) == 0


@pytest.mark.parametrize("each", [3, 70])
def test_matrices_beyond_32_bits(each):
    G, N, K = 70, 8192, 8192
    torch.manual_seed(each)
    w, ws = codes(G, N, K), torch.rand(G, N // 128, K // 128, device=DEV) * 1e-4
    x, xs = states(2 * each, K, torch.Generator(device=DEV).manual_seed(2))
    offs = torch.zeros(G + 1, dtype=torch.int32, device=DEV)
    offs[G - 1], offs[G] = each, 2 * each                  # the last two experts
    y, st = torch.empty(2 * each, N, device=DEV), workspace()
    moe.moe_fp8_matmul(x, xs, w, ws, y, st, offsets=offs)
    for e in range(2):
        a = slice(e * each, (e + 1) * each)
        check(y[a], *definition(x[a], xs[a], w[G - 2 + e].view(E4M3), ws[G - 2 + e]), K)
    assert moe.moe_read_device_status(st) == 0


@pytest.mark.parametrize("N", [16384, 16387])
def test_results_beyond_32_bits(N):
    M, K = 140000, 16
    g = torch.Generator(device=DEV).manual_seed(N)
    x, xs = states(M, K, g)
    w, ws = matrices(1, N, K, g)
    y = torch.full((M, N), 7.0, device=DEV)
    moe.moe_fp8_matmul(x, xs, w[0], ws[0], y, workspace())
    for a in (slice(0, 40), slice(M // 2, M // 2 + 40), slice(M - 200, M)):
        check(y[a], *definition(x[a], xs[a], w[0], ws[0]), K)
