"""How exact moe_matmul's sums are, over a whole matrix of results: the bounds that moe.h states.

fp32 results.  The tensor cores cut a running sum off instead of rounding it, so an error grows with its length: over the
whole depth K it would be about K 2^-30 of the results (2e-6 at 2048, 7e-6 at 7168), and half of that where all terms have
one sign and the sum grows evenly.  Running sums of at most 640 values are off by 640 2^-30 = 6e-7 at most, and what adds
them up by a rounding (2^-24) for each of the at most 14 of them, of which the square root counts: 2.2e-7.  Together 6.4e-7;
1e-6 in the norm is what moe.h promises, and what sums over the whole depth miss at every K here.

bf16 results: off by a rounding (2^-8 at most, and as often up as down) and towards zero by what running sums of at most 8192
values are, 2^-15 of themselves, whatever the depth."""
import pytest
import torch

from test_gpu_matmul import sorted_rows, workspace

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("quantized_routed_expert_router_gb300")

DEV = "cuda"

# few rows; 32 and 128 places a tile, whole depth and in parts; two blocks a tile, whole depth and in parts
SIZES = [(5, 2048, None), (16, 640, None), (30, 6144, None), (37, 264, None), (300, 1032, None), (1100, 1536, None),
         (2600, 2056, None), (4100, 1544, None), (None, 520, (9, 0, 20, 1, 31)), (None, 272, tuple(range(1, 50))),
         (None, 1040, (300, 260, 0, 270)), (None, 1040, (97, 100, 101, 90) * 8), (None, 1544, (700, 900, 3, 641))]


def values(M, K, g, signed, large=0):
    """normal values, with some large channels, or of one sign"""
    x = torch.randn(M, K, generator=g, device=DEV)
    if not signed:
        return (x.abs() + 0.5).to(torch.bfloat16)
    x[:, torch.randint(0, K, (large,), generator=g, device=DEV)] *= 12
    return x.to(torch.bfloat16)


def exact(x, w):
    return x.double() @ w.double().t()


@pytest.mark.parametrize("M,N,counts", SIZES)
@pytest.mark.parametrize("K", [2048, 4096, 7168])
@pytest.mark.parametrize("signed", [True, False])
def test_fp32_results(M, N, counts, K, signed):
    g = torch.Generator(device=DEV).manual_seed(N + K)
    offs = rows = None
    if counts:
        M = sum(counts)
        offs, rows = sorted_rows(counts, M, g)
    x = values(M, K, g, signed, K // 200)
    w = values((len(counts) if counts else 1) * N, K, g, signed).mul_(K ** -0.5)
    w = w.view(len(counts), N, K) if counts else w
    y, st = torch.empty(M, N, device=DEV), workspace()
    moe.moe_matmul(x, w, y, st, offsets=offs, rows=rows)
    if counts:
        want = torch.empty(M, N, dtype=torch.float64, device=DEV)
        for e in range(len(counts)):
            p, q = int(offs[e]), int(offs[e + 1])
            want[p:q] = exact(x[rows[p:q].long()], w[e])
    else:
        want = exact(x, w)
    off = float((y.double() - want).norm() / want.norm())
    assert off <= 1e-6, off
    assert moe.moe_read_device_status(st) == 0


@pytest.mark.parametrize("M", [37, 1024])
@pytest.mark.parametrize("K", [8192, 65536])
def test_bf16_results_lean_by_no_more_than_their_depth_allows(M, K):
    """The mean of M N errors: roundings of at most 2^-8, evenly spread, leave 2^-8 / sqrt(3 M N), here five times that."""
    g = torch.Generator(device=DEV).manual_seed(M + K)
    N = 1024
    x, w = values(M, K, g, False), values(N, K, g, False).mul_(K ** -0.5)
    y, st = torch.empty(M, N, dtype=torch.bfloat16, device=DEV), workspace()
    moe.moe_matmul(x, w, y, st)
    want = exact(x, w)
    off = (y.double() - want) / want
    assert float(off.abs().max()) <= 2.0 ** -8 + K * 2.0 ** -30
    assert abs(float(off.mean())) <= K * 2.0 ** -30 + 5 * 2.0 ** -8 / (3 * M * N) ** 0.5
    assert moe.moe_read_device_status(st) == 0


@pytest.mark.parametrize("M,N", [(37, 1024), (1024, 1024), (4100, 1544)])
@pytest.mark.parametrize("K", [8192, 65536, 262144])
def test_bf16_results_lie_between_two_roundings(M, N, K):
    """Each result is the rounding of a value that is off by at most 2^-14 of itself towards zero, at any depth, and by the
    roundings of the fp32 sums, at most 40 of 2^-24.  (The errors of very deep sums of one sign do not average out: they
    are all near one value.)"""
    g = torch.Generator(device=DEV).manual_seed(M + K)
    x, w = values(M, K, g, False), values(N, K, g, False).mul_(K ** -0.5)
    y, st = torch.empty(M, N, dtype=torch.bfloat16, device=DEV), workspace()
    moe.moe_matmul(x, w, y, st)
    want = sum(exact(x[:, k:k + 65536], w[:, k:k + 65536]) for k in range(0, K, 65536))
    low, high = want * (1 - 2.0 ** -14), want * (1 + 40 * 2.0 ** -24)
    assert bool((y >= low.to(torch.bfloat16)).all()) and bool((y <= high.to(torch.bfloat16)).all())
    assert moe.moe_read_device_status(st) == 0


# depths past those that bf16 results sum in one piece, on every kind of tile
DEEP = [(37, 272, None), (520, 1040, None), (2600, 2064, None), (None, 528, (9, 0, 20, 1, 31)), (None, 272, tuple(range(1, 50))),
        (None, 1040, (300, 260, 0, 270)), (None, 1040, (97, 100, 101, 90) * 8), (None, 1552, (700, 900, 3, 641))]


@pytest.mark.parametrize("M,N,counts", DEEP)
@pytest.mark.parametrize("act", [moe.ACT_SILU, moe.ACT_SWIGLU, moe.ACT_GELU_GRAD])
def test_deep_bf16_results(M, N, counts, act):
    """Against fp32 results of the same call, which are off by 1e-6 of the largest slope at most: a rounding of y and of the
    residual's sum (2^-8), and a running sum of at most 8192 values, 17 addends of 2^-23 cut off for each 16 of them, of a sum
    no larger than the terms' magnitudes."""
    K = 72 * 1024 + 8
    g = torch.Generator(device=DEV).manual_seed(N)
    offs = rows = None
    grad, G = act == moe.ACT_GELU_GRAD, len(counts) if counts else 1
    if counts:
        M = sum(counts)
        offs, rows = sorted_rows(counts, M, g)
    x = values(M, K, g, True, K // 200)
    wide = 2 * N if act == moe.ACT_SWIGLU else N
    w = values(G * wide, K, g, True).mul_(0.2 * K ** -0.5)
    w = w.view(G, wide, K) if counts else w
    start = torch.randn(M, N, generator=g, device=DEV).to(torch.bfloat16)
    out = {}
    for dtype in (torch.float32, torch.bfloat16):
        y, st = start.to(dtype).clone(), workspace()
        z = y if grad else torch.empty(M, wide, dtype=dtype, device=DEV)
        moe.moe_matmul(x, w, y, st, act=act, residual=None if grad else y, z=z, offsets=offs, rows=rows)
        assert moe.moe_read_device_status(st) == 0
        out[dtype] = (y.double(), z.double())
    (y, z), (y2, z2) = out[torch.float32], out[torch.bfloat16]
    for a, b in ((y, y2),) if grad else ((y, y2), (z, z2)):
        assert float((a - b).norm() / a.norm()) <= 2.0 ** -8
        assert abs(float(((b - a) * a.sign()).sum() / a.abs().sum())) <= 17 * 2.0 ** -23 * 8192 / 16
