"""The activations of moe_matmul where sigma is small, on values that are exact in fp32: the product is 0 or 1 and the bias,
or z, is the value.

Tolerance, u = 2^-24: sigma is off by (5 + 1.3 |v|) u of itself, and 0 below 2^-126.  silu adds one rounding.  The slope
sigma (1 + v (1 - sigma)) is off by sigma's error times its derivative, at most 1 + 2 |v| of it, and by four roundings of
terms up to sigma (1 + |v|)."""
import pytest
import torch

from test_gpu_matmul import workspace

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("quantized_routed_expert_router_gb300")

DEV = "cuda"
U, LOW = 2.0 ** -24, 2.0 ** -126


def values():
    far = torch.tensor([-1e30, -1e4, -0.0, 0.0, 1e4, 1e30])
    return torch.cat([far, torch.linspace(-130, 95, 957), torch.linspace(-89, -86, 957)]).to(DEV)


@pytest.mark.parametrize("M", [4, 40, 2500])
@pytest.mark.parametrize("act", [moe.ACT_SILU, moe.ACT_SWIGLU, moe.ACT_SILU_GRAD, moe.ACT_SWIGLU_GRAD])
def test_small_sigmas(M, act):
    v = values()
    N = v.numel()
    grad = act in (moe.ACT_SILU_GRAD, moe.ACT_SWIGLU_GRAD)
    x = torch.zeros(M, 8, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(2 * N if act == moe.ACT_SWIGLU else N, 8, dtype=torch.bfloat16, device=DEV)
    one, bias, z = torch.ones_like(v), None, None
    if grad:
        x[:, 0] = 1
        w[:, 0] = 1
        z = (torch.cat([v, one]) if act == moe.ACT_SWIGLU_GRAD else v).expand(M, -1).contiguous()
    else:
        bias = torch.cat([v, one]) if act == moe.ACT_SWIGLU else v
    y = torch.empty(M, 2 * N if act == moe.ACT_SWIGLU_GRAD else N, device=DEV)
    st = workspace()
    moe.moe_matmul(x, w, y, st, act=act, bias=bias, z=z)
    v = v.double()
    s = torch.sigmoid(v)
    rel = (5 + 1.3 * v.abs()) * U
    silu, silu_tol = v * s, (rel + 2 * U) * (v * s).abs() + LOW * v.abs()
    slope, slope_tol = s * (1 + v * (1 - s)), (1 + 2 * v.abs()) * (s * (rel + 8 * U) + LOW)
    want, tol = (slope, slope_tol) if grad else (silu, silu_tol)
    if act == moe.ACT_SWIGLU_GRAD:
        want, tol = torch.cat([slope, silu]), torch.cat([slope_tol, silu_tol])
    assert bool(((y.double() - want).abs() <= tol).all())
    assert moe.moe_read_device_status(st) == 0
