"""How many tiles moe_matmul takes, as its header states it.  Stand-in addresses, so only where no GPU is visible: a call
that is not refused ends at the query of the driver."""
import ctypes

import pytest

import quantized_routed_expert_router_gb300 as moe
from test_abi import host_only

UNSUP = 2
P = 1 << 20
ALL = 1 << 24      # places


def call(M, N, act=0, offsets=None, G=1):
    return moe.lib().moe_matmul(P, ALL, None, M, offsets, G, P, 0, None, act, None, None, N, 8, P, 0, P, 1 << 20,
                                ctypes.c_void_p(0))


@host_only
@pytest.mark.parametrize("M,N,kw,refused", [
    (ALL, 2047 * 128, {}, False), (ALL, 2048 * 128 - 127, {}, True), (ALL, 2048 * 128, {}, True),
    (ALL - 32, 2048 * 128, {}, False), (ALL - 31, 2048 * 128, {}, True),            # whole tiles of 32 places
    (ALL, 1500 * 128, {}, False),                                                   # more than 2^30 of 16 places
    (ALL, 1023 * 128, dict(act=3), False), (ALL, 1024 * 128, dict(act=3), True),    # gate and up columns
    (ALL - 64, 2048 * 128, dict(offsets=P), False), (ALL - 32, 2048 * 128, dict(offsets=P), True),
    (ALL, 2040 * 128, dict(offsets=P, G=1024), False), (ALL, 2045 * 128, dict(offsets=P, G=1024), True)])
def test_number_of_tiles(M, N, kw, refused):
    status = call(M, N, **kw)
    assert status != 0 and (status == UNSUP) == refused
