"""First calls of a process made while a graph is captured: what a launch looks up once (shared memory limits, registers,
clusters that fit at once) must not disturb the capture.  A process of its own, as first calls come once in one."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
import quantized_routed_expert_router_gb300 as moe
dev, BF16 = "cuda", torch.bfloat16
st = torch.zeros(moe.moe_matmul_workspace_bytes(), dtype=torch.uint8, device=dev)
work = []
# few rows, depth in parts (of 32 and of 128 places), whole depth, two blocks a tile; bf16 and fp32
for M, N, K in ((3, 272, 512), (40, 512, 4096), (100, 512, 4096), (100, 8192, 256), (2500, 2048, 256)):
    for dtype in (BF16, torch.float32):
        work.append((torch.randint(-2, 3, (M, K), device=dev).to(BF16), torch.randint(-2, 3, (N, K), device=dev).to(BF16),
                     torch.zeros(M, N, dtype=dtype, device=dev)))
l = torch.randn(64, 40, device=dev)
ids, w = torch.zeros(64, 4, dtype=torch.int32, device=dev), torch.zeros(64, 4, device=dev)
d = torch.zeros(64, 40, device=dev)
pos = torch.arange(256, dtype=torch.int32, device=dev).reshape(64, 4)
o, y = torch.randn(256, 24, device=dev), torch.zeros(64, 24, device=dev)
xs = torch.zeros(256, 24, device=dev)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for x, m, out in work:
        moe.moe_matmul(x, m, out, st)
    moe.moe_topk(l, moe.SOFTMAX, True, ids, w)
    moe.moe_topk_grad(l, ids, w, moe.SOFTMAX, False, d)
    moe.moe_combine_rows(o, pos, y, weights=w)
    moe.moe_dispatch_rows(y, pos, xs)
    moe.moe_combine_grad(y, pos, weights=w, o=o, do=xs)
assert all(bool((out == 0).all()) for _, _, out in work)
graph.replay()
torch.cuda.synchronize()
assert moe.moe_read_device_status(st) == 0
for x, m, out in work:
    want = (x.double() @ m.double().t()).to(out.dtype)        # whole numbers below 2^24: nothing is lost
    assert torch.equal(out, want), (tuple(x.shape), tuple(m.shape), out.dtype)
got = [t.clone() for t in (ids, w, d, y, xs)]
for t in (ids, w, d, y, xs):
    t.zero_()
moe.moe_topk(l, moe.SOFTMAX, True, ids, w)
moe.moe_topk_grad(l, ids, w, moe.SOFTMAX, False, d)
moe.moe_combine_rows(o, pos, y, weights=w)
moe.moe_dispatch_rows(y, pos, xs)
moe.moe_combine_grad(y, pos, weights=w, o=o, do=xs)
assert all(torch.equal(a, b) for a, b in zip(got, (ids, w, d, y, xs)))
print("alright")
"""


def test_first_calls_in_a_capture():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "alright" in r.stdout, r.stderr[-1500:]
