"""The first calls of a process, made by several host threads at once with other sizes: a kernel's shared memory limit
is raised on first use, and one thread's need must not lower it under another's launch.

First calls come once in a process, so each round is a process of its own.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import threading
import torch
import quantized_routed_expert_router_gb300 as moe
E, H, k = 64, 1024, 4
dev = "cuda"
router = torch.randn(E, H, device=dev)
work = []
for i in range(8):
    T = 16 if i % 2 else 1                     # 64 KB of shared memory, or 32
    new = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device=dev)
    work.append((T, torch.randn(T, H, device=dev), new(T, k, dtype=torch.int32), new(T, k), new(T, E),
                 new(moe.moe_route_workspace_bytes(T, E, H), dtype=torch.uint8), torch.cuda.Stream()))
torch.cuda.synchronize()
start, wrong = threading.Barrier(len(work)), []
def first(T, x, ids, w, logits, ws, stream):
    start.wait()
    try:
        moe.moe_route(x, None, router, moe.F32, E, None, k, moe.SOFTMAX, True, ids, w, logits, ws, stream=stream)
    except moe.MoeError as e:
        wrong.append((T, str(e)))
threads = [threading.Thread(target=first, args=a) for a in work]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
assert not wrong, wrong
for T, x, ids, w, logits, ws, stream in work:
    want = x.double() @ router.double().t()
    # fp32 dots of 1024 values: each of at most 64 additions in a row and the product rounded, of the magnitudes' sum
    tol = 65 * 2.0 ** -24 * (x.double().abs() @ router.double().abs().t())
    assert bool(((logits.double() - want).abs() <= tol).all())
print("alright")
"""


@pytest.mark.parametrize("process", range(8))
def test_first_calls_of_threads(process):
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "alright" in r.stdout, r.stderr[-600:]
