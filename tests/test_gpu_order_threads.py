"""moe_expert_order from several host threads at once: one stream and one workspace each is all that is needed."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("quantized_routed_expert_router_gb300")

DEV = "cuda"


def order_of(ids, E):
    """the same by a stable sort"""
    T, k = ids.shape
    key = ids.reshape(-1).long()
    by = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=E)
    pos = torch.empty_like(by)
    pos[by] = torch.arange(T * k, device=by.device)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return counts.int(), offsets.int(), (by // k).int(), pos.reshape(T, k).int()


# more than 682 experts take more shared memory than a launch has without asking; numbers of experts that differ from
# thread to thread, one chunk of pairs and several
@pytest.mark.parametrize("T,experts", [(30, (1024, 700)), (1500, (1024, 700, 64)), (30, (1024, 900, 768, 683))])
def test_threads_do_not_disturb_one_another(T, experts):
    k, calls = 8, 1500
    work, wrong = [], []
    for i, E in enumerate(experts):
        g = torch.Generator().manual_seed(T + i)
        ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).to(DEV)
        want = order_of(ids, E)
        out = [torch.full_like(w, -9) for w in want]
        ws = torch.empty(max(16, moe.moe_expert_order_workspace_bytes(T, k, E)), dtype=torch.uint8, device=DEV)
        work.append((ids, E, ws, out, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    start = threading.Barrier(len(work))

    def loop(ids, E, ws, out, _, stream):
        start.wait()
        for _ in range(calls):
            try:
                moe.moe_expert_order(ids, E, ws, counts=out[0], offsets=out[1], rows=out[2], pos=out[3], stream=stream)
            except moe.MoeError as e:
                wrong.append((E, str(e)))
    threads = [threading.Thread(target=loop, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong, (len(wrong), wrong[:3])
    for ids, E, ws, out, want, _ in work:
        assert all(torch.equal(o, w) for o, w in zip(out, want)), E
