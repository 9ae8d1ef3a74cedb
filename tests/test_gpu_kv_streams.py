"""Counters and workspaces of attention calls on other streams than the current one."""
import pytest
import torch

from kv_cases import Step
from skinny_gemm_gb300 import ops

pytestmark = pytest.mark.gpu


def test_a_captured_call_on_a_forked_stream(monkeypatch):
    """Without a reserved set left, a captured call's counters are zeroed on the call's own stream, and their memory is
    not handed to the capturing stream's next tensors."""
    step = Step(8, 2, 256, 16, [6000], [1], seed=23)
    cache = step.cache()
    want = step.run(cache=cache)
    monkeypatch.setattr(ops, "_kv_capture_sets", {})
    table, cu, lens = step.dev()
    q, out, side, g = step.q.cuda(), torch.empty_like(want), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    busy = torch.zeros(1 << 26, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        with torch.cuda.stream(side):
            busy.add_(1)  # the call begins after the other branch is done
        ops.kv_attention(q, cache, table, cu, lens, 1, 6001, out=out, stream=side)
        ones = [torch.full((ops.KV_COUNTERS,), 1, dtype=torch.int32, device="cuda") for _ in range(4)]
        cur.wait_stream(side)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    assert all(bool((t == 1).all()) for t in ones) and ops.device_status() == 0
