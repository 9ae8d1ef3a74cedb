"""The example's steps (projections, plan, append, attention, output projection) and the state that calls leave."""
import importlib.util
import os

import pytest
import torch

from kv_cases import Step
from skinny_gemm_gb300 import ops

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_attention.py")
    spec = importlib.util.spec_from_file_location("paged_attention", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("kw", [
    dict(hidden=512, q_heads=8, kv_heads=2, dim=64, block=16, prompts=(130, 1, 33, 16), steps=20, draft=3, max_len=512),
    dict(hidden=1024, q_heads=8, kv_heads=2, dim=256, block=64, prompts=(1100,), steps=5, draft=5, max_len=2048),
])
def test_example(kw):
    layer, reqs, y = _example().run(report=lambda s: None, **kw)
    assert y.shape == (len(kw["prompts"]) * kw["draft"], kw["hidden"]) and bool(torch.isfinite(y.float()).all())


def test_replayed_steps_equal_eager_ones():
    """The same tokens through a captured step and through eager calls: the same cache and outputs, bit for bit."""
    m = _example()
    torch.manual_seed(3)
    xs = [torch.randn(2, 512, device="cuda").to(torch.bfloat16) for _ in range(9)]
    prompt = torch.randn(50, 512, device="cuda").to(torch.bfloat16)
    one = torch.ones(2, dtype=torch.int32, device="cuda")
    results = []
    for captured in (False, True):
        torch.manual_seed(4)  # the free list
        layer, reqs = m.Layer(512, 4, 2, 128, 20, 16, seed=9), m.Requests(2, 160, 20, 16)
        reqs.step(layer, prompt, torch.tensor([31, 19], dtype=torch.int32, device="cuda"), 31)
        outs = [reqs.step(layer, xs[0], one, 1)]
        if captured:
            x, g = xs[1].clone(), torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(g):
                out = reqs.step(layer, x, one, 1)
            for t in xs[1:]:
                x.copy_(t)
                g.replay()
                outs.append(out.clone())
        else:
            outs += [reqs.step(layer, t, one, 1) for t in xs[1:]]
        results.append((outs, layer.cache, reqs))
    (a, ca, ra), (b, cb, rb) = results
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert torch.equal(ra.table, rb.table) and torch.equal(ra.cached, rb.cached) and torch.equal(ra.head, rb.head)
    used = ra.table[ra.table >= 0].long()
    assert torch.equal(ca.k_scale[used], cb.k_scale[used]) and torch.equal(ca.v_scale[used], cb.v_scale[used])


def test_counters_and_workspaces():
    """Counters are zero after calls; a captured call has a set of its own; the kept workspace grows and is kept."""
    small = Step(8, 2, 128, 32, [700, 64, 5], [3, 1, 2], seed=17)
    large = Step(8, 2, 128, 32, [9000, 5000, 1], [2, 1, 2], seed=18)
    ca, cb = small.cache(), large.cache()
    want_s, want_l = small.run(cache=ca), large.run(cache=cb)
    for _ in range(3):
        assert torch.equal(small.run(cache=ca), want_s) and torch.equal(large.run(cache=cb), want_l)
    table, cu, lens = large.dev()
    q, g = large.q.cuda(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ops.kv_attention(q, cb, table, cu, lens, 2, 9002)
    taken = ops._kv_capture_sets[0][1]
    assert taken > 0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):  # the graph beside eager calls on another stream
        with torch.cuda.stream(s):
            g.replay()
        assert torch.equal(small.run(cache=ca), want_s)
    torch.cuda.synchronize()
    assert torch.equal(out, want_l)
    for c, _ in ops._kv_counter_cache.values():
        assert int(c.abs().max()) == 0
    assert int(ops._kv_capture_sets[0][0].abs().max()) == 0
    assert ops.device_status() == 0


def test_no_capture_sets_left(monkeypatch):
    """A captured call without a reserved set zeroes counters in its graph."""
    step = Step(8, 2, 256, 16, [3000], [1], seed=19)
    cache = step.cache()
    want = step.run(cache=cache)
    monkeypatch.setattr(ops, "_kv_capture_sets", {})
    table, cu, lens = step.dev()
    q, g = step.q.cuda(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ops.kv_attention(q, cache, table, cu, lens, 1, 3001)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)


def test_kernels_without_dependent_launch(monkeypatch):
    """W4A16_PDL=0: the same bits."""
    step = Step(12, 4, 64, 64, [2500, 300], [2, 5], seed=20)
    cache = step.cache()
    want = step.run(cache=cache)
    monkeypatch.setenv("W4A16_PDL", "0")
    ops.lib().w4a16_debug_reload_env()
    try:
        assert torch.equal(step.run(cache=cache), want)
    finally:
        monkeypatch.delenv("W4A16_PDL")
        ops.lib().w4a16_debug_reload_env()


def test_counters_are_zeroed_after_a_timeout(monkeypatch):
    """What device_status does when a wait ran out (the flag word is faked; no kernel waits)."""
    step = Step(8, 2, 128, 32, [9000], [1], seed=21)
    cache = step.cache()
    want = step.run(cache=cache)
    for c, _ in ops._kv_counter_cache.values():
        c.fill_(3)
    ops._kv_capture_sets[0][0].fill_(5)

    class Lib:
        def __getattr__(self, name):
            return getattr(real, name)

        def w4a16_device_status(self, stream, flags):
            flags._obj.value = ops.DEVICE_TIMEOUT
            return ops.ERR_DEVICE

    real = ops.lib()
    with monkeypatch.context() as m:
        m.setattr(ops, "lib", lambda: Lib())
        assert ops.device_status() == ops.DEVICE_TIMEOUT
    assert torch.equal(step.run(cache=cache), want) and ops.device_status() == 0
