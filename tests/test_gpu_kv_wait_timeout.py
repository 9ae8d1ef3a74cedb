"""The paged attention's bounded waits run out, on the GPU, without faulting it.

W4A16_FAULT=wait makes the first slot of keys of one CTA wait for an arrival
more than there will be.  Every copy still lands; all roles of that CTA give up
after about a second, wait (bounded) for what is in flight, free their tensor
memory and leave, and the flag is raised."""
import time

import pytest
import torch

from kv_cases import Step, assert_close
from skinny_gemm_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,dim,cached,new", [
    (4, 2, 64, [40], [1]),                      # one tile: the copies end before their slot is waited for
    (8, 2, 256, [9000, 3, 700], [1, 1, 1]),     # divided groups whose parts never come
    (28, 4, 128, [5000, 0, 900], [40, 60, 7]),  # several segments a CTA, staged queries ahead
    (8, 2, 128, [3000] * 40, [2] * 40)])        # two CTAs an SM, more tiles than slots
def test_waits_run_out_and_the_context_survives(hq, hkv, dim, cached, new, monkeypatch):
    step = Step(hq, hkv, dim, 64, cached, new, seed=hq)
    cache = step.cache()
    want = step.run(cache=cache)
    n = ops.kv_attention_workspace_bytes(len(new), step.T, hq, cache, max(new), max(step.lens))
    ws = torch.zeros(n + 4096, dtype=torch.uint8, device="cuda")
    assert ops.device_status() == 0
    monkeypatch.setenv("W4A16_FAULT", "wait")
    ops.lib().w4a16_debug_reload_env()
    try:
        t0 = time.perf_counter()
        step.run(cache=cache, workspace=ws[:n])
        flags = ops.device_status()  # synchronises: the kernel has ended
        elapsed = time.perf_counter() - t0
    finally:
        monkeypatch.delenv("W4A16_FAULT")
        ops.lib().w4a16_debug_reload_env()
    assert flags == ops.DEVICE_TIMEOUT, f"flags {flags:#x}: the planted wait did not run out"
    assert elapsed < 20, f"the bounded waits took {elapsed:.1f} s"
    assert bool((ws[n:] == 0).all())
    for c, _ in ops._kv_counter_cache.values():
        assert int(c.abs().max()) == 0
    assert torch.equal(step.run(cache=cache), want) and ops.device_status() == 0
    if hkv == 2 and dim != 128:
        ref, bound = step.reference()
        assert_close(want, ref, bound)
