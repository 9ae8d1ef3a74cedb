"""The paged cache's calls take tensors of one device, the current one (stand-ins for CUDA tensors; no GPU)."""
import contextlib

import pytest
import torch

from skinny_gemm_gb300 import ops


class On(torch.Tensor):
    """A host tensor that says it is on a CUDA device."""

    where = 0
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.where))

    def get_device(self):
        return self.where


def on(where, *shape, dtype=torch.int32):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(On)
    t.where = where
    return t


class Lib:
    calls = 0

    def __getattr__(self, name):
        def call(*args):
            Lib.calls += 1
            return 256 if name.endswith("bytes") else ops.OK
        return call


class Stream:
    cuda_stream = 7

    def __init__(self, index):
        self.device_index = index


@pytest.fixture()
def current(monkeypatch):
    """Device 0 is the current one; nothing is launched."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 5, raising=False)
    monkeypatch.setattr(ops, "lib", lambda: Lib())
    monkeypatch.setattr(ops, "_kv_counters", lambda raw, device: (None, 0))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    Lib.calls = 0


def _cache(where):
    f8, f32 = torch.float8_e4m3fn, torch.float32
    return ops.KVCache(*(on(where, 4, 2, 16, 64, dtype=f8) for _ in range(2)), *(on(where, 4, 2, dtype=f32) for _ in range(2)))


def _plan(at=0, stream=None, **other):
    w = {n: other.get(n, at) for n in ("cached", "new", "table", "free", "head", "cu", "lens", "slots", "positions", "head_out")}
    out = ops.KVPlan(on(w["cu"], 4), on(w["lens"], 3), on(w["slots"], 5), on(w["positions"], 5), on(w["head_out"], 1))
    return ops.kv_plan(on(w["cached"], 3), on(w["new"], 3), on(w["table"], 3, 2), on(w["free"], 9), 5, 16,
                       head=on(w["head"], 1), out=out, stream=stream)


def _append(at=0, stream=None, **other):
    w = {n: other.get(n, at) for n in ("k", "v", "cache", "slots")}
    bf = torch.bfloat16
    return ops.kv_append(on(w["k"], 5, 2, 64, dtype=bf), on(w["v"], 5, 2, 64, dtype=bf), _cache(w["cache"]), on(w["slots"], 5),
                         stream=stream)


def _attend(at=0, stream=None, **other):
    w = {n: other.get(n, at) for n in ("q", "cache", "table", "cu", "lens", "out", "workspace")}
    bf = torch.bfloat16
    return ops.kv_attention(on(w["q"], 5, 4, 64, dtype=bf), _cache(w["cache"]), on(w["table"], 3, 2), on(w["cu"], 4),
                            on(w["lens"], 3), 2, 32, out=on(w["out"], 5, 4, 64, dtype=bf), stream=stream,
                            workspace=on(w["workspace"], 256, dtype=torch.uint8))


@pytest.mark.parametrize("call,names", [
    (_plan, ("cached", "new", "table", "free", "head", "cu", "lens", "slots", "positions", "head_out")),
    (_append, ("k", "v", "cache", "slots")),
    (_attend, ("q", "cache", "table", "cu", "lens", "out", "workspace"))])
def test_one_device(current, call, names):
    call()
    assert Lib.calls == 1
    call(stream=Stream(0))
    assert Lib.calls == 2
    for n in names:
        with pytest.raises(ValueError, match="cuda:"):
            call(**{n: 1})
    with pytest.raises(ValueError, match="cuda:1"):
        call(at=1)  # all together, but not on the current device
    with pytest.raises(ValueError, match="cuda:0"):
        call(stream=Stream(1))
    with pytest.raises(ValueError, match="cuda:1"):
        call(at=1, stream=Stream(1))  # (the library launches on the current device)
    assert Lib.calls == 2


def test_counters_of_the_device_whose_wait_ran_out(current, monkeypatch):
    """Only they are zeroed, and only when that device is idle: another device's calls may be running."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: type("S", (), {"cuda_stream": 3, "synchronize": lambda self: None})())
    idle = []
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: idle.append(0))
    counters = {(d, s): (torch.full((4,), 9), 0) for d in (0, 1) for s in (5, 6)}
    sets = {d: [torch.full((8,), 9), 2] for d in (0, 1)}
    monkeypatch.setattr(ops, "_kv_counter_cache", counters)
    monkeypatch.setattr(ops, "_kv_capture_sets", sets)

    class Out(Lib):
        def w4a16_device_status(self, stream, flags):
            flags._obj.value = ops.DEVICE_TIMEOUT
            return ops.ERR_DEVICE

    monkeypatch.setattr(ops, "lib", lambda: Out())
    assert ops.device_status() == ops.DEVICE_TIMEOUT and idle
    for d in (0, 1):
        for t in [c[0] for k, c in counters.items() if k[0] == d] + [sets[d][0]]:
            assert bool((t == 9 * d).all()), d
