"""Which stream's memory the microscaled 4-bit calls with stream= allocate (stand-ins for CUDA tensors; no GPU)."""
import contextlib

import pytest
import torch

from skinny_gemm_gb300 import ops
from test_kv_devices_cpu import Stream, current, on  # noqa: F401  (fixture)


@pytest.fixture()
def streams(current, monkeypatch):  # noqa: F811
    """The streams that are current ones, the innermost last."""
    inside = []

    @contextlib.contextmanager
    def as_current(s):
        inside.append(s)
        yield
        inside.pop()

    monkeypatch.setattr(torch.cuda, "stream", as_current)
    return inside


@pytest.mark.parametrize("shape", [(4, 64), (2, 3, 64)])
def test_gated_rows_are_made_on_the_stream(streams, monkeypatch, shape):
    gate, up = on(0, *shape, dtype=torch.bfloat16), on(0, *shape, dtype=torch.bfloat16)
    stack, made = torch.stack, []
    monkeypatch.setattr(torch, "stack", lambda *a: made.append(list(streams)) or stack(*a))
    monkeypatch.setattr(ops, "fp4_quant", lambda x, format, stream=None: (tuple(x.shape), stream))
    s = Stream(0)
    assert ops.FP4Matrix.gated(gate, up, stream=s) == ((*shape[:-2], 2 * shape[-2], 64), s) and made == [[s]]
    assert ops.FP4Matrix.gated(gate, up)[1] is None and made == [[s], []]
    with pytest.raises(ValueError):
        ops.FP4Matrix.gated(gate, up, stream=Stream(1))
    assert len(made) == 2


def test_results_are_made_on_the_stream(streams, monkeypatch):
    """... and the stream that was current keeps them from being given back while it reads; a call without stream= does neither."""
    made, kept, here = [], [], Stream(0)

    class Made(torch.Tensor):
        def record_stream(self, s):
            kept.append(s)

    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: made.append(list(streams)) or torch.zeros(shape, dtype=dtype).as_subclass(Made))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: here)
    s = Stream(0)
    m = ops.FP4Matrix.empty(3, 64, stream=s)
    assert made == [[s], [s]] and kept == [here, here] and (m.N, m.K) == (3, 64)
    ops.FP4Matrix.empty(3, 64, format="mx", stream=here)
    assert made[2:] == [[here]] and len(kept) == 2  # (the current one: nothing to tell)
    ops.FP4Matrix.empty(3, 64)
    assert made[3:] == [[], []] and len(kept) == 2
