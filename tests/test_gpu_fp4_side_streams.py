"""Microscaled 4-bit calls with stream=: all that a call does of its own runs on that stream, whatever the current one is busy with."""
import zlib

import pytest
import torch

import fp4_cases as fc
from skinny_gemm_gb300 import ops

pytestmark = pytest.mark.gpu
BUSY = 200_000_000  # clocks, some 0.1 s


def gen(*seed):
    return torch.Generator().manual_seed(zlib.crc32(repr(seed).encode()))


def rows(seed, *shape):
    return fc.activations(gen(seed), shape[0] if len(shape) == 2 else shape[0] * shape[1], shape[-1]).view(shape).cuda()


def same(a, b):
    return torch.equal(a.codes, b.codes) and torch.equal(ops.fp4_dequant(a), ops.fp4_dequant(b))


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("shape", [(512, 320), (3, 130, 96)])
def test_gated_on_a_stream(fmt, shape):
    """The interleaved rows are made on the stream that quantises them: the current one is busy, and then uses the memory."""
    gate, up = rows(1, *shape), rows(2, *shape)
    both = torch.stack((gate, up), -2).flatten(-3, -2)
    want = ops.fp4_quant(both, fmt)
    s = torch.cuda.Stream()
    poison = torch.full_like(both, float("nan"))  # what memory of that size holds on the current stream
    torch.cuda.synchronize()
    del poison
    torch.cuda._sleep(BUSY)
    w = ops.FP4Matrix.gated(gate, up, fmt, stream=s)
    poison = torch.full_like(both, float("nan"))
    torch.cuda.synchronize()
    assert same(w, want) and same(ops.FP4Matrix.gated(gate, up, fmt), want)
    # and the other way round: the stream is busy while the current one goes on
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    w = ops.FP4Matrix.gated(gate, up, fmt, stream=s)
    again = [torch.full_like(both, float("nan")) for _ in range(3)]
    torch.cuda.synchronize()
    assert same(w, want) and len(again) == 3
    if len(shape) == 3:
        assert (w.E, w.N) == (shape[0], 2 * shape[1])
        values = ops.fp4_dequant(w).view(shape[0], shape[1], 2, shape[2])
        assert torch.equal(values[:, :, 0], ops.fp4_dequant(ops.fp4_quant(gate, fmt)))
        assert torch.equal(values[:, :, 1], ops.fp4_dequant(ops.fp4_quant(up, fmt)))


def calls(fmt):
    """Calls that allocate what they return, and a tensor of that."""
    x, w = rows(3, 128, 320), ops.fp4_quant(rows(4, 256, 320), fmt)
    experts, ids = ops.fp4_quant(rows(5, 4, 256, 320), fmt), torch.randint(0, 4, (128, 2), generator=gen(6), dtype=torch.int32).cuda()
    return [lambda s: ops.fp4_mm(x, w, stream=s), lambda s: ops.fp4_mm(x[:3], w, stream=s), lambda s: ops.fp4_mm(x[:40], w, stream=s), lambda s: ops.fp4_mm(ops.fp4_quant(x, fmt, stream=s), w, stream=s),
               lambda s: ops.fp4_gated(x, w, "silu", stream=s), lambda s: ops.fp4_mm_id(x, experts, ids, stream=s), lambda s: ops.fp4_dequant(w, stream=s),
               lambda s: ops.fp4_quant(x, fmt, stream=s)._flat] + ([lambda s: ops.fp4_quant(x, fmt, stream=s).row_scale] if fmt == "nv" else [])


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("which", range(9))
def test_results_made_on_a_stream(fmt, which):
    """A result's memory is not what the current stream still writes, and is not given away while the current stream still reads."""
    all_calls = calls(fmt)
    if which >= len(all_calls):
        return
    call, s = all_calls[which], torch.cuda.Stream()
    want = call(None).clone()
    call(s)  # (the stream's workspace is there)
    torch.cuda.synchronize()
    old = torch.empty_like(want)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    old.zero_().fill_(7)  # (later, to memory that the allocator has back)
    del old
    got = call(s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del got
    first = call(s)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    copy = first.clone()  # (later)
    del first
    with torch.cuda.stream(s):
        other = [torch.full_like(want, 9) for _ in range(3)]  # (now, to memory that the stream has to give)
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and len(other) == 3


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_captured_beside_the_capturing_stream(fmt):
    """Calls on a stream that a capture has forked, whose results and temporaries are made and given back in it."""
    x, w = rows(7, 70, 320), ops.fp4_quant(rows(8, 256, 320), fmt)
    want = [ops.fp4_mm(x, w), ops.fp4_gated(x[:3], w), ops.fp4_mm(ops.fp4_quant(x, fmt), w)]
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        got = [ops.fp4_mm(x, w, stream=s), ops.fp4_gated(x[:3], w, stream=s)]
        for _ in range(3):
            last = ops.fp4_mm(ops.fp4_quant(x, fmt, stream=s), w, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        total = got[0] + last
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip([*got, last], want)) and torch.equal(total, want[0] + want[2])
    again = [ops.fp4_mm(x, w, stream=s) for _ in range(20)]  # (the allocator goes on after the capture)
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[0]) for y in again) and ops.device_status() == 0
