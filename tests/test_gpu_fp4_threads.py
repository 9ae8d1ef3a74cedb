"""Host threads that call on one stream: PyTorch's current stream is the same one in all of them, and so is its workspace."""
import threading
import zlib

import pytest
import torch

import fp4_cases as fc
from skinny_gemm_gb300 import ops

pytestmark = pytest.mark.gpu


def gen(*seed):
    return torch.Generator().manual_seed(zlib.crc32(repr(seed).encode()))


def at_once(calls, rounds, stream=None):
    """Each call `rounds` times in a thread of its own, all on one stream; every result is the bits of the call by itself."""
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got, errors, start = [[] for _ in calls], [], threading.Barrier(len(calls))

    def work(i):
        try:
            with torch.cuda.stream(stream):
                start.wait(60)
                for _ in range(rounds):
                    got[i].append(calls[i]())
        except Exception as e:  # noqa: BLE001 (told by the test)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    wrong = [sum(not torch.equal(y, w) for y in g) for g, w in zip(got, want)]
    assert wrong == [0] * len(calls) and ops.device_status() == 0


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M", [40, 300])
def test_products(fmt, M):
    """The same sizes and weights, other rows."""
    w = ops.fp4_quant(fc.activations(gen(1), 256, 512).cuda(), fmt)
    xs = [fc.activations(gen(2, i), M, 512).cuda() for i in range(3)]
    at_once([lambda x=x: ops.fp4_mm(x, w) for x in xs], 400)


def test_products_of_several_sizes():
    """Rows quantised in the product, before it, and by the caller; gated ones; on a stream that is not the default one."""
    w, d = (ops.fp4_quant(fc.activations(gen(3, n), n, 512).cuda()) for n in (640, 130))
    x = [fc.activations(gen(4, m), m, 512).cuda() for m in (2, 20, 64, 333)]
    q = ops.fp4_quant(x[2])
    s = torch.cuda.Stream()
    at_once([lambda: ops.fp4_mm(x[0], w), lambda: ops.fp4_gated(x[1], w, "gelu"), lambda: ops.fp4_mm(q, d), lambda: ops.fp4_gated(x[3], w)], 300, s)
    at_once([lambda: ops.fp4_mm(x[1], d, stream=s), lambda: ops.fp4_mm(x[2], w, stream=s), lambda: ops.fp4_mm(x[3], d, stream=s)], 300)


@pytest.mark.parametrize("T,top,E", [(40, 2, 6), (300, 4, 9), (1100, 1, 3)])
def test_routed(T, top, E):
    """Other routes of other tokens; a launch for the places, the quantiser's and the product's."""
    w = ops.fp4_quant(fc.activations(gen(5), E * 130, 256).view(E, 130, 256).cuda())
    calls = []
    for i, t in enumerate((T, T, T // 2)):
        x = fc.activations(gen(6, i), t, 256).cuda()
        ids = torch.randint(0, E, (t, top), generator=gen(7, i), dtype=torch.int32).cuda()
        calls.append(lambda x=x, ids=ids: ops.fp4_mm_id(x, w, ids))
    at_once(calls, 200)


def test_beside_attention():
    """The paged cache's attention has the same workspace: partial results, and a second launch that joins them."""
    B, hq, hkv, dim, block, n = 2, 8, 2, 64, 16, 2000
    cache = ops.KVCache.empty(B * n // block, hkv, block, dim)
    table = torch.arange(B * n // block, dtype=torch.int32, device="cuda").view(B, -1)
    slots = torch.arange(B * n, dtype=torch.int32, device="cuda")
    ops.kv_append(*(torch.randn(B * n, hkv, dim, generator=gen(8, i)).to(torch.bfloat16).cuda() for i in range(2)), cache, slots)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = [torch.randn(B, hq, dim, generator=gen(9, i)).to(torch.bfloat16).cuda() for i in range(2)]
    w, x = ops.fp4_quant(fc.activations(gen(10), 256, 512).cuda()), fc.activations(gen(11), 100, 512).cuda()
    at_once([lambda: ops.kv_attention(q[0], cache, table, cu, lens, 1, n), lambda: ops.fp4_mm(x, w), lambda: ops.kv_attention(q[1], cache, table, cu, lens, 1, n)], 300)
