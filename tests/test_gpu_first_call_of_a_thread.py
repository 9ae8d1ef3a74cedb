"""A host thread whose first CUDA call is one of the library's: nothing has made the device's context current in it."""
import threading

import pytest
import torch

from skinny_gemm_gb300 import ops, synth

pytestmark = pytest.mark.gpu


def bf16(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def four_bit(M, fmt="nv"):
    x, w = bf16(1, M, 512), ops.fp4_quant(bf16(2, 300, 512), fmt)
    q = ops.fp4_quant(x, fmt)
    return {"mm": lambda out: ops.fp4_mm(x, w, out=out), "mm_q": lambda out: ops.fp4_mm(q, w, out=out), "gated": lambda out: ops.fp4_gated(q, w, out=out)}


def affine(M):
    x, w = bf16(3, M, 512), ops.W4Matrix.from_host(synth.make_weights(4, 512, 512))
    return lambda out: ops.mm(x, w, out=out)


def attention():
    cache = ops.KVCache.empty(64, 2, 16, 64)
    ops.kv_append(bf16(5, 1024, 2, 64), bf16(6, 1024, 2, 64), cache, torch.arange(1024, dtype=torch.int32, device="cuda"))
    table = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 64)
    cu, lens = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([1024], dtype=torch.int32, device="cuda")
    q = bf16(7, 1, 8, 64)
    return lambda out: ops.kv_attention(q, cache, table, cu, lens, 1, 1024, out=out)


CALLS = {**{f"fp4_{name} {M}": lambda name=name, M=M: four_bit(M)[name] for name in ("mm", "mm_q", "gated") for M in (1, 40, 300)},
         **{f"mm {M}": lambda M=M: affine(M) for M in (1, 5, 64)}, "attention": attention}


@pytest.mark.parametrize("name", CALLS)
def test_first_call(name):
    call = CALLS[name]()
    want = call(None).clone()
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    errors = []

    def work():
        try:
            call(out)
        except Exception as e:  # noqa: BLE001 (told by the test)
            errors.append(e)

    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        t = threading.Thread(target=work)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert not errors and torch.equal(out, want), errors
    assert ops.device_status() == 0
