"""Calls with stream= that allocate what they return: that is the stream's memory, whatever the current one is busy with."""
import pytest
import torch

from skinny_gemm_gb300 import ops, synth

pytestmark = pytest.mark.gpu
BUSY = 200_000_000  # clocks, some 0.1 s


def bf16(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def affine():
    w, e = ops.W4Matrix.from_host(synth.make_weights(1, 512, 512)), ops.W4Matrix.from_host(synth.make_weights(2, 256, 512, 3))
    x, ids = bf16(3, 40, 512), torch.arange(40, dtype=torch.int32, device="cuda") % 3
    return {"mm": lambda s: ops.mm(x, w, stream=s), "mm_argmax": lambda s: ops.mm_argmax(x, w, stream=s)[0], "mm_argmax values": lambda s: ops.mm_argmax(x, w, stream=s)[1],
            "mm_group": lambda s: ops.mm_group([x, x], [w, w], stream=s)[1], "mm_id": lambda s: ops.mm_id(x, e, ids, stream=s), "embed": lambda s: ops.embed(ids, w, stream=s),
            "unpack": lambda s: ops.unpack(w, stream=s), "dequant": lambda s: ops.dequant(w, stream=s)}


def ternary():
    blocks = torch.from_numpy(synth.make_stq1(4, 64, 512).reshape(-1).copy()).cuda()
    w, e = ops.STQ1Matrix.from_blocks(blocks, 64, 512), ops.STQ1Matrix.from_host(synth.make_stq1(5, 64, 512, 3), 64, 512, 3)
    x, ids = bf16(6, 40, 512).float(), torch.arange(40, dtype=torch.int32, device="cuda") % 3
    return {"stq1_mm": lambda s: ops.stq1_mm(x, w, stream=s), "stq1_mm_id": lambda s: ops.stq1_mm_id(x, e, ids, stream=s),
            "stq1_get_rows": lambda s: ops.stq1_get_rows(ids, w, stream=s), "stq1 from_blocks": lambda s: ops.STQ1Matrix.from_blocks(blocks, 64, 512, stream=s).packed}


def cache():
    c = ops.KVCache.empty(64, 2, 16, 64)
    ops.kv_append(bf16(7, 1024, 2, 64), bf16(8, 1024, 2, 64), c, torch.arange(1024, dtype=torch.int32, device="cuda"))
    table = torch.arange(64, dtype=torch.int32, device="cuda").view(2, 32)
    cu, lens = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 40, 41], [512, 300]))
    q = bf16(9, 41, 8, 64)
    new, free = torch.tensor([3, 2], dtype=torch.int32, device="cuda"), torch.arange(64, dtype=torch.int32, device="cuda")
    at = torch.tensor([40, 500], dtype=torch.int32, device="cuda")
    return {"kv_attention": lambda s: ops.kv_attention(q, c, table, cu, lens, 40, 512, stream=s),
            "kv_plan": lambda s: ops.kv_plan(at, new, table.clone() if s is None else table, free, 5, 16, stream=s).positions}


CALLS = {**dict.fromkeys(("mm", "mm_argmax", "mm_argmax values", "mm_group", "mm_id", "embed", "unpack", "dequant"), affine),
         **dict.fromkeys(("stq1_mm", "stq1_mm_id", "stq1_get_rows", "stq1 from_blocks"), ternary), "kv_attention": cache, "kv_plan": cache}


@pytest.mark.parametrize("name", CALLS)
def test_results_made_on_a_stream(name):
    """A result's memory is not what the current stream still writes, and is not given away while the current stream still reads."""
    call, s = CALLS[name]()[name], torch.cuda.Stream()
    want = call(None).clone()
    torch.cuda.synchronize()
    call(s)  # (the stream's workspace is there)
    torch.cuda.synchronize()
    n = -(-want.untyped_storage().nbytes() // 512) * 512
    old = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for t in old:
        t.fill_(7)  # (later, to memory that the allocator has back)
    del old, t
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
        other = [torch.full((n,), 9, dtype=torch.uint8, device="cuda") for _ in range(4)]  # (now, to memory that the stream has to give)
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and len(other) == 4 and ops.device_status() == 0
