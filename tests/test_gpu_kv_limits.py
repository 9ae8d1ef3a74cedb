"""The paged attention at the ends of its ranges: lengths, windows, offsets, scales and workspaces."""
import pytest
import torch

from kv_cases import Step, assert_close, make_lengths, ref_plan
from skinny_gemm_gb300 import ops

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("hq,hkv,dim", [(8, 2, 128), (4, 4, 64)])
def test_windows_longer_than_any_request(hq, hkv, dim):
    """A window up to 2^31 - 1 is no window: prompts of several row tiles from an empty cache, and beside others."""
    step = Step(hq, hkv, dim, 16, [0, 3, 200, 0], [300, 130, 40, 1], seed=dim)
    cache = step.cache()
    want = step.run(cache=cache)
    ref, bound = step.reference()
    assert_close(want, ref, bound)
    for window in (max(step.lens), TOP - 33, TOP - 8, TOP - 1, TOP):
        assert torch.equal(step.run(window=window, cache=cache), want), window
    assert ops.device_status() == 0


@pytest.mark.parametrize("B,cut,T,hq,dim,max_len", [(5, 2, 1, 8, 128, 1024), (21, 2, 2, 8, 256, 384), (3, 2, 2, 4, 64, 5000),
                                                    (70, 50, 69, 8, 128, 2000), (2, 1, 40, 8, 128, 3000)])
def test_offsets_that_step_back_refuse_the_step(B, cut, T, hq, dim, max_len):
    """cu that decreases somewhere: the flag, zeros in every row, nothing outside the workspace; the next call is right."""
    hkv, block = 2, 16
    step = Step(hq, hkv, dim, block, [max_len - 1], [1], seed=B)
    cache = step.cache()
    table = torch.from_numpy(step.table).cuda().repeat(B, 1)
    q = torch.randn(T, hq, dim, device="cuda").to(torch.bfloat16)
    if B == T + 1:  # one request's end before its beginning, the others in order
        cu = [i if i < cut else i - 1 for i in range(B + 1)]
        cu[cut] = cut - 2
    else:
        cu = [T * (i % 2) for i in range(B + 1)]
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), max_len, dtype=torch.int32, device="cuda")
    n = ops.kv_attention_workspace_bytes(B, T, hq, cache, T, max_len)
    ws = torch.full((n + (1 << 20),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 7.0)
    ops.kv_attention(q, cache, table, cu, lens, T, max_len, out=out, workspace=ws[:n])
    assert ops.device_status() & ops.DEVICE_KV_RANGE
    assert bool((ws[n:] == 0xFF).all())
    assert torch.equal(out, torch.zeros_like(out))
    ref, bound = step.reference()
    assert_close(step.run(cache=cache, workspace=ws), ref, bound)
    assert ops.device_status() == 0


@pytest.mark.parametrize("B,new_max", [(6, 2), (5, 3000), (300, 60), (1500, 40)])
def test_lengths_advanced_in_place(B, new_max):
    """lens is the cached array, in steps of one and of many CTAs; twice in one captured graph."""
    block = 16
    cached, new = make_lengths(B, 300, new_max, B, block)
    need = sum(-(-(c + 2 * n) // block) for c, n in zip(cached, new))
    width = max(-(-(c + 2 * n) // block) for c, n in zip(cached, new))
    table = [[1000 + b * width + j if j * block < c else -1 for j in range(width)] for b, c in enumerate(cached)]
    free, T = list(range(500000, 500000 + need)), sum(new)
    lens, fresh, t, f = (torch.tensor(x, dtype=torch.int32).cuda() for x in (cached, new, table, free))
    plans = [ops.KVPlan.empty(B, T) for _ in range(2)]
    for p in plans:
        p.lens = lens
    start = lens.clone()

    def steps():
        ops.kv_plan(lens, fresh, t, f, T, block, out=plans[0])
        ops.kv_plan(lens, fresh, t, f, T, block, head=plans[0].head, out=plans[1])

    steps()
    for captured in (False, True):
        if captured:
            lens.copy_(start)
            t.copy_(torch.tensor(table, dtype=torch.int32))
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                steps()
            g.replay()
        tw, c, h = table, cached, 0
        for p in plans:
            tw, cu, c, slots, pos, h = ref_plan(c, new, tw, free, h, T, block)
            assert p.cu.tolist() == cu and p.slots.tolist() == slots and p.positions.tolist() == pos and p.head.tolist() == [h]
        assert t.tolist() == tw and lens.tolist() == c
    assert ops.device_status() == 0
