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


def _with_scales(step, exponents, zeros=()):
    """The step with V scales 2^e for its blocks in order of position (codes small enough for bf16 outputs), and blocks
    of zeros."""
    step.v = step.v.float().clamp(-200, 200).to(torch.float8_e4m3fn)
    for b, n in enumerate(step.lens):
        for j in range(-(-n // step.block)):
            i = int(step.table[b, j])
            step.vs[i] = 2.0 ** exponents[j % len(exponents)]
            if j in zeros:
                step.v[i] = 0
    return step


@pytest.mark.parametrize("high", [40, 70, 71, 100, 120])
@pytest.mark.parametrize("cached", [16, 130, 1030, 5000])
def test_value_scales_far_apart_keep_their_weight_in_the_sum(high, cached):
    """A block of zeros (scale 2^-64) beside scales up to 2^120, in one tile, in two, in two groups and in many: equal
    scores weigh the same whatever their V scales."""
    step = Step(4, 2, 128, 16, [cached], [1], seed=high)
    n = -(-step.lens[0] // 16)
    _with_scales(step, [-64] * (n - 1) + [high], zeros=range(n - 1))
    step.q[0, 0] = 0  # equal weights
    out = step.run()
    ref, bound = step.reference()
    assert_close(out, ref, bound, f"{high} {cached}")
    i = int(step.table[0, n - 1])
    m = step.lens[0] - 16 * (n - 1)
    want = step.v[i, 0, :m].double().sum(0) * 2.0 ** high / step.lens[0]
    assert bool(((out[0, 0].double().cpu() - want).abs() <= 2.0 ** -7 * step.v[i, 0, :m].double().abs().sum(0) * 2.0 ** high / step.lens[0]).all())
    assert ops.device_status() == 0


@pytest.mark.parametrize("hq,hkv,dim,block", [(8, 2, 128, 16), (8, 2, 256, 64), (28, 4, 64, 32)])
@pytest.mark.parametrize("exponents", [(-64, 120), (120, -64, 0, 37, -30), (-64, 3, 71), (0, -60, 60, 100)])
def test_value_scales_over_the_whole_range(hq, hkv, dim, block, exponents):
    """Scales from 2^-64 to 2^120 in any order, peaked and flat rows; and a verify row is the one-token step."""
    cached, M = [5, 300, 2600, 1020], 3
    step = _with_scales(Step(hq, hkv, dim, block, cached, [M] * 4, seed=block), exponents)
    cache = step.cache()
    for scale in (0.002, None, 1.0):
        out = step.run(cache=cache, scale=scale)
        ref, bound = step.reference(scale=scale)
        assert_close(out, ref, bound, f"{scale}")
        table = torch.from_numpy(step.table).cuda()
        cu = torch.arange(5, dtype=torch.int32).cuda()
        for m in range(M):
            lens = torch.tensor([c + m + 1 for c in cached], dtype=torch.int32).cuda()
            one = ops.kv_attention(step.q.view(4, M, hq, dim)[:, m].contiguous().cuda(), cache, table, cu, lens, 1,
                                   max(step.lens), scale=scale)
            assert torch.equal(one, out.view(4, M, hq, dim)[:, m]), (scale, m)


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("new,window", [(1, 200), (3, 1), (5, 130), (2, 1500)])
def test_the_longest_request(block, new, window):
    """The last tokens of a request of 2^31 - 1, seen through a window (its table repeats a few blocks)."""
    hq, hkv, dim, few = 4, 2, 64, 7
    step = Step(hq, hkv, dim, block, [few * block - 1], [1], seed=block + new)  # a cache of seven full blocks
    ids = [int(i) for i in step.table[0, :few]]
    width = (TOP + block) // block
    table = torch.tensor(ids, dtype=torch.int32, device="cuda").repeat(-(-width // few))[:width].view(1, -1)
    q = torch.randn(new, hq, dim, generator=torch.Generator().manual_seed(new)).to(torch.bfloat16)
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, new], [TOP]))
    out = ops.kv_attention(q.cuda(), step.cache(), table, cu, lens, new, TOP, window=window)
    assert ops.device_status() == 0
    for m in range(new):
        see = range(TOP - new + m - window + 1, TOP - new + m + 1)
        at = [(ids[p // block % few], p % block) for p in see]
        for h in range(hkv):
            k, v = (torch.stack([c[i, h, o].double() * s[i, h].double() for i, o in at]) for c, s in
                    ((step.k, step.ks), (step.v, step.vs)))
            w = torch.softmax(q[m, 2 * h:2 * h + 2].double() @ k.T / dim ** 0.5, 1)
            # as in the reference of these tests: the output's and the weights' rounding (the rest is below a hundredth)
            bound = 1.02 * 2.0 ** -8 * ((w @ v).abs() + w @ v.abs()) + 2.0 ** -20 * (w @ v.abs()).amax()
            assert bool(((out[m, 2 * h:2 * h + 2].double().cpu() - w @ v).abs() <= bound).all()), (m, h)


def test_a_negative_head_counts_as_zero_and_is_flagged():
    cached, new, table, free = [16, 0], [3, 20], [[5, -1], [-1, -1]], [7, 8, 9, 10]
    t, f = (torch.tensor(x, dtype=torch.int32).cuda() for x in (table, free))
    p = ops.kv_plan(*(torch.tensor(x, dtype=torch.int32).cuda() for x in (cached, new)), t, f, 23, 16,
                    head=torch.tensor([-3], dtype=torch.int32).cuda())
    assert ops.device_status() == ops.DEVICE_KV_RANGE
    want = ref_plan(cached, new, table, free, 0, 23, 16)
    assert (t.tolist(), p.cu.tolist(), p.lens.tolist(), p.slots.tolist(), p.positions.tolist(), int(p.head)) == want


@pytest.mark.parametrize("hq,hkv,dim,loose", [(32, 8, 64, 1 << 25), (64, 2, 256, 1 << 22), (12, 4, 128, 1 << 26)])
@pytest.mark.parametrize("window", [0, 700])
def test_rows_in_several_launches(hq, hkv, dim, loose, window):
    """A bound on the lengths that makes partial results outgrow one launch: the same bits as with a tight one, in ragged
    steps whose requests lie across launches, with padding rows and with requests that are left out."""
    block = 128
    cached, new = [0, 700, 3000, 5, 64, 1100, 0, 2500], [30, 1, 7, 0, 3, 40, 1, 9]
    step = Step(hq, hkv, dim, block, cached, new, seed=hq)
    cache, T = step.cache(), step.T + 3
    table, cu, lens = step.dev()
    wide = torch.full((len(new), loose // block), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = torch.cat([step.q, torch.ones(3, hq, dim, dtype=torch.bfloat16)]).cuda()
    want = ops.kv_attention(q, cache, table, cu, lens, max(new), max(step.lens), window=window)
    one = ops.kv_attention_workspace_bytes(len(new), 1, hq, cache, max(new), loose, window)
    n = ops.kv_attention_workspace_bytes(len(new), T, hq, cache, max(new), loose, window)
    assert n < 4.2 * (1 << 30) and (window > 0 or T * one > 2 * n)  # (several launches)
    out = torch.full_like(q, 7.0)
    assert torch.equal(ops.kv_attention(q, cache, wide, cu, lens, max(new), loose, window=window, out=out), want)
    assert bool((want[step.T:] == 0).all()) and ops.device_status() == 0
    ref, bound = step.reference(window=window)
    assert_close(out[:step.T], ref, bound)
    # the 30 and the 40 rows are too many, or the offsets step back
    few = ops.kv_attention(q, cache, wide, cu, lens, 9, loose, window=window)
    keep = torch.ones(T, dtype=torch.bool)
    keep[:30] = keep[41:81] = False
    assert ops.device_status() == ops.DEVICE_KV_RANGE
    assert torch.equal(few[keep], want[keep]) and bool((few[~keep] == 0).all())
    cu[4] = 3
    assert bool((ops.kv_attention(q, cache, wide, cu, lens, max(new), loose, window=window) == 0).all())
    assert ops.device_status() == ops.DEVICE_KV_RANGE
