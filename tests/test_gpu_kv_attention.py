"""w4a16_kv_attention against softmax attention in 64 bits (tests/kv_cases.py derives the bound), and its guarantees."""
import numpy as np
import pytest
import torch

from kv_cases import Step, assert_close, make_lengths
from skinny_gemm_gb300 import ops

pytestmark = pytest.mark.gpu

HEADS = [(8, 2, 256), (4, 1, 256), (8, 8, 128), (28, 4, 128), (12, 4, 64), (3, 3, 64), (32, 1, 128), (16, 1, 256),
         (5, 1, 256), (64, 8, 128)]


def _check(step, window=0, scale=None, what=""):
    out = step.run(window=window, scale=scale)
    ref, bound = step.reference(window=window, scale=scale)
    r = assert_close(out, ref, bound, what)
    assert ops.device_status() == 0
    return r


@pytest.mark.parametrize("hq,hkv,dim", HEADS)
@pytest.mark.parametrize("block", [16, 64])
def test_decode(hq, hkv, dim, block):
    """One new token a request; lengths 1, around blocks' and tiles' ends, and a few hundred."""
    lens = [1, 2, block - 1, block, block + 1, 127, 128, 129, 255, 256, 300, 777]
    _check(Step(hq, hkv, dim, block, [n - 1 for n in lens], [1] * len(lens), seed=hq + block))


@pytest.mark.parametrize("hq,hkv,dim,block", [(8, 2, 256, 64), (28, 4, 128, 32), (12, 4, 64, 128), (32, 1, 128, 16)])
@pytest.mark.parametrize("M", [2, 3, 5, 8, 17])
def test_verify(hq, hkv, dim, block, M):
    """M new tokens a request, from the request's first token on."""
    cached = [0, 1, 126, 127, 500, 1020]
    _check(Step(hq, hkv, dim, block, cached, [M] * len(cached), seed=M))


@pytest.mark.parametrize("hq,hkv,dim,block", [(8, 2, 256, 32), (8, 8, 128, 16), (12, 4, 64, 64)])
def test_ragged_chunks(hq, hkv, dim, block):
    """Prompt chunks of 0 to 200 tokens over 0 to 600 cached ones, in one call."""
    cached, new = make_lengths(5, 600, 200, dim, block)
    _check(Step(hq, hkv, dim, block, cached, new, seed=dim))


@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 700])
@pytest.mark.parametrize("hq,hkv,dim,block", [(8, 2, 256, 16), (14, 2, 128, 64)])
def test_window(hq, hkv, dim, block, window):
    cached = [0, 5, 99, 127, 128, 640, 1300]
    _check(Step(hq, hkv, dim, block, cached, [3, 1, 5, 2, 4, 8, 3], seed=window), window=window)


def test_long_cache():
    """A request long enough to be split over every SM, beside short ones."""
    _check(Step(8, 2, 256, 64, [20000, 3, 1000], [1, 2, 1], seed=4))
    _check(Step(8, 8, 128, 16, [9000], [3], seed=5), window=8000)


def test_many_requests():
    cached, new = make_lengths(150, 300, 3, 6, 16)
    _check(Step(8, 2, 128, 16, cached, new, seed=6))


def test_scales_far_apart():
    """Block scales that differ by up to 2^20 within a tile, and score scales from tiny to peaked."""
    step = Step(8, 2, 128, 16, [700, 90], [2, 3], seed=7, scale_spread=20)
    _check(step, what="spread")
    step = Step(8, 2, 256, 16, [700, 90], [2, 3], seed=8)
    for scale in (1e-6, 0.01, 1.0, 8.0):
        _check(step, scale=scale, what=f"scale {scale}")


def test_peaked_and_uniform_rows():
    """Rows where one token takes all the weight, and rows of equal weights over a long cache (a sink and a tail)."""
    step = Step(8, 1, 128, 64, [3000], [2], seed=9)
    step.q[0] = 0  # uniform weights
    _check(step)
    k0 = step.k.float()
    i = int(step.table[0, 0])
    k0[i, 0, 0] = 448.0 * torch.sign(step.q[1, 0].float())  # head 0 of the second row: the first token above all others
    step.k = k0.to(torch.float8_e4m3fn)
    step.ks[i, 0] = 2.0 ** -4
    _check(step)


def test_large_and_tiny_queries():
    """Query rows with an outlier of 2^12 times the rest, tiny rows, and a zero row."""
    step = Step(4, 1, 256, 64, [400], [4], seed=10)
    step.q[0, :, 17] = 2.0 ** 12
    step.q[1] *= 2.0 ** -60
    step.q[2] = 0
    step.q[3] *= 2.0 ** 6
    _check(step, scale=2.0 ** -9)


def test_nan_where_a_row_does_not_look():
    """NaN codes in tokens of later rows and before the window: earlier rows keep their values; rows that see a NaN
    key are NaN; rows that see a NaN value are NaN in that column."""
    step = Step(8, 2, 128, 32, [150, 40], [4, 4], seed=11)
    want = step.run()
    cache = step.cache()
    for b in range(2):
        for pos, what in ((step.lens[b] - 1, cache.k), (step.lens[b] - 2, cache.v)):
            i = int(step.table[b, pos // 32])
            what[i, :, pos % 32, 5] = float("nan")
    got = step.run(cache=cache)
    for b in range(2):
        t = int(step.cu[b])
        assert torch.equal(got[t:t + 2], want[t:t + 2])
        g, w = got[t + 2].float(), want[t + 2].float()  # sees the NaN value, not the NaN key
        assert torch.isnan(g[:, 5]).all()
        keep = torch.ones(128, dtype=torch.bool, device=g.device)
        keep[5] = False
        assert torch.equal(g[:, keep], w[:, keep])
        assert torch.isnan(got[t + 3].float()).all()
    # before the window
    step = Step(8, 2, 128, 32, [150], [3], seed=12)
    want, cache = step.run(window=20), step.cache()
    cache.v[int(step.table[0, 129 // 32]), :, 129 % 32] = float("nan")
    cache.k[int(step.table[0, 130 // 32]), :, 130 % 32] = float("nan")
    assert torch.equal(step.run(window=20, cache=cache), want)


def test_non_finite_queries_stay_in_their_row():
    step = Step(8, 2, 256, 64, [200, 100], [2, 2], seed=13)
    want = step.run()
    step.q[1, 3, 7], step.q[2, 0, 0] = float("inf"), float("nan")
    got = step.run()
    bad = torch.zeros(4, 8, dtype=torch.bool, device=got.device)
    bad[1, 3] = bad[2, 0] = True
    assert torch.isnan(got[bad].float()).all()
    assert torch.equal(got[~bad], want[~bad])


def test_rows_that_see_nothing():
    """Padding rows, requests without new tokens, and requests whose blocks are all missing give zeros."""
    step = Step(8, 2, 128, 16, [50, 0, 30], [2, 0, 1], seed=14)
    table, cu, lens = step.dev()
    q = torch.cat([step.q, torch.full((5, 8, 128), float("nan"), dtype=torch.bfloat16)]).cuda()
    out = torch.full_like(q, 7.0)
    ops.kv_attention(q, step.cache(), table, cu, lens, 2, 64, out=out)
    assert ops.device_status() == 0
    ref, bound = step.reference()
    assert_close(out[:3], ref, bound)
    assert torch.equal(out[3:], torch.zeros_like(out[3:]))
    table[2] = -1
    table[0, 1] = 10 ** 9
    ops.kv_attention(q, step.cache(), table, cu, lens, 2, 64, out=out)
    assert ops.device_status() & ops.DEVICE_KV_RANGE
    assert torch.equal(out[2:], torch.zeros_like(out[2:]))
    # tokens 16..31 of request 0 are not there: the rest attends as if they were masked
    step.table[0, 1] = step.table[0, 0]
    keep = step.ks.clone()
    assert torch.isfinite(out[:2].float()).all()
    ids = [int(i) for i in step.table[0, :4]]
    see = [p for p in range(51) if not 16 <= p < 32]
    k = torch.stack([step.k[ids[p // 16], 0, p % 16].double() * keep[ids[p // 16], 0].double() for p in see])
    v = torch.stack([step.v[ids[p // 16], 0, p % 16].double() * step.vs[ids[p // 16], 0].double() for p in see])
    w = torch.softmax(step.q[0, 0].double() @ k.T / 128 ** 0.5, 0)
    err = (out[0, 0].double().cpu() - w @ v).abs()
    assert bool((err <= 2.0 ** -8 * (w @ v).abs() + 2.0 ** -7 * (w @ v.abs())).all())


def test_bounds_that_do_not_hold_are_flagged():
    """Requests longer than max_len or with more rows than max_new: their rows are zeros, the others' are right."""
    step = Step(8, 2, 128, 16, [50, 300, 20], [1, 1, 3], seed=15)
    table, cu, lens = step.dev()
    ref, bound = step.reference()
    out = ops.kv_attention(step.q.cuda(), step.cache(), table, cu, lens, 3, 100)
    assert ops.device_status() & ops.DEVICE_KV_RANGE
    assert_close(out[[0, 2, 3, 4]], ref[[0, 2, 3, 4]], bound[[0, 2, 3, 4]])
    assert torch.equal(out[1], torch.zeros_like(out[1]))
    out = ops.kv_attention(step.q.cuda(), step.cache(), table, cu, lens, 1, 304)
    assert ops.device_status() & ops.DEVICE_KV_RANGE
    assert_close(out[:2], ref[:2], bound[:2])
    assert torch.equal(out[2:], torch.zeros_like(out[2:]))


@pytest.mark.parametrize("hq,hkv,dim", [(8, 2, 256), (28, 4, 128), (12, 4, 64), (16, 1, 128)])
@pytest.mark.parametrize("window", [0, 150])
def test_verify_rows_equal_single_token_steps(hq, hkv, dim, window):
    """Row m of an M-row step equals, bit for bit, the one-token step at its position over the same cache, alone or
    in another batch."""
    cached, M = [0, 100, 126, 900, 1021, 2045, 2600], 7
    step = Step(hq, hkv, dim, 16, cached, [M] * len(cached), seed=hq)
    cache = step.cache()
    whole = step.run(window=window, cache=cache).view(len(cached), M, hq, dim)
    table = torch.from_numpy(step.table).cuda()
    q = step.q.cuda().view(len(cached), M, hq, dim)
    B = len(cached)
    for m in (0, 3, M - 1):
        cu = torch.arange(B + 1, dtype=torch.int32).cuda()
        lens = torch.tensor([c + m + 1 for c in cached], dtype=torch.int32).cuda()
        one = ops.kv_attention(q[:, m].contiguous(), cache, table, cu, lens, 1, 2607, window=window)
        assert torch.equal(one.view(torch.int16), whole[:, m].contiguous().view(torch.int16)), m
        for b in (1, 3, 6):
            alone = ops.kv_attention(q[b, m:m + 1], cache, table[b:b + 1], cu[:2], lens[b:b + 1], 1, cached[b] + m + 1,
                                     window=window)
            assert torch.equal(alone.view(torch.int16), one[b:b + 1].view(torch.int16)), (m, b)


def test_calls_repeat_bit_for_bit():
    step = Step(8, 2, 256, 64, [5000, 17], [5, 2], seed=16)
    cache = step.cache()
    a = step.run(cache=cache)
    for _ in range(3):
        assert torch.equal(step.run(cache=cache), a)


def test_strided_queries_streams_graphs_and_guards():
    """The q columns of a fused projection; another stream than the tensors' own; a captured call; no write outside
    the output and the workspace."""
    step = Step(8, 2, 128, 32, [700, 64, 5], [3, 1, 2], seed=17)
    cache = step.cache()
    table, cu, lens = step.dev()
    want = step.run(cache=cache)
    fused = torch.randn(step.T, 12 * 128, device="cuda").to(torch.bfloat16)
    fused[:, :8 * 128] = step.q.cuda().view(step.T, -1)
    q = fused[:, :8 * 128].view(step.T, 8, 128)
    assert torch.equal(ops.kv_attention(q, cache, table, cu, lens, 3, 703), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    on_s = ops.kv_attention(q, cache, table, cu, lens, 3, 703, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(on_s, want)
    n = ops.kv_attention_workspace_bytes(3, step.T, 8, cache, 3, 703)
    ws = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    buf = torch.full((step.T + 8, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[4:4 + step.T]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.kv_attention(q, cache, table, cu, lens, 3, 703, out=out, workspace=ws[:n])
    for _ in range(2):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    assert bool((buf[:4] == 3.0).all()) and bool((buf[-4:] == 3.0).all()) and bool((ws[n:] == 0xA5).all())


def test_a_cache_past_two_to_the_31_bytes():
    """Blocks whose bytes lie past 2^31 in K and V."""
    heads, block, dim = 2, 64, 256
    blocks = (1 << 31) // (heads * block * dim) + 200
    cache = ops.KVCache(*(torch.zeros(blocks, heads, block, dim, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                          for _ in range(2)),
                        *(torch.ones(blocks, heads, dtype=torch.float32, device="cuda") for _ in range(2)))
    step = Step(8, 2, dim, block, [250, 70], [1, 2], seed=18)
    far = blocks - step.k.shape[0]
    cache.k[far:], cache.v[far:] = step.k.cuda(), step.v.cuda()
    cache.k_scale[far:], cache.v_scale[far:] = step.ks.cuda(), step.vs.cuda()
    want = step.run()
    table, cu, lens = step.dev()
    got = ops.kv_attention(step.q.cuda(), cache, torch.where(table >= 0, table + far, table), cu, lens, 2, 251)
    assert torch.equal(got, want)
    x = torch.randn(1, 2, dim, device="cuda").to(torch.bfloat16)
    ops.kv_append(x, x, cache, torch.tensor([(blocks - 1) * block], dtype=torch.int32, device="cuda"))
    assert bool((cache.k[blocks - 1, :, 0].float() != 0).any())
    assert ops.device_status() == 0
