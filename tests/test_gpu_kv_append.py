"""w4a16_kv_append against the definition in 64 bits: codes and scales are equal, not near."""
import math

import numpy as np
import pytest
import torch

from kv_cases import FINITE, need_scale, ref_append, round_e4m3
from skinny_gemm_gb300 import ops

pytestmark = pytest.mark.gpu


def test_the_rounding_reference():
    """round_e4m3 gives the nearest value, by search over all of them (ties to the even code)."""
    r = np.random.RandomState(0)
    y = np.concatenate([r.uniform(-448, 448, 2000), np.ldexp(r.uniform(-1, 1, 2000), r.randint(-12, 9, 2000)),
                        (FINITE[1:] + FINITE[:-1]) / 2])
    got = round_e4m3(y)
    d = np.abs(y[:, None] - FINITE[None])
    assert np.array_equal(np.abs(y - got), d.min(1)) and np.isin(got, FINITE).all()
    ties = round_e4m3((FINITE[1:] + FINITE[:-1]) / 2)
    codes = torch.tensor(ties).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.all(codes % 2 == 0)


def _fill(blocks, heads, block, dim, seed):
    g = torch.Generator().manual_seed(seed)
    k, v = ((torch.randn(blocks, heads, block, dim, generator=g) * 80).clamp(-448, 448).to(torch.float8_e4m3fn)
            for _ in range(2))
    ks, vs = (torch.exp2(torch.randint(-9, -4, (blocks, heads), generator=g).float()) for _ in range(2))
    return k, v, ks, vs


def _check(k_new, v_new, slots, heads, dim, block, blocks, seed=0, dev=None):
    k, v, ks, vs = _fill(blocks, heads, block, dim, seed)
    cache = ops.KVCache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda())
    kd, vd = dev if dev is not None else (k_new.cuda(), v_new.cuda())
    ops.kv_append(kd, vd, cache, torch.tensor(slots, dtype=torch.int32).cuda())
    for x, codes, scale, gc, gs in ((k_new, k, ks, cache.k, cache.k_scale), (v_new, v, vs, cache.v, cache.v_scale)):
        c, s = codes.double().numpy().copy(), scale.double().numpy().copy()
        ref_append(x.double().numpy(), slots, c, s, block)
        assert np.array_equal(gs.double().cpu().numpy(), s)
        assert np.array_equal(gc.double().cpu().numpy(), c, equal_nan=True)
    return cache


def _slots(runs, block):
    """[(block id, offset, tokens)] as slots."""
    return [i * block + o + j for i, o, n in runs for j in range(n)]


@pytest.mark.parametrize("heads,dim", [(1, 64), (2, 256), (3, 128), (8, 128)])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_runs(heads, dim, block):
    """Runs of every kind: one token, part of a block, whole blocks, after held rows (some scales grow, some stay)."""
    runs = [(3, 0, 1), (5, block - 1, 1), (6, 0, 5), (9, 2, 5), (0, 0, block), (1, 0, block), (2, 0, 3),
            (4, 7, block - 7), (7, 1, 1), (8, block // 2, 4), (11, 1, 9)]
    slots = _slots(runs, block)
    g = torch.Generator().manual_seed(dim + block)
    size = torch.exp2(torch.randint(-3, 3, (len(slots), heads, 1), generator=g).float())
    k, v = ((torch.randn(len(slots), heads, dim, generator=g) * size).to(torch.bfloat16) for _ in range(2))
    _check(k, v, slots, heads, dim, block, 12, seed=block)
    assert ops.device_status() == 0


@pytest.mark.parametrize("n", [1, 2, 4, 5, 31, 32, 33, 64, 100])
def test_run_lengths_and_a_growing_scale(n):
    """A run after held rows whose scale grows by 1 to 2^20: subnormal codes round to even, tiny ones vanish."""
    block, heads, dim = 128, 2, 256
    for grow in (0, 1, 4, 9, 20):
        slots = _slots([(1, 17, n)], block)
        g = torch.Generator().manual_seed(n + grow)
        x = (torch.randn(n, heads, dim, generator=g) * 2.0 ** (grow + 1)).to(torch.bfloat16)
        _check(x, -x, slots, heads, dim, block, 3, seed=n)


def test_every_bf16_magnitude_sets_the_scale():
    """The scale rule at every bf16 exponent and significand around 448 * 2^e (zero and subnormals: 2^-64)."""
    bits = torch.arange(0, 0x7F80, 7, dtype=torch.int32)
    near = torch.tensor([(e << 7) + m for e in range(0, 255) for m in (0, 95, 96, 97, 127)], dtype=torch.int32)
    x = torch.cat([bits, near])
    x = x[: x.numel() // 8 * 8].to(torch.int16).view(torch.bfloat16)
    T = x.numel()
    rows = torch.zeros(T, 1, 64, dtype=torch.bfloat16)
    rows[:, 0, 5] = -x
    slots = [16 * i for i in range(T)]
    _check(rows, rows * 0, slots, 1, 64, 16, T)
    assert need_scale(448.0) == 1.0 and need_scale(449.0) == 2.0 and need_scale(0.0) == 2.0 ** -64


def test_non_finite_values():
    """NaN and infinities become the NaN code and do not touch the scale."""
    block, heads, dim = 16, 2, 128
    g = torch.Generator().manual_seed(3)
    x = torch.randn(23, heads, dim, generator=g).to(torch.bfloat16)
    x[0, 0, 3], x[0, 1, 127], x[4, 0, 0], x[9, 1, 64] = math.nan, math.inf, -math.inf, math.inf
    x[22] = math.inf
    slots = _slots([(2, 0, 1), (3, 3, 13), (4, 0, 8), (1, 6, 1)], block)
    cache = _check(x, x.flip(0), slots, heads, dim, block, 5)
    assert torch.isnan(cache.k.float()).any()


def test_strided_rows_and_skipped_tokens():
    """The k and v columns of a fused projection, padding slots -1, slots outside the cache (flagged)."""
    block, heads, dim, blocks = 32, 2, 256, 6
    slots = _slots([(5, 4, 3)], block) + [-1] * 3 + _slots([(0, 0, 32), (1, 0, 2)], block) + [-1]
    T = len(slots)
    qkv = torch.randn(T, 12 * dim, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    d = qkv.cuda()
    _check(qkv[:, 8 * dim:10 * dim].view(T, 2, dim), qkv[:, 10 * dim:].view(T, 2, dim), slots, heads, dim, block, blocks,
           dev=(d[:, 8 * dim:10 * dim].view(T, 2, dim), d[:, 10 * dim:].view(T, 2, dim)))
    assert ops.device_status() == 0
    bad = list(slots)
    bad[0], bad[-1] = blocks * block, -2
    want = list(slots)
    want[0] = -1
    k, v, ks, vs = _fill(blocks, heads, block, dim, 0)
    cache = ops.KVCache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda())
    x = qkv[:, :2 * dim].reshape(T, 2, dim)
    ops.kv_append(x.cuda(), x.cuda(), cache, torch.tensor(bad, dtype=torch.int32).cuda())
    assert ops.device_status() & ops.DEVICE_KV_RANGE
    c, s = k.double().numpy().copy(), ks.double().numpy().copy()
    ref_append(x.double().numpy(), want, c, s, block)
    assert np.array_equal(cache.k.double().cpu().numpy(), c) and np.array_equal(cache.k_scale.double().cpu().numpy(), s)


def test_one_by_one_equals_a_fresh_block_up_to_the_scale():
    """Appending a block token by token ends with the scale of the whole block; the codes differ from the one-call
    write only where re-coding rounded a subnormal (half a step of the final scale's subnormals)."""
    block, heads, dim = 64, 2, 128
    g = torch.Generator().manual_seed(9)
    x = (torch.randn(block, heads, dim, generator=g) * torch.exp2(torch.arange(block).float() / 8)[:, None, None]).to(torch.bfloat16)
    once, steps = (ops.KVCache(*(t.cuda() for t in _fill(2, heads, block, dim, 1))) for _ in range(2))
    sl = torch.arange(block, dtype=torch.int32).cuda()
    ops.kv_append(x.cuda(), x.cuda(), once, sl)
    for i in range(block):
        ops.kv_append(x[i:i + 1].cuda(), x[i:i + 1].cuda(), steps, sl[i:i + 1])
    assert torch.equal(once.k_scale[0], steps.k_scale[0])
    a, b = once.k[0].float(), steps.k[0].float()
    assert float((a - b).abs().max()) <= 2.0 ** -9  # one subnormal step
    assert torch.equal(steps.k[1].view(torch.uint8).cpu(), _fill(2, heads, block, dim, 1)[0][1].view(torch.uint8))


def test_empty_call():
    cache = ops.KVCache.empty(2, 1, 16, 64)
    e = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    ops.kv_append(e, e, cache, torch.empty(0, dtype=torch.int32, device="cuda"))
