"""How the work is cut must not show: row tiles of every size, groups divided between CTAs, rows of one, several and
many groups, in a batch and alone."""
import pytest
import torch

from kv_cases import Step, assert_close
from skinny_gemm_gb300 import ops

pytestmark = pytest.mark.gpu


def _alone(step, b, cache, window):
    """Request b's rows from a call of its own."""
    lo, hi = int(step.cu[b]), int(step.cu[b + 1])
    table = torch.from_numpy(step.table[b:b + 1]).cuda()
    cu = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
    lens = torch.tensor([step.lens[b]], dtype=torch.int32, device="cuda")
    return ops.kv_attention(step.q[lo:hi].cuda(), cache, table, cu, lens, hi - lo, step.lens[b], window=window)


# query rows of a key head: 1, 2, 4, 7, 8, 12, 16, 20, 24, 28, 32 and several tiles of them
@pytest.mark.parametrize("hq,hkv,dim,M", [
    (2, 2, 256, 1), (4, 2, 256, 1), (8, 2, 256, 1), (8, 2, 256, 2), (8, 2, 256, 3), (8, 2, 256, 4), (8, 2, 256, 5),
    (8, 2, 256, 8), (8, 2, 256, 11), (14, 2, 128, 1), (4, 2, 128, 4), (24, 2, 128, 1), (8, 1, 128, 2), (8, 1, 128, 3),
    (14, 2, 128, 4), (8, 1, 128, 7), (8, 2, 64, 1), (4, 1, 64, 3), (16, 1, 64, 1), (8, 1, 64, 3), (16, 1, 64, 5)])
@pytest.mark.parametrize("window", [0, 1500])
def test_a_batch_and_its_requests_alone(hq, hkv, dim, M, window):
    cached = [3000, 0, 9000 + dim, 127, 1023, 5, 1021]
    step = Step(hq, hkv, dim, 64, cached, [M] * len(cached), seed=hq + M)
    cache = step.cache()
    out = step.run(cache=cache, window=window)
    for b in range(len(cached)):
        assert torch.equal(_alone(step, b, cache, window), out[step.cu[b]:step.cu[b + 1]]), b
    ref, bound = step.reference(window=window)
    assert_close(out, ref, bound, f"{hq} {hkv} {dim} {M} {window}")
    assert ops.device_status() == 0


def test_more_requests_than_lanes():
    """The range of a CTA begins in any of 70 (and 1100) requests, empty ones among them."""
    for B, n in ((70, 400), (1100, 40)):
        cached = [(37 * b * b) % n if b % 5 else 0 for b in range(B)]
        new = [0 if b % 7 == 3 else 1 + b % 2 for b in range(B)]
        step = Step(4, 2, 64, 16, cached, new, seed=B)
        cache = step.cache()
        out = step.run(cache=cache)
        for b in (0, 31, 32, 33, 64, B - 2, B - 1):
            if new[b]:
                assert torch.equal(_alone(step, b, cache, 0), out[step.cu[b]:step.cu[b + 1]]), b
        ref, bound = step.reference()
        assert_close(out, ref, bound, str(B))


@pytest.mark.parametrize("heads,dim,block", [(9, 64, 16), (20, 128, 16), (12, 128, 32), (33, 64, 64), (5, 256, 16)])
@pytest.mark.parametrize("T", [70, 2300])
def test_append_heads_in_several_ctas(heads, dim, block, T):
    """More heads than a CTA takes, few tokens and many; runs that begin inside blocks and cross CTAs."""
    import test_gpu_kv_append as A

    runs, at = [], 0
    for i in range(10 ** 6):
        n = min(1 + (7 * i * i) % (2 * block), block, T - at)
        runs.append((i, (3 * i) % (block - n + 1), n))
        at += n
        if at == T:
            break
    slots = [b * block + o + k for b, o, n in runs for k in range(n)]
    g = torch.Generator().manual_seed(T + heads)
    k, v = ((torch.randn(T, heads, dim, generator=g) * torch.rand(T, heads, 1, generator=g) * 4).to(torch.bfloat16) for _ in "kv")
    A._check(k, v, slots, heads, dim, block, len(runs), seed=heads)
