"""w4a16_kv_plan against a plain loop: tables, slots, positions, the free list; edges and out-of-range inputs."""
import numpy as np
import pytest
import torch

from kv_cases import make_lengths, ref_plan
from skinny_gemm_gb300 import ops

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.tensor(a, dtype=torch.int32).cuda()


def _case(B, T_max, new_max, block, seed, max_blocks=None, free_short=0):
    r = np.random.RandomState(seed)
    cached, new = make_lengths(B, T_max, new_max, seed, block)
    need = sum(-(-(c + n) // block) - -(-c // block) for c, n in zip(cached, new))
    width = max_blocks or max(-(-(c + n) // block) for c, n in zip(cached, new)) + 2
    ids = r.permutation(100000)
    table = np.full((B, width), -7, np.int64)
    for b in range(B):
        have = min(-(-cached[b] // block), width)
        table[b, :have] = ids[1000 * 0 + b * 37:b * 37 + have] if have <= 37 else r.randint(0, 90000, have)
    free = ids[-(need + 4 - free_short):]
    return cached, new, table.tolist(), free.tolist()


def _check(cached, new, table, free, head, T, block):
    t, f = _i32(table), _i32(free)
    p = ops.kv_plan(_i32(cached), _i32(new), t, f, T, block, head=None if head is None else _i32([head]))
    want = ref_plan(cached, new, table, free, head or 0, T, block)
    got = (t.tolist(), p.cu.tolist(), p.lens.tolist(), p.slots.tolist(), p.positions.tolist(), p.head.tolist()[0])
    for name, g, w in zip(("table", "cu", "lens", "slots", "positions", "head"), got, want):
        assert g == w, name


@pytest.mark.parametrize("B,T_max,new_max,block", [
    (1, 0, 1, 16), (1, 1000, 1, 64), (3, 300, 5, 16), (33, 2000, 8, 32), (257, 1500, 3, 128),
    (1500, 300, 4, 16), (2100, 100, 1, 64), (5, 1200, 3000, 16), (40, 100, 700, 64)])
def test_matches_the_loop(B, T_max, new_max, block):
    cached, new, table, free = _case(B, T_max, new_max, block, B + block)
    for head in (None, 3):
        _check(cached, new, table, free, head, sum(new), block)
    assert ops.device_status() == 0


def test_padded_batches():
    """Rows past the last token get slot and position -1."""
    cached, new, table, free = _case(9, 400, 4, 16, 5)
    _check(cached, new, table, free, 1, sum(new) + 41, 16)
    _check([0] * 3, [0] * 3, [[-1]] * 3, [5], None, 10, 16)  # nothing at all joins
    assert ops.device_status() == 0


def test_no_requests():
    p = ops.kv_plan(_i32([]), _i32([]), torch.empty(0, 4, dtype=torch.int32, device="cuda"), _i32([1, 2]), 5, 16)
    assert p.cu.tolist() == [0] and p.slots.tolist() == [-1] * 5 and p.head.tolist() == [0]


def test_free_list_runs_out():
    cached, new, table, free = _case(20, 300, 60, 16, 8, free_short=11)
    _check(cached, new, table, free, 0, sum(new), 16)
    assert ops.device_status() & ops.DEVICE_KV_RANGE


def test_table_too_narrow():
    cached, new = [10, 40, 0], [100, 3, 1]
    table = [[4, -1], [5, 6], [-1, -1]]
    t = _i32(table)
    p = ops.kv_plan(_i32(cached), _i32(new), t, _i32(list(range(50, 70))), 104, 16)
    assert ops.device_status() & ops.DEVICE_KV_RANGE
    want = ref_plan([10], [100], [table[0]], list(range(50, 70)), 0, 100, 16)
    assert t.tolist()[0] == want[0][0] and p.slots.tolist()[:100] == want[3]
    assert p.slots.tolist()[100:] == [-1, -1, -1, 51 * 16]  # request 1 stands past its two blocks
    assert p.positions.tolist()[100:] == [40, 41, 42, 0] and p.head.tolist() == [2]


def test_bad_lengths_stay_inside():
    """Negative lengths count as 0, tokens past T are dropped, the flag is raised."""
    t = _i32([[1, -1], [-1, -1], [-1, -1]])
    p = ops.kv_plan(_i32([16, -5, 2147483647]), _i32([3, 2, -1]), t, _i32([7, 8, 9]), 4, 16)
    assert ops.device_status() & ops.DEVICE_KV_RANGE
    assert p.cu.tolist() == [0, 3, 4, 4]
    assert p.slots.tolist() == [7 * 16, 7 * 16 + 1, 7 * 16 + 2, 8 * 16] and p.positions.tolist() == [16, 17, 18, 0]
    assert p.lens.tolist()[:2] == [19, 1] and p.head.tolist() == [2]
    ops.kv_plan(_i32([0]), _i32([2]), _i32([[-1, -1]]), _i32([3]), 2, 16)
    assert ops.device_status() == 0


def test_a_missing_block_of_an_earlier_step_gives_no_slot():
    t = _i32([[3, -1, -1]])
    p = ops.kv_plan(_i32([20]), _i32([14]), t, _i32([8]), 14, 16)  # tokens 16..19 have no block
    assert p.slots.tolist() == [-1] * 12 + [8 * 16, 8 * 16 + 1]
    assert ops.device_status() & ops.DEVICE_KV_RANGE


def test_steps_chain_through_the_head_in_a_graph():
    """Three decode steps captured once: each plan takes its blocks after the last one's, without the host."""
    B, block = 6, 16
    cached, one = _i32([14, 15, 16, 0, 31, 47]), _i32([1] * B)
    table = torch.full((B, 8), -1, dtype=torch.int32)
    for b, c in enumerate([14, 15, 16, 0, 31, 47]):
        for j in range(-(-c // block)):
            table[b, j] = 100 + 10 * b + j
    free, start = _i32(list(range(40))), table.clone()
    table = table.cuda()
    plans = [ops.KVPlan.empty(B, B) for _ in range(3)]
    ops.kv_plan(cached, one, table, free, B, block, out=plans[0])
    table.copy_(start)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        have, head = cached, None
        for p in plans:
            ops.kv_plan(have, one, table, free, B, block, head=head, out=p)
            have, head = p.lens, p.head
    g.replay()
    c, h, t = [14, 15, 16, 0, 31, 47], 0, start.tolist()
    for p in plans:
        t, _, c, slots, pos, h = ref_plan(c, [1] * B, t, list(range(40)), h, B, block)
        assert p.slots.tolist() == slots and p.positions.tolist() == pos and p.head.tolist() == [h]
    assert table.tolist() == t
