"""Microscaled 4-bit matrices on the GPU: quantisation bit for bit, products, gated and routed forms against float64."""
import zlib

import numpy as np
import pytest
import torch

import fp4_cases as fc

pytestmark = pytest.mark.gpu


def gen(*seed):
    return torch.Generator().manual_seed(zlib.crc32(repr(seed).encode()))


def check_quant(ops, x, fmt, q):
    codes, byte, factor = fc.quant(x.cpu(), fmt)
    got = q.codes.cpu().numpy().reshape(codes.shape[0], -1)
    at = fc.tile_index(*byte.shape)
    assert np.array_equal(q.scales.cpu().numpy()[at], byte)
    got = np.stack([got & 15, got >> 4], -1).reshape(codes.shape)
    assert np.array_equal(np.where(got == 8, 0, got), np.where(codes == 8, 0, codes))  # (either zero)
    # blocks past K, up to the atoms' end
    nb = byte.shape[1]
    pad = -(-nb // 4) * 4
    assert not q.scales.cpu().numpy()[fc.tile_index(byte.shape[0], pad)[:, nb:]].any()
    if fmt == "nv":
        assert np.array_equal(q.row_scale.cpu().numpy().astype(np.float64), factor)
    y = ops.fp4_dequant(q).cpu().double().numpy().reshape(codes.shape)
    want = fc.values(codes, byte, factor, fmt)
    assert np.array_equal(y, torch.from_numpy(want).to(torch.bfloat16).double().numpy(), equal_nan=True)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,K", [(1, 32), (1, 2560), (3, 96), (7, 2304), (33, 160), (129, 64), (300, 1568), (2, 16384), (5, 40000)])
def test_quant(fmt, M, K):
    from skinny_gemm_gb300 import ops

    x = fc.activations(gen(fmt, M, K), M, K).cuda()
    check_quant(ops, x, fmt, ops.fp4_quant(x, fmt))


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_quant_edges(fmt):
    """Zeros of both signs, ties of codes and scales, the largest and smallest values, one huge beside tiny ones, NaN and infinities."""
    from skinny_gemm_gb300 import ops

    big = torch.finfo(torch.bfloat16).max
    rows = [torch.zeros(64), -torch.zeros(64), torch.full((64,), big), torch.full((64,), -2.0 ** -133),
            torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 8), -torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0] * 8),
            torch.arange(64) * 2.0 ** -130, torch.tensor([2.0 ** 100] + [1.0] * 63), torch.tensor([1.0] * 32 + [2.0 ** -20] * 32),
            torch.tensor([float("inf")] + [1.0] * 63), torch.tensor([1.0] * 40 + [float("nan")] + [2.0] * 23),
            torch.full((64,), float("-inf")), torch.tensor([float("nan")] * 16 + [2688.0] + [1.0] * 47),
            torch.tensor([2688.0 * 2.0 ** 5] + [1.0] * 63), torch.tensor([2704.0] + [3.0] * 63), torch.tensor([7.5] * 32 + [7.0, -7.96875] * 16)]
    rows += [torch.full((64,), (128 + i) * 2.0 ** -3) for i in range(0, 128, 3)]
    x = torch.stack([r.float() for r in rows]).to(torch.bfloat16).cuda()
    check_quant(ops, x, fmt, ops.fp4_quant(x, fmt))


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_quant_strided_and_experts(fmt):
    from skinny_gemm_gb300 import ops

    wide = fc.activations(gen(1), 9, 704).cuda()
    x = wide[:, 128:128 + 320]
    check_quant(ops, x, fmt, ops.fp4_quant(x, fmt))
    w = fc.activations(gen(2), 3 * 130, 96).view(3, 130, 96).cuda()
    q = ops.fp4_quant(w, fmt)
    assert (q.E, q.N) == (3, 130)
    n = ops.fp4_scale_bytes(130, 96, fmt)
    for e in range(3):
        one = ops.FP4Matrix(q.codes.view(3, 130, -1)[e], q.scales[e * n:(e + 1) * n],
                            None if q.row_scale is None else q.row_scale[e * 130:(e + 1) * 130], 130, 96, 1, fmt)
        check_quant(ops, w[e], fmt, one)
    assert torch.equal(ops.fp4_dequant(q).view(3, 130, 96)[1], ops.fp4_dequant(ops.fp4_quant(w[1].contiguous(), fmt)))


def product(ops, fmt, M, N, K, act=None, seed=0):
    g = gen(fmt, M, N, K, act, seed)
    codes, byte, factor, wv = fc.weights(g, 1, N, K, fmt)
    w = fc.matrix(ops, codes, byte, factor, 1, fmt)
    x = fc.activations(g, M, K)
    return x.cuda(), w, fc.values(*fc.quant(x, fmt), fmt), wv


def check(y, want, bound):
    err = np.abs(y.double().cpu().numpy().reshape(want.shape) - want)
    assert np.isfinite(err).all() and (err <= bound).all(), f"{(err / bound).max()} of the bound"


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,N,K", [(1, 128, 256), (1, 1, 32), (2, 127, 64), (5, 129, 96), (15, 300, 288), (16, 128, 1024),
                                   (17, 256, 320), (33, 100, 1568), (64, 257, 512), (65, 130, 2304), (127, 64, 160),
                                   (129, 300, 800), (300, 515, 544), (1, 2050, 5120), (9, 20000, 64)])
def test_mm(fmt, M, N, K):
    from skinny_gemm_gb300 import ops

    x, w, xv, wv = product(ops, fmt, M, N, K)
    y = ops.fp4_mm(x, w)
    assert y.shape == (M, N) and ops.device_status() == 0
    want = xv @ wv.T
    check(y, want, fc.product_bound(want, xv, wv))
    assert torch.equal(y, ops.fp4_mm(ops.fp4_quant(x, fmt), w))


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,F,K", [(1, 64, 256), (3, 1, 32), (20, 65, 288), (70, 200, 96), (200, 333, 320)])
def test_gated(fmt, act, M, F, K):
    from skinny_gemm_gb300 import ops

    x, w, xv, wv = product(ops, fmt, M, 2 * F, K, act)
    y = ops.fp4_gated(x, w, act)
    assert y.shape == (M, F) and ops.device_status() == 0
    gate, up = xv @ wv[0::2].T, xv @ wv[1::2].T
    check(y, fc.act64(gate, act) * up, fc.gated_bound(gate, up, xv, wv[0::2], wv[1::2], act))


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("T,top,E,N,K,act", [(1, 1, 2, 128, 256, None), (8, 1, 8, 200, 320, None), (5, 3, 4, 129, 96, "silu"),
                                             (100, 2, 3, 64, 160, None), (300, 4, 40, 130, 288, "gelu"), (700, 1, 2, 100, 64, None)])
def test_mm_id(fmt, T, top, E, N, K, act):
    from skinny_gemm_gb300 import ops

    if act:
        N += N % 2
    g = gen(fmt, T, top, E, N, K)
    codes, byte, factor, wv = fc.weights(g, E, N, K, fmt)
    w = fc.matrix(ops, codes, byte, factor, E, fmt)
    x = fc.activations(g, T, K)
    ids = torch.randint(0, E, (T, top), generator=g, dtype=torch.int32)
    ids[: T // 2] = ids[0, 0]  # one expert has most of the rows, and a row may choose it twice
    y = ops.fp4_mm_id(x.cuda(), w, ids.cuda(), act=act)
    assert ops.device_status() == 0
    xv, wv = fc.values(*fc.quant(x, fmt), fmt), wv.reshape(E, N, K)
    for e in range(E):
        t, j = np.nonzero(ids.numpy() == e)
        if not len(t):
            continue
        got = y[torch.from_numpy(t), torch.from_numpy(j)]
        if act is None:
            want = xv[t] @ wv[e].T
            check(got, want, fc.product_bound(want, xv[t], wv[e]))
        else:
            gate, up = xv[t] @ wv[e, 0::2].T, xv[t] @ wv[e, 1::2].T
            check(got, fc.act64(gate, act) * up, fc.gated_bound(gate, up, xv[t], wv[e, 0::2], wv[e, 1::2], act))


def test_mm_id_bad_ids():
    """An id outside the experts: a row of zeros and the flag; the other rows as without it."""
    from skinny_gemm_gb300 import ops

    g = gen(3)
    codes, byte, factor, wv = fc.weights(g, 4, 96, 64, "nv")
    w = fc.matrix(ops, codes, byte, factor, 4, "nv")
    x = fc.activations(g, 6, 64).cuda()
    ids = torch.tensor([[0, 1], [-1, 2], [3, 4], [2, 2], [1 << 30, -5], [3, 0]], dtype=torch.int32).cuda()
    good = torch.where((ids >= 0) & (ids < 4), ids, 0)
    want = ops.fp4_mm_id(x, w, good)
    assert ops.device_status() == 0
    out = torch.full((6, 2, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    y = ops.fp4_mm_id(x, w, ids, out=out)
    assert ops.device_status() == ops.DEVICE_BAD_ID
    bad = ((ids < 0) | (ids >= 4))[..., None]
    assert torch.equal(y, torch.where(bad, torch.zeros_like(want), want))


def test_not_finite():
    """A block with a NaN or an infinity makes its row of the product NaN, and no other."""
    from skinny_gemm_gb300 import ops

    for fmt in ("nv", "mx"):
        x, w, _, _ = product(ops, fmt, 20, 130, 320)
        want = ops.fp4_mm(x, w)
        x2 = x.clone()
        x2[3, 17], x2[11, 300] = float("inf"), float("nan")
        y = ops.fp4_mm(x2, w)
        hit = torch.zeros(20, dtype=torch.bool, device="cuda")
        hit[[3, 11]] = True
        assert y[hit].isnan().all() and torch.equal(y[~hit], want[~hit])


def test_empty_and_out():
    from skinny_gemm_gb300 import ops

    x, w, _, _ = product(ops, "nv", 4, 100, 64)
    assert ops.fp4_mm(x[:0], w).shape == (0, 100)
    assert ops.fp4_mm_id(x[:0], w, torch.empty(0, 2, dtype=torch.int32, device="cuda")).shape == (0, 2, 100)
    assert ops.fp4_dequant(ops.fp4_quant(x[:0])).shape == (0, 64)
    guard = torch.full((6, 100), 3.0, dtype=torch.bfloat16, device="cuda")
    ops.fp4_mm(x, w, out=guard[1:5])
    assert (guard[0] == 3).all() and (guard[5] == 3).all() and torch.equal(guard[1:5], ops.fp4_mm(x, w))
    x3 = x.view(2, 2, 64)
    assert torch.equal(ops.fp4_mm(x3, w).view(4, 100), guard[1:5])


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,N,K", [(256, 256, 256), (256, 256, 512), (130, 100, 96), (257, 520, 2304), (1000, 1300, 320), (2100, 2570, 64), (600, 4104, 2816)])
def test_mm_many_rows(fmt, M, N, K):
    """The pair kernel: one tile, ragged edges of both sides, several tiles a pair."""
    from skinny_gemm_gb300 import ops

    x, w, xv, wv = product(ops, fmt, M, N, K)
    y = ops.fp4_mm(x, w)
    assert ops.device_status() == 0
    want = xv @ wv.T
    check(y, want, fc.product_bound(want, xv, wv))


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,N,K", [(70, 64, 2048), (130, 200, 8192), (300, 1111, 2080), (129, 2570, 4128), (300, 2500, 9024), (500, 1281, 10272)])
def test_mm_split_over_pairs(fmt, M, N, K):
    """Few tiles and a long K: two and four pairs share a tile, whole and ragged ones."""
    from skinny_gemm_gb300 import ops

    x, w, xv, wv = product(ops, fmt, M, N, K)
    y = ops.fp4_mm(x, w)
    assert ops.device_status() == 0
    want = xv @ wv.T
    check(y, want, fc.product_bound(want, xv, wv))
    for _ in range(5):
        assert torch.equal(ops.fp4_mm(x, w), y)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("T,top,E,N,K", [(100, 1, 2, 300, 4096), (90, 2, 3, 514, 2336), (60, 1, 1, 1000, 8192)])
def test_mm_id_split_over_pairs(fmt, T, top, E, N, K):
    from skinny_gemm_gb300 import ops

    g = gen(fmt, T, top, E, N, K)
    codes, byte, factor, wv = fc.weights(g, E, N, K, fmt)
    w = fc.matrix(ops, codes, byte, factor, E, fmt)
    x = fc.activations(g, T, K)
    ids = torch.randint(0, E, (T, top), generator=g, dtype=torch.int32)
    y, z = ops.fp4_mm_id(x.cuda(), w, ids.cuda()), ops.fp4_mm_id(x.cuda(), w, ids.cuda(), act="gelu")
    assert ops.device_status() == 0
    xv, wv = fc.values(*fc.quant(x, fmt), fmt), wv.reshape(E, N, K)
    for e in range(E):
        t, j = np.nonzero(ids.numpy() == e)
        at = torch.from_numpy(t), torch.from_numpy(j)
        want = xv[t] @ wv[e].T
        check(y[at], want, fc.product_bound(want, xv[t], wv[e]))
        gate, up = want[:, 0::2], want[:, 1::2]
        check(z[at], fc.act64(gate, "gelu") * up, fc.gated_bound(gate, up, xv[t], wv[e, 0::2], wv[e, 1::2], "gelu"))


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_many_rows(fmt, act):
    from skinny_gemm_gb300 import ops

    for M, F, K in ((300, 200, 288), (700, 1111, 96), (150, 333, 4096), (260, 1200, 5152)):
        x, w, xv, wv = product(ops, fmt, M, 2 * F, K, act)
        y = ops.fp4_gated(x, w, act)
        assert ops.device_status() == 0
        gate, up = xv @ wv[0::2].T, xv @ wv[1::2].T
        check(y, fc.act64(gate, act) * up, fc.gated_bound(gate, up, xv, wv[0::2], wv[1::2], act))


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("N,K", [(300, 2560), (2560, 1024), (10240, 512), (40000, 96), (100, 256)])
def test_rows_do_not_depend_on_the_batch(fmt, N, K):
    """Up to 64 rows a row's result is the one-row call's, bit for bit."""
    from skinny_gemm_gb300 import ops

    x, w, _, _ = product(ops, fmt, 64, N, K)
    one = torch.cat([ops.fp4_mm(x[i:i + 1], w) for i in (0, 3, 15, 31, 50, 63)])
    for M in (4, 5, 16, 17, 32, 33, 55, 64):
        y = ops.fp4_mm(x[:M], w)
        for j, i in enumerate((0, 3, 15, 31, 50, 63)):
            if i < M:
                assert torch.equal(y[i], one[j]), (M, i)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,N,K", [(1, 200, 16384), (1, 3000, 4640), (2, 129, 4064), (3, 40, 2688), (5, 77, 10240), (7, 300, 1120), (16, 140, 512), (16, 5000, 320), (12, 60, 32)])
def test_rows_quantised_in_the_product(fmt, M, N, K):
    """Few rows, which the product may quantise itself: the same bits as from fp4_quant, NaN and infinities among the values."""
    from skinny_gemm_gb300 import ops

    x, w, xv, wv = product(ops, fmt, M, N, K)
    y = ops.fp4_mm(x, w)
    want = xv @ wv.T
    check(y, want, fc.product_bound(want, xv, wv))
    x[M // 2, K - 3] = float("nan")
    x[0, 1] = float("-inf")
    wide = torch.zeros(M, K + 64, dtype=torch.bfloat16, device="cuda")
    wide[:, 32:32 + K] = x
    y, z = ops.fp4_mm(wide[:, 32:32 + K], w), ops.fp4_mm(ops.fp4_quant(x, fmt), w)
    assert y[0].isnan().all() and y[M // 2].isnan().all()
    assert torch.equal(y.view(torch.int16), z.view(torch.int16)) or torch.equal(y.nan_to_num(7.0), z.nan_to_num(7.0))
    assert ops.device_status() == 0
