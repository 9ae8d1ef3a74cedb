"""Microscaled 4-bit matrices made and made again: row factors that a caller brings."""
import zlib

import pytest
import torch

import fp4_cases as fc
from skinny_gemm_gb300 import ops

pytestmark = pytest.mark.gpu


def gen(*seed):
    return torch.Generator().manual_seed(zlib.crc32(repr(seed).encode()))


@pytest.mark.parametrize("E,N,K", [(1, 1, 32), (1, 300, 320), (3, 130, 2304)])
def test_mx_rows_quantised_over_factors(E, N, K):
    """An mx matrix may have row factors; rows quantised into it have factors of 1, whatever was there."""
    x = fc.activations(gen(E, N, K), E * N, K).cuda()
    x = x if E == 1 else x.view(E, N, K)
    want = ops.fp4_quant(x, "mx")
    old = torch.rand(E * N, generator=gen(1)).cuda() * 100 - 3
    old[0] = float("nan")
    w = ops.FP4Matrix(torch.zeros_like(want.codes), torch.zeros_like(want.scales), old, N, K, E, "mx")
    assert ops.fp4_quant(x, "mx", out=w) is w
    assert torch.equal(ops.fp4_dequant(w), ops.fp4_dequant(want))
    rows = fc.activations(gen(2), 5, K).cuda()
    if E == 1:
        assert torch.equal(ops.fp4_mm(rows, w), ops.fp4_mm(rows, want))
        assert torch.equal(ops.fp4_mm(w, ops.fp4_quant(rows, "mx")), ops.fp4_mm(want, ops.fp4_quant(rows, "mx")))
    else:
        ids = torch.tensor([0, 1, 2, 1, 0], dtype=torch.int32, device="cuda")
        assert torch.equal(ops.fp4_mm_id(rows, w, ids), ops.fp4_mm_id(rows, want, ids))
    assert ops.device_status() == 0


def test_mx_scales_and_factors_at_their_ends():
    """Values of mx matrices whose scales and row factors are large, small or one of each: zeros stay zeros."""
    N, K = 40, 64
    codes = (torch.arange(N * K).view(N, K) % 16).numpy().astype("uint8")
    byte = torch.tensor([[254, 1], [250, 130], [0, 254], [3, 0], [127, 254]] * 8, dtype=torch.uint8).numpy()
    factor = torch.tensor([2.0 ** 20, 1.375 * 2.0 ** 100, 1.25 * 2.0 ** -90, 1.5 * 2.0 ** 126, 2.0 ** -126, 1.0, 0.75, -1.5] * 5).numpy()
    w = fc.matrix(ops, codes, byte, factor, 1, "mx")
    want = fc.values(codes, byte, None, "mx") * factor.astype("float64")[:, None]  # (exact: 2 + 4 significant bits)
    assert torch.equal(ops.fp4_dequant(w).double(), torch.from_numpy(want).to(torch.bfloat16).double().cuda())


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("E", [1, 3])
def test_one_factor_for_all_rows(fmt, E):
    """A checkpoint's one factor of a matrix: a number, a tensor of one on either side, or one each row."""
    g = gen(fmt, E)
    N, K, f = 70, 96, 0.375
    codes, byte, _, _ = fc.weights(g, E, N, K, fmt)
    lead = (N,) if E == 1 else (E, N)
    c, s = (torch.from_numpy(a).view(*lead, -1).cuda() for a in (fc.pack(codes), byte))
    want = torch.from_numpy(fc.values(codes, byte, None, fmt) * f).to(torch.bfloat16).cuda().view(*lead, K)
    for factor in (f, torch.tensor(f), torch.tensor([f], device="cuda"), torch.tensor(f, dtype=torch.float64, device="cuda"), torch.full(lead, f, device="cuda"), torch.full(lead, f)):
        w = ops.FP4Matrix.from_rows(c, s, factor, fmt)
        assert torch.equal(ops.fp4_dequant(w), want)
    assert torch.equal(ops.fp4_dequant(ops.FP4Matrix.from_rows(c, s, 2, fmt)).float(), want.float() / f * 2)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [1, 5, 16, 40, 64, 70, 300])
def test_gated_of_quantised_rows(fmt, act, M):
    """One quantisation for both a gated and a plain product: the bits of the calls that quantise themselves."""
    x = fc.activations(gen(3, M), M, 320).cuda()
    w = ops.FP4Matrix.gated(fc.activations(gen(4), 140, 320).cuda(), fc.activations(gen(5), 140, 320).cuda(), fmt)
    q = ops.fp4_quant(x, fmt)
    assert torch.equal(ops.fp4_gated(q, w, act), ops.fp4_gated(x, w, act)) and torch.equal(ops.fp4_mm(q, w), ops.fp4_mm(x, w))
    assert ops.device_status() == 0
