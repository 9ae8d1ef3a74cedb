"""The gated form where the gate is far below zero: act(g) is small, and not yet too small for the output's type."""
import numpy as np
import pytest
import torch

import fp4_cases as fc
from skinny_gemm_gb300 import ops

pytestmark = pytest.mark.gpu


def exact(gates, up, K):
    """x of one row, and W's rows (gate and up in turn): the products are the given gates, multiples of 1/8 of at most 96, and
    `up`, a power of two.  A block of W for each power of eight: code c and scale 8^i make c 8^i, two codes a digit of 0 to 7."""
    F = len(gates)
    codes, byte = np.zeros((2 * F, K), np.uint8), np.full((2 * F, K // 32), 127, np.uint8)
    x = torch.zeros(K)
    digits = {0: (0, 0), 1: (2, 0), 2: (4, 0), 3: (5, 0), 4: (6, 0), 5: (6, 2), 6: (7, 0), 7: (7, 2)}  # e2m1 codes that add up to it
    for block, power in enumerate((-1, 0, 1, 2)):  # 8^-1 .. 8^2
        byte[0::2, block] = 127 + 3 * power
        x[32 * block] = x[32 * block + 5] = 1.0  # (a block of ones and zeros is held exactly)
        for i, g in enumerate(gates):
            d = int(abs(g) * 8) // 8 ** block % 8
            codes[2 * i, [32 * block, 32 * block + 5]] = [c + (8 if g < 0 and c else 0) for c in digits[d]]
    codes[1::2, 0] = 2
    byte[1::2, 0] = 127 + int(np.log2(up))
    return x.to(torch.bfloat16), codes, byte


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [1, 5, 40, 100])
@pytest.mark.parametrize("power", [0, 40, 100])
def test_gates_far_below_zero(act, M, power):
    g = np.concatenate([np.arange(-96, -80, 0.125), np.arange(-80, 96, 1.0), [-0.125, 0.125]])
    if act == "gelu":  # (its exponent is a cubic: the same range of values)
        g = np.concatenate([np.arange(-12, -7, 0.125), np.arange(-96, 96, 3.0), np.arange(-7, 7, 0.25)])
    K = 128
    x, codes, byte = exact(g, 2.0 ** power, K)
    w, wv = fc.matrix(ops, codes, byte, None, 1, "mx"), fc.values(codes, byte, None, "mx")
    xv = x.double().numpy()[None]
    assert np.array_equal((xv @ wv[0::2].T)[0], g) and (wv[1::2] @ xv[0] == 2.0 ** power).all()
    t = g if act == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    want = g / (1 + np.exp(np.minimum(-t, 700.0))) * 2.0 ** power
    # gate and up are exact.  t: two constants and four operations of gelu's, 2^-24 each relative to it (silu has none), and its
    # product with log2(e) for 2^x, two more: act(g) is off by 8 |t| 2^-24 relative to itself; the kernel takes 24 from that
    # product, 2^-20 for its rounding where it is below 32; 2 ulp each of 2^x and the division and four products, 8 of 2^-23.
    # What leaves fp32's normal range is off by its steps, 2^-149: of 2^x or the reciprocal by four, times |g|, of act by two.  The
    # output: half a step of bf16, and of its subnormals.
    rel = 8 * np.abs(t) * 2.0 ** -24 + 2.0 ** -20 + 8 * 2.0 ** -23
    small = (np.abs(g) * 2.0 ** -147 + 2.0 ** -148) * 2.0 ** power
    bound = np.abs(want) * (rel + 2.0 ** -8 * (1 + rel)) + small * (1 + 2.0 ** -8) + 2.0 ** -133
    y = ops.fp4_gated(x.expand(M, K).contiguous().cuda(), w, act)
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= bound).all(), (g[(err > bound).any(0)], (err / bound).max())
    assert ops.device_status() == 0
