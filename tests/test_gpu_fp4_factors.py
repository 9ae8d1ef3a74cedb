"""Row factors from one end of their range to the other: a product is what its definition says wherever that fits the output's type."""
import zlib

import numpy as np
import pytest
import torch

import fp4_cases as fc
from skinny_gemm_gb300 import ops

pytestmark = pytest.mark.gpu

# rows quantised in the product (one CTA a tile, a cluster), 17 to 64 rows, pairs, pairs that share a tile, several tiles a pair
SIZES = [(3, 200, 320), (1, 64, 4096), (40, 130, 2304), (17, 20000, 64), (64, 70, 96), (70, 140, 320), (130, 200, 8192), (300, 520, 320)]


def gen(*seed):
    return torch.Generator().manual_seed(zlib.crc32(repr(seed).encode()))


def check(y, want, bound):
    got = y.double().cpu().numpy().reshape(want.shape)
    assert np.isfinite(got).all(), f"{(~np.isfinite(got)).sum()} not finite"
    err = np.abs(got - want)
    assert (err <= bound).all(), f"{(err / bound).max()} of the bound"


def sparse(M, N, K, factor, top):
    """Rows of x with 2^top and, in a block that W does not leave out, 2^(top - 17): the sums are far below the factors' product,
    or zero.  W has its factors around `factor`, in the first of its nv blocks that are not x's peak's."""
    x = torch.zeros(M, K)
    x[:, 0] = 2.0 ** top
    x[:, 24] = 2.0 ** (top - 17) * (1 + torch.arange(M) % 3)
    codes, byte = np.zeros((N, K), np.uint8), np.full((N, K // 16), 1, np.uint8)  # (scales of 2^-9)
    codes[:, 24] = np.arange(N) % 4  # 0, 0.5, 1, 1.5
    return x.to(torch.bfloat16), codes, byte, (factor * (1 + np.arange(N) % 7 / 8)).astype(np.float32)


def dense(M, N, K, factor, shift):
    g = gen(M, N, K)
    codes, byte, _, _ = fc.weights(g, 1, N, K, "nv")
    x = fc.activations(g, M, K).float().clamp(-30, 30) * 2.0 ** shift
    return x.to(torch.bfloat16), codes, byte, (factor * (1 + torch.rand(N, generator=g).numpy())).astype(np.float32)


# (the factors of x are 2^11 to 2^12 below its rows' peaks)
CASES = {"both large": (sparse, 2.0 ** 66, 75), "large, small sums": (sparse, 2.0 ** 100, 40), "W's smallest, x large": (sparse, 2.0 ** -126, 111),
         "both small": (dense, 2.0 ** -60, -74), "W's smallest, x small": (dense, 2.0 ** -126, 7), "W large, x smallest": (dense, 2.0 ** 108, -122),
         "ordinary": (dense, 2.0 ** -9, 0)}


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("which", sorted(CASES))
def test_products(which, M, N, K):
    make, factor, power = CASES[which]
    x, codes, byte, f = make(M, N, K, factor, power)
    w, wv = fc.matrix(ops, codes, byte, f, 1, "nv"), fc.values(codes, byte, f, "nv")
    xv = fc.values(*fc.quant(x, "nv"), "nv")
    want = xv @ wv.T
    assert np.abs(want).max() < 2.0 ** 127 and np.abs(want).max() > 2.0 ** -126
    x = x.cuda()
    y = ops.fp4_mm(x, w)
    check(y, want, fc.product_bound(want, xv, wv))
    assert torch.equal(y, ops.fp4_mm(ops.fp4_quant(x), w))
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    check(ops.fp4_mm_id(x, w, ids), want, fc.product_bound(want, xv, wv))
    if N % 2 == 0 and abs(np.log2(np.abs(want).max())) < 60:  # (the product of two of them is there too)
        gate, up = want[:, 0::2], want[:, 1::2]
        check(ops.fp4_gated(x, w, "silu"), fc.act64(gate, "silu") * up, fc.gated_bound(gate, up, xv, wv[0::2], wv[1::2], "silu"))
    assert ops.device_status() == 0


@pytest.mark.parametrize("M,N,K", SIZES)
def test_factors_that_are_not_powers_of_two(M, N, K):
    """Rows of x from elsewhere, whose factors are any numbers: zero, one that is subnormal, and large ones beside small ones."""
    g = gen(M, N, K)
    xc, xb, _, _ = fc.weights(g, 1, M, K, "nv")
    wc, wb, _, _ = fc.weights(g, 1, N, K, "nv")
    fx = (torch.rand(M, generator=g).numpy() + 0.5) * 2.0 ** (np.arange(M) % 5 * 55 - 100.0)  # 2^-100 to 2^120
    fw = (torch.rand(N, generator=g).numpy() + 0.5) * 2.0 ** -60
    fx[0], fw[N // 2] = 0.0, 1.25 * 2.0 ** -133
    fx, fw = fx.astype(np.float32), fw.astype(np.float32)
    xv, wv = fc.values(xc, xb, fx, "nv"), fc.values(wc, wb, fw, "nv")
    y = ops.fp4_mm(fc.matrix(ops, xc, xb, fx, 1, "nv"), fc.matrix(ops, wc, wb, fw, 1, "nv"))
    want = xv @ wv.T
    check(y, want, fc.product_bound(want, xv, wv))
    assert not y[0].any() and ops.device_status() == 0
