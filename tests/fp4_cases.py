"""Plain 64-bit forms of the microscaled 4-bit operators, on the CPU, from their definitions.

Codes, scales and factors are computed element by element: the nearest of the eight magnitudes by distance, ties to the
even code; scales by search over the scale type's own values.  Products are float64 matrix products of the values.
"""
import functools
import math

import numpy as np
import torch

MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
BLOCK = {"nv": 16, "mx": 32}


@functools.lru_cache(maxsize=None)
def e4m3_values():
    b = np.arange(127, dtype=np.uint8)  # 0 .. 0x7E: the finite values that are not negative
    return torch.from_numpy(b.copy()).view(torch.float8_e4m3fn).double().numpy()


def nearest(y, table):
    """Index into an increasing table of the nearest value, ties to the even index, beyond the last the last."""
    hi = np.clip(np.searchsorted(table, y), 0, len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = np.abs(table[hi] - y), np.abs(y - table[lo])
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def quant(x, fmt):
    """(codes [M, K], scale bytes [M, K / block], factors [M] or None) of bf16 rows."""
    M, K = x.shape
    b = x.double().numpy().reshape(M, K // BLOCK[fmt], BLOCK[fmt])
    bad = ~np.isfinite(b).all(-1)
    peak = np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1)
    with np.errstate(divide="ignore"):
        if fmt == "mx":
            e = np.where(peak > 0, np.frexp(peak)[1] - 1 - 2, -127)
            byte = np.clip(e, -127, 127) + 127
            unit, factor, nan = np.ldexp(1.0, byte - 127), None, 255
        else:
            top = np.abs(np.where(np.isfinite(b), b, 0.0)).max((1, 2))
            m, e = np.frexp(top / 2688)
            e = np.where(top > 0, np.where(m == 0.5, e - 1, e), -126)
            factor = np.ldexp(1.0, np.maximum(e, -126))
            byte = nearest(peak / factor[:, None] / 6, e4m3_values())
            unit, nan = e4m3_values()[byte] * factor[:, None], 127
    y = np.where(np.isfinite(b), b, 0.0) / np.where(unit == 0, 1.0, unit)[..., None]
    c = nearest(np.abs(y), MAGNITUDES) + 8 * np.signbit(b)
    c = np.where((unit == 0)[..., None] | bad[..., None], 0, c)
    return c.reshape(M, K).astype(np.uint8), np.where(bad, nan, byte).astype(np.uint8), factor


def values(codes, byte, factor, fmt):
    """float64 values of codes and scale bytes in row order."""
    v = np.where(codes > 7, -1.0, 1.0) * MAGNITUDES[codes % 8]
    if fmt == "mx":
        s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    else:
        s = torch.from_numpy(byte.copy()).view(torch.float8_e4m3fn).double().numpy()
        if factor is not None:
            s = s * np.asarray(factor, np.float64)[:, None]
    return v * np.repeat(s, BLOCK[fmt], 1)


def pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def tile_index(N, nb):
    """Where scale byte (row, block) lies."""
    r, k = np.meshgrid(np.arange(N), np.arange(nb), indexing="ij")
    return (r // 128 * math.ceil(nb / 4) + k // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + k % 4


def weights(g, E, N, K, fmt, spread=1.0):
    """Random codes, scale bytes and factors of E experts, and their values: every code, scales over some octaves."""
    codes = torch.randint(0, 16, (E * N, K), generator=g).numpy().astype(np.uint8)
    nb = K // BLOCK[fmt]
    if fmt == "mx":
        byte = torch.randint(118, 130, (E * N, nb), generator=g).numpy().astype(np.uint8)
        factor = None
    else:
        byte = torch.randint(0x20, 0x60, (E * N, nb), generator=g).numpy().astype(np.uint8)
        factor = (spread * torch.rand(E * N, generator=g) + 0.01).numpy().astype(np.float32)
    return codes, byte, factor, values(codes, byte, factor, fmt)


def matrix(ops, codes, byte, factor, E, fmt, device="cuda"):
    N, K = codes.shape[0] // E, codes.shape[1]
    lead = (N,) if E == 1 else (E, N)
    return ops.FP4Matrix.from_rows(torch.from_numpy(pack(codes)).view(*lead, -1).to(device),
                                   torch.from_numpy(byte).view(*lead, -1).to(device),
                                   None if factor is None else torch.from_numpy(factor).view(lead).to(device), fmt)


def activations(g, M, K):
    x = torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))
    return (x * (1 + 9 * (torch.rand(K, generator=g) < 0.02))).to(torch.bfloat16)


def act64(gate, act):
    if act == "silu":
        return gate / (1 + np.exp(np.minimum(-gate, 700)))
    return 0.5 * gate * (1 + np.tanh(math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3)))


def product_bound(y, xv, wv):
    """How far bf16(y) may be from y = xv wv^T.

    The sums: an instruction adds 64 exact products to the accumulator with at least 23 bits below the largest of its
    terms (a cut, not a rounding), 65 cuts of at most 2^-23 of a partial sum of magnitudes; K / 64 instructions; the
    row factors one rounding of 2^-24 each.  Together K 2^-23 (1 + 1 / 64) + 2^-22 of sum |x w|, taken as 1.1 K 2^-23
    for K >= 32 plus 2^-22.  The output: half a step of bf16, 2^-8 of the value, and the smallest subnormal.
    """
    mass = np.abs(xv) @ np.abs(wv).T
    K = xv.shape[1]
    err = (1.1 * K * 2.0 ** -23 + 2.0 ** -22) * mass
    return err + (np.abs(y) + err) * 2.0 ** -8 + 2.0 ** -133


def gated_bound(gate, up, xv, wg, wu, act):
    """... of bf16(act(gate) up).  Both activations have |act'| <= 1.13 and |act(g)| <= |g|; computed in fp32 from a
    gate that is off by dg they are off by 1.13 dg and some roundings: 16 of 2^-24 relative to |g| (the exponential's,
    the tanh's and the products')."""
    K = xv.shape[1]
    c = 1.1 * K * 2.0 ** -23 + 2.0 ** -22
    dg, du = c * (np.abs(xv) @ np.abs(wg).T), c * (np.abs(xv) @ np.abs(wu).T)
    a = act64(gate, act)
    da = 1.13 * dg + 16 * 2.0 ** -24 * (np.abs(gate) + dg)
    err = da * np.abs(up) + (np.abs(a) + da) * du + 2.0 ** -23 * np.abs(a * up)
    return err + (np.abs(a * up) + err) * 2.0 ** -8 + 2.0 ** -133
