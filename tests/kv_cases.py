"""Plain 64-bit references and input builders for the paged key/value cache tests."""
from __future__ import annotations

import math

import numpy as np
import torch

E4M3_MAX, MIN_EXP = 448.0, -64


def e4m3_values() -> np.ndarray:
    """The value of every e4m3 code: sign, 4 exponent bits (bias 7), 3 significand bits; 0x7F / 0xFF are NaN."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        out[c] = math.nan if (c & 127) == 127 else (-v if c & 128 else v)
    return out


VALUES = e4m3_values()
FINITE = np.array(sorted(set(VALUES[np.isfinite(VALUES)])))


def round_e4m3(y: np.ndarray) -> np.ndarray:
    """y (finite, |y| <= 448) to the nearest e4m3 value, ties to the even significand."""
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -30))), -6.0)
    step = np.exp2(e - 3)
    return np.round(y / step) * step


def need_scale(peak: float) -> float:
    e = MIN_EXP
    while peak > E4M3_MAX * math.ldexp(1.0, e):
        e += 1
    return math.ldexp(1.0, e)


def ref_plan(cached, new, table, free, head, T, block):
    """kv_plan by loops: (table, cu, lens, slots, positions, head)."""
    table = [list(r) for r in table]
    cu, lens, slots, pos, at = [0], [], [-1] * T, [-1] * T, head
    t = 0
    for b in range(len(cached)):
        have, length = -(-cached[b] // block), cached[b] + new[b]
        for j in range(have, min(-(-length // block), len(table[b]))):
            table[b][j] = free[at] if at < len(free) else -1
            at += 1
        for p in range(cached[b], length):
            pos[t] = p
            j = p // block
            e = table[b][j] if j < len(table[b]) else -1
            slots[t] = e * block + p % block if e >= 0 else -1
            t += 1
        cu.append(t)
        lens.append(length)
    return table, cu, lens, slots, pos, min(at, max(head, len(free)))


def ref_append(x, slots, codes, scale, block):
    """kv_append of one of k, v by loops: x float64 [T, H, D]; codes float64 values
    [blocks, H, block, D] and scale [blocks, H] are changed in place."""
    T, H, _ = x.shape
    t = 0
    while t < T:
        if slots[t] < 0:
            t += 1
            continue
        i, o = divmod(int(slots[t]), block)
        n = 1
        while t + n < T and slots[t + n] == slots[t] + n and o + n < block:
            n += 1
        for h in range(H):
            rows = x[t:t + n, h]
            fin = np.isfinite(rows)
            s = need_scale(float(np.abs(rows[fin]).max(initial=0.0)))
            if o:
                s = max(s, float(scale[i, h]))
                codes[i, h, :o] = round_e4m3(codes[i, h, :o] * (float(scale[i, h]) / s))
            codes[i, h, o:o + n] = np.where(fin, round_e4m3(np.where(fin, rows, 0.0) / s), np.nan)
            scale[i, h] = s
        t += n


def make_lengths(B, T_max, new_max, seed, block):
    """Lengths with the edges in them: 0, 1, around a block's and a tile's end."""
    r = np.random.RandomState(seed)
    edge = [0, 1, block - 1, block, block + 1, 127, 128, 129, 1023, 1024, 1025]
    cached = [int(x) for x in r.randint(0, T_max + 1, B)]
    for i in range(B):
        if r.rand() < 0.5:
            cached[i] = min(T_max, edge[r.randint(len(edge))])
    new = [int(x) for x in r.randint(0, new_max + 1, B)]
    new[r.randint(B)] = new_max
    return cached, new


class Step:
    """A cache filled with random codes and one step's queries over it.

    Codes outside the requests' tokens are the NaN code, scales outside their
    blocks NaN: nothing a row does not see may reach it."""

    def __init__(self, hq, hkv, dim, block, cached, new, seed=0, spare=3, scale_spread=2):
        g = torch.Generator().manual_seed(seed)
        r = np.random.RandomState(seed)
        self.hq, self.hkv, self.dim, self.block = hq, hkv, dim, block
        self.cached, self.new = list(cached), list(new)
        self.lens = [c + n for c, n in zip(cached, new)]
        B = len(cached)
        need = [-(-n // block) for n in self.lens]
        self.max_blocks = max(1, max(need)) + 1
        blocks = sum(need) + spare
        ids = r.permutation(blocks)
        self.table = np.full((B, self.max_blocks), -1, np.int32)
        k = torch.full((blocks, hkv, block, dim), math.nan)
        v = torch.full((blocks, hkv, block, dim), math.nan)
        ks = torch.full((blocks, hkv), math.nan)
        vs = torch.full((blocks, hkv), math.nan)
        at = 0
        for b in range(B):
            for j in range(need[b]):
                i = int(ids[at])
                at += 1
                self.table[b, j] = i
                n = min(block, self.lens[b] - j * block)
                k[i, :, :n] = torch.randn(hkv, n, dim, generator=g) * 60
                v[i, :, :n] = torch.randn(hkv, n, dim, generator=g) * 60
                ks[i] = torch.exp2(torch.randint(-6 - scale_spread, -6 + 1, (hkv,), generator=g).float())
                vs[i] = torch.exp2(torch.randint(-6 - scale_spread, -6 + 1, (hkv,), generator=g).float())
        self.k, self.v = k.clamp(-448, 448).to(torch.float8_e4m3fn), v.clamp(-448, 448).to(torch.float8_e4m3fn)
        self.ks, self.vs = ks, vs
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.T = int(self.cu[-1])
        self.q = (torch.randn(self.T, hq, dim, generator=g) * 1.5).to(torch.bfloat16)

    def cache(self):
        from skinny_gemm_gb300 import ops
        return ops.KVCache(self.k.cuda(), self.v.cuda(), self.ks.cuda(), self.vs.cuda())

    def dev(self):
        """(table, cu, lens) on the GPU."""
        return (torch.from_numpy(self.table).cuda(), torch.from_numpy(self.cu).cuda(),
                torch.tensor(self.lens, dtype=torch.int32).cuda())

    def run(self, window=0, scale=None, cache=None, **kw):
        from skinny_gemm_gb300 import ops
        table, cu, lens = self.dev()
        return ops.kv_attention(self.q.cuda(), cache or self.cache(), table, cu, lens, max(1, max(self.new)),
                                max(1, max(self.lens)), scale=scale, window=window, **kw)

    def reference(self, window=0, scale=None):
        """(out, bound) in float64 [T, hq, dim].

        The bound, with w the normalised weights, A = sum w |v|:
          * output rounding to bf16: 2^-8 |y|
          * weights rounded to two e4m3 terms, the second at 2^-4 of the first: 2^-8 relative each, 2^-8 A;
            below the codes' normal range an absolute step, with a tile's largest w * v_scale at 256 the second
            term's half step is 2^-10 / 16 / 256 = 2^-22 of it: F = 2^-22 sum over tiles of max(w vs) sum |v code|
          * scores in fp32: |dz| <= (dim + 8) 2^-23 scale sum |q k|, which moves weights and their sum: 2 max|dz| A
          * sums and exponentials in fp32: (len / 128 + 32) 2^-23 A, doubled for weights and sum
        """
        scale = 1 / math.sqrt(self.dim) if scale is None else scale
        out = torch.zeros(self.T, self.hq, self.dim, dtype=torch.float64)
        bound = torch.zeros_like(out)
        G = self.hq // self.hkv
        for b in range(len(self.lens)):
            L, n = self.lens[b], self.new[b]
            if n == 0 or L == 0:
                continue
            ids = [int(i) for i in self.table[b, :-(-L // self.block)]]
            kc, vc = (c.view(torch.uint8)[ids].view(c.dtype).double().transpose(0, 1).reshape(self.hkv, -1, self.dim)[:, :L]
                      for c in (self.k, self.v))
            ks = self.ks[ids].double().T.repeat_interleave(self.block, 1)[:, :L]
            vs = self.vs[ids].double().T.repeat_interleave(self.block, 1)[:, :L]
            tile = torch.arange(L) // 128
            for m in range(n):
                pos = L - n + m
                lo = max(0, pos - window + 1) if window else 0
                see = slice(lo, pos + 1)
                for h in range(self.hkv):
                    q = self.q[self.cu[b] + m, h * G:(h + 1) * G].double()
                    k, v = kc[h, see] * ks[h, see, None], vc[h, see] * vs[h, see, None]
                    z = q @ k.T * scale
                    dz = (self.dim + 8) * 2.0 ** -23 * scale * (q.abs() @ k.abs().T).amax(1, keepdim=True)
                    w = torch.softmax(z, 1)
                    y, A = w @ v, w @ v.abs()
                    t = tile[see] - tile[see][0]
                    top = torch.zeros(G, int(t[-1]) + 1, dtype=torch.float64)
                    top = top.scatter_reduce(1, t.expand(G, -1), w * vs[h, see], "amax")
                    per = torch.zeros(int(t[-1]) + 1, self.dim, dtype=torch.float64).index_add(0, t, vc[h, see].abs())
                    F = 2.0 ** -22 * (top @ per)
                    rel = 2.0 ** -8 + 2 * dz + 2 * (L / 128 + 32) * 2.0 ** -23
                    r = slice(h * G, (h + 1) * G)
                    out[self.cu[b] + m, r] = y
                    bound[self.cu[b] + m, r] = 1.01 * (2.0 ** -8 * y.abs() + rel * A + F)
        return out, bound


def assert_close(got: torch.Tensor, ref: torch.Tensor, bound: torch.Tensor, what: str = "") -> float:
    g = got.double().cpu()
    assert torch.isfinite(g).all(), f"{what}: non-finite outputs"
    err = (g - ref).abs()
    bad = err > bound
    if bad.any():
        i = int(torch.argmax(err - bound))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside tolerance; worst {g.flatten()[i]} "
                             f"for {ref.flatten()[i]}, bound {bound.flatten()[i]:.3e}, "
                             f"at {np.unravel_index(i, tuple(bad.shape))}")
    return float((err / bound.clamp_min(1e-300)).max()) if bound.numel() else 0.0
