"""Microscaled 4-bit floating point, both operands: what a decoding loop calls where weights and activations are e2m1 codes.

Four operators, all over matrices of e2m1 codes with one scale per block of a row. Format "nv": blocks of 16 with e4m3
scales and a power of two per row; format "mx": blocks of 32 with power-of-two scales.

* ``quant``  rows of bf16 into codes and scales, and back into bf16 (the values that the codes stand for);
* ``mm``     y = x W^T: bf16 activations quantised row by row, times packed weights, bf16 out;
* ``gated``  h = act(x G^T) * (x U^T) over gate and up weights in one matrix, their rows interleaved;
* ``mm_id``  routed experts: row (t, j) of the output is W[ids[t, j]] x[t].

``run`` is either the plain form (elementary torch operations in 32 bits) or, with ``own`` set, the framework's entry points.
The shapes 10240 x 2560, 262144 x 2560, 9216 x 2304 and 8 x 6144 x 2048 are those of this repository's benchmark.
"""
import math

import numpy as np
import torch

own = False

BLOCK = {"nv": 16, "mx": 32}


def listed():
    return [
        # quant: the activation row of one decoded token, the smallest call
        dict(name="quant_nv_decode", op="quant", format="nv", M=1, K=2560),
        # quant: an odd chunk of a prompt over a hidden size that is no multiple of 512
        dict(name="quant_mx_chunk", op="quant", format="mx", M=333, K=2304),
        # quant: a long prompt's feed-forward activations
        dict(name="quant_nv_prompt", op="quant", format="nv", M=4001, K=10240),
        # mm: one token through the gate projection of a decode layer
        dict(name="mm_nv_decode", op="mm", format="nv", M=1, N=10240, K=2560),
        # mm: a verify step's five rows through the down projection
        dict(name="mm_mx_verify", op="mm", format="mx", M=5, N=2560, K=10240),
        # mm: one token through a tied LM head, all weight traffic
        dict(name="mm_nv_head", op="mm", format="nv", M=1, N=262144, K=2560),
        # mm: an odd prompt chunk through the down projection
        dict(name="mm_mx_chunk", op="mm", format="mx", M=777, N=2560, K=10240),
        # mm: a long prompt, bound by the tensor cores
        dict(name="mm_nv_prompt", op="mm", format="nv", M=4096, N=10240, K=2560),
        # gated: five verify rows through a feed-forward block's first half, hidden size 2304
        dict(name="gated_nv_verify", op="gated", format="nv", M=5, F=9216, K=2304, act="gelu"),
        # gated: a prompt chunk
        dict(name="gated_mx_chunk", op="gated", format="mx", M=1500, F=10240, K=2560, act="silu"),
        # mm_id: eight tokens, each to one of eight experts
        dict(name="mm_id_nv_decode", op="mm_id", format="nv", T=8, top=1, E=8, N=6144, K=2048),
        # mm_id: a prompt chunk, four of 64 experts a token, in no even shares
        dict(name="mm_id_nv_chunk", op="mm_id", format="nv", T=500, top=4, E=64, N=1536, K=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


SHAPES = ((10240, 2560), (2560, 10240), (9216, 2304), (2048, 2560), (512, 2560), (12288, 1536), (16384, 16384), (262144, 2560))
MOST_FLOPS = 2 * 4096 * 10240 * 2560


def draw(rng):
    op = rng.choice(("quant", "mm", "mm", "gated", "mm_id"))
    case = dict(op=op, format=rng.choice(("nv", "mx")))
    if op == "quant":
        M = _log(rng, 1, 4000)
        return dict(case, M=M, K=32 * _log(rng, 1, min(512, 1_200_000 // M)))
    if op == "mm_id":
        E, top = _log(rng, 2, 96), rng.choice((1, 1, 2, 4, 6))
        N, K = _log(rng, 50, 6144), 32 * _log(rng, 3, 80)
        E = max(2, min(E, 300_000_000 // (N * K)))
        top = min(top, E)
        T = _log(rng, 1, 1500)
        return dict(case, T=max(1, min(T, MOST_FLOPS // (2 * N * K * top))), top=top, E=E, N=N, K=K)
    N, K = rng.choice(SHAPES) if rng.random() < 0.5 else (_log(rng, 30, 20000), 32 * _log(rng, 2, 400))
    if op == "gated":
        N = min(N, 20000)
    M = _log(rng, 1, max(1, min(4000, MOST_FLOPS // (4 * N * K))))
    if op == "gated":
        return dict(case, M=M, F=N, K=K, act=rng.choice(("silu", "gelu")))
    return dict(case, M=M, N=N, K=K)


def _ceil(a, b):
    return -(-a // b)


# ---- inputs ----------------------------------------------------------------------------------


def _activations(rows, K, g):
    """About N(0, 1) times a size of the row's own, a few columns ten times larger, as hidden states are."""
    x = torch.randn(rows, K, device="cuda", generator=g)
    x *= torch.exp(0.7 * torch.randn(rows, 1, device="cuda", generator=g))
    return (x * (1 + 9 * (torch.rand(K, device="cuda", generator=g) < 0.01))).to(torch.bfloat16)


def _tile(scales, E, N):
    """Scale bytes [E * N, blocks] in the order in which they are kept: for each expert, 128 rows and 4 blocks of
    K the 512 bytes (row % 32, row / 32, block), rows and blocks padded with zero bytes."""
    nb = scales.shape[1]
    rows, cols = _ceil(N, 128) * 128, _ceil(nb, 4) * 4
    full = torch.zeros(E, rows, cols, dtype=torch.uint8, device=scales.device)
    full[:, :N, :nb] = scales.view(E, N, nb)
    return full.view(E, rows // 128, 4, 32, cols // 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(-1).contiguous()


def _untile(scales, E, N, nb):
    rows, cols = _ceil(N, 128) * 128, _ceil(nb, 4) * 4
    full = scales.view(E, rows // 128, cols // 4, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, rows, cols)
    return full[:, :N, :nb].reshape(E * N, nb)


def _weights(E, N, K, fmt, g):
    """Codes, scales and row factors of about N(0, 1 / K) weights, made some rows at a time."""
    codes, scales, factor = [], [], []
    step = max(1, (1 << 27) // K)
    for at in range(0, E * N, step):
        w = torch.randn(min(step, E * N - at), K, device="cuda", generator=g) / math.sqrt(K)
        c, s, f = _plain_quant(w.to(torch.bfloat16), fmt)
        codes.append(c[:, 0::2] | (c[:, 1::2] << 4))
        scales.append(s)
        factor.append(f)
    return torch.cat(codes), _tile(torch.cat(scales), E, N), torch.cat(factor) if fmt == "nv" else None


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, fmt, K = case["op"], case["format"], case["K"]
    s = dict(case)
    s["x"] = _activations(case["T"] if op == "mm_id" else case["M"], K, g)
    if op == "quant":
        return s
    E, N = case.get("E", 1), 2 * case["F"] if op == "gated" else case["N"]
    s["E"], s["N"] = E, N
    s["codes"], s["scales"], s["factor"] = _weights(E, N, K, fmt, g)
    if op == "mm_id":
        # a router's choice: the `top` largest of scores that favour some experts; the most rows of one expert is the
        # bound that a program with fixed buffers keeps
        score = torch.randn(case["T"], E, device="cuda", generator=g) + torch.randn(E, device="cuda", generator=g)
        s["ids"] = torch.topk(score, case["top"], dim=1).indices.to(torch.int32).contiguous()
        s["most"] = int(torch.bincount(s["ids"].view(-1).long(), minlength=E).max())
    return s


# ---- the plain forms -------------------------------------------------------------------------


def _exp2i(e):
    """2**e for whole e in -127..127, by its bits (a library's powers may be off by a rounding)."""
    return torch.where(e < -126, torch.full_like(e, 1 << 22), (e + 127) << 23).to(torch.int32).view(torch.float32)


def _plain_quant(x, fmt):
    """Codes (a byte each) [M, K], scale bytes [M, K / block] and row factors [M] of bf16 rows."""
    M, K = x.shape
    x = x.float()
    b = x.view(M, K // BLOCK[fmt], BLOCK[fmt])
    peak = b.abs().amax(-1)
    if fmt == "mx":
        e = torch.where(peak == 0, torch.full_like(peak, -127, dtype=torch.int32), torch.frexp(peak)[1] - 3).clamp_min(-127)
        y = b * _exp2i(-e[..., None])
        scale, factor = (e + 127).to(torch.uint8), None
    else:
        top = peak.amax(-1)
        m, e = torch.frexp(top)  # 2688 = 6 * 448 = 0.65625 * 2**12
        e = torch.where(m > 0.65625, e - 11, e - 12)
        factor = _exp2i(torch.where(top == 0, torch.full_like(e, -126), e.clamp_min(-126)))
        part = (peak / factor[:, None] / 6).to(torch.float8_e4m3fn)
        scale, held = part.view(torch.uint8), part.float()[..., None]
        y = torch.where(held == 0, torch.zeros_like(b), b / factor[:, None, None] / torch.where(held == 0, torch.ones_like(held), held))
    a = y.abs()
    c = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    c = torch.where(torch.signbit(x.view_as(y)), c + 8, c)
    return c.view(M, K), scale, factor


def _values(codes, scale, factor, fmt):
    """fp32 values of codes (a byte each) [M, K] with their scale bytes and row factors."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    M, K = codes.shape
    v = table[codes.int()].view(M, -1, BLOCK[fmt])
    if fmt == "mx":
        return (v * _exp2i(scale.int()[..., None] - 127)).view(M, K)
    return (v * scale.view(torch.float8_e4m3fn).float()[..., None] * factor[:, None, None]).view(M, K)


def _plain_weights(s):
    c = s["codes"]
    return _values(torch.stack([c & 15, c >> 4], -1).view(c.shape[0], -1), _untile(s["scales"], s["E"], s["N"], s["K"] // BLOCK[s["format"]]),
                   s["factor"], s["format"])


def _plain(s):
    op, fmt = s["op"], s["format"]
    codes, scale, factor = _plain_quant(s["x"], fmt)
    x = _values(codes, scale, factor, fmt)
    if op == "quant":
        return [x.to(torch.bfloat16)] + ([factor] if fmt == "nv" else [])
    w = _plain_weights(s)
    if op == "mm":
        return (x @ w.T).to(torch.bfloat16)
    if op == "gated":
        p = (x @ w.T).view(s["M"], s["F"], 2)
        gate, up = p[..., 0], p[..., 1]
        if s["act"] == "silu":
            act = gate / (1 + torch.exp(-gate))
        else:
            act = 0.5 * gate * (1 + torch.tanh(math.sqrt(2 / math.pi) * (gate + 0.044715 * gate * gate * gate)))
        return (act * up).to(torch.bfloat16)
    # each expert's rows side by side, padded to the most that one has
    E, T, top, N, K = s["E"], s["T"], s["top"], s["N"], s["K"]
    ids = s["ids"].view(-1).long()
    order = torch.argsort(ids, stable=True)
    count = torch.zeros(E, dtype=torch.long, device="cuda").index_add_(0, ids, torch.ones_like(ids))
    first = torch.cumsum(count, 0) - count
    place = ids[order] * s["most"] + torch.arange(T * top, device="cuda") - first[ids[order]]
    padded = torch.zeros(E * s["most"], K, device="cuda")
    padded[place] = x[order // top]
    y = torch.bmm(padded.view(E, s["most"], K), w.view(E, N, K).transpose(1, 2)).view(-1, N)
    out = torch.empty(T * top, N, dtype=torch.bfloat16, device="cuda")
    out[order] = y[place].to(torch.bfloat16)
    return out.view(T, top, N)


# ---- the framework's -------------------------------------------------------------------------


def _own(s):
    from skinny_gemm_gb300 import ops

    op, fmt = s["op"], s["format"]
    if op == "quant":
        q = ops.fp4_quant(s["x"], format=fmt)
        return [ops.fp4_dequant(q)] + ([q.row_scale] if fmt == "nv" else [])
    w = s.get("w")
    if w is None:  # the handle that a program keeps for each matrix
        w = s["w"] = ops.FP4Matrix(s["codes"], s["scales"], s["factor"], s["N"], s["K"], E=s["E"], format=fmt)
    if op == "mm":
        return ops.fp4_mm(s["x"], w)
    if op == "gated":
        return ops.fp4_gated(s["x"], w, act=s["act"])
    return ops.fp4_mm_id(s["x"], w, s["ids"])


def run(state):
    return _own(state) if own else _plain(state)


def _held(rows, K, fmt):
    """Bytes of a matrix of codes, scales and row factors."""
    return rows * (K / 2 + K / BLOCK[fmt] + (4 if fmt == "nv" else 0))


def work(case):
    op, fmt, K = case["op"], case["format"], case["K"]
    if op == "quant":
        # the values in, codes, scales and factors out; those in again, the values out
        M = case["M"]
        return dict(bytes=2 * 2 * M * K + 2 * _held(M, K, fmt), flops=4 * M * K)
    if op == "mm_id":
        # at least one expert's weights for each of the first token's choices; every expert's where all get rows
        T, top, E, N = case["T"], case["top"], case["E"], case["N"]
        touched = min(E, E * (1 - (1 - 1 / E) ** (T * top)))
        return dict(bytes=2 * T * K + 4 * T * top + _held(touched * N, K, fmt) + 2 * T * top * N, flops=2 * T * top * N * K)
    M, N = case["M"], 2 * case["F"] if op == "gated" else case["N"]
    return dict(bytes=2 * M * K + _held(N, K, fmt) + 2 * M * (N // 2 if op == "gated" else N), flops=2 * M * N * K)


# ---- the definitions in 64 bits ----------------------------------------------------------------


def _two(e):
    """2**e in 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _log2(y, up=False):
    """The whole number below (or above) log2(y), for y > 0."""
    m, e = torch.frexp(y)
    return torch.where(m == 0.5, e - 1, e) if up else e - 1


def _exact_rows(x, fmt):
    """(values, row factors) in 64 bits that the rows' codes stand for."""
    n = BLOCK[fmt]
    b = x.double().unflatten(1, (-1, n))
    peak = b.abs().amax(-1, keepdim=True)
    if fmt == "mx":
        # the power of two of the largest element, over that of the largest code (4)
        unit = _two((_log2(peak.clamp_min(2.0 ** -200)) - 2).clamp_min(-127))
        factor = None
    else:
        # the smallest power of two under which the largest element is at most 6 * 448
        factor = _two(_log2(peak.amax(1, keepdim=True).clamp_min(2.0 ** -200) / 2688, up=True).clamp_min(-126))
        want = peak / factor / 6
        step = _two(_log2(want.clamp_min(2.0 ** -40)).clamp_min(-6) - 3)
        scale = torch.round(want / step) * step  # to e4m3, ties to even
        unit = scale * factor
    y = (b / torch.where(unit == 0, torch.ones_like(unit), unit)).abs()
    step = _two(_log2(y.clamp_min(2.0 ** -40)).clamp(0, 2) - 1)
    code = (torch.round(y / step) * step).clamp_max(6.0)  # to e2m1, ties to even
    value = torch.where(unit == 0, torch.zeros_like(code), code) * unit * torch.sign(b)
    return value.flatten(1), None if factor is None else factor.flatten()


def _exact_weights(s, rows):
    """64-bit values of the given rows (a slice of the experts' stacked ones)."""
    fmt, N, K = s["format"], s["N"], s["K"]
    r = torch.arange(rows.start, rows.stop, device="cuda")
    lo, hi = s["codes"][rows] & 15, s["codes"][rows] >> 4
    c = torch.empty(len(r), K, dtype=torch.long, device="cuda")
    c[:, 0::2], c[:, 1::2] = lo.long(), hi.long()
    e, m = (c % 8) // 2, c % 2
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * _two(e - 1)) * torch.where(c > 7, -1.0, 1.0)
    # the scale of row r of an expert and block k lies at 512 (k / 4) + 16 (r % 32) + 4 (r / 32 % 4) + k % 4 of its 128 rows' part
    k = torch.arange(K // BLOCK[fmt], device="cuda")
    groups = _ceil(len(k), 4)
    tiles = (r // N) * _ceil(N, 128) + r % N // 128
    at = (tiles * groups * 512 + r % N % 32 * 16 + r % N % 128 // 32 * 4)[:, None] + (k // 4 * 512 + k % 4)[None]
    byte = s["scales"][at]
    f = _two(byte.long() - 127) if fmt == "mx" else byte.view(torch.float8_e4m3fn).double() * s["factor"][rows].double()[:, None]
    return v * f.repeat_interleave(BLOCK[fmt], 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, fmt = case["op"], case["format"]
    x, factor = _exact_rows(s["x"], fmt)
    if op == "quant":
        return [x] + ([factor] if fmt == "nv" else [])
    E, N = s["E"], s["N"]
    if op == "mm_id":
        ids = s["ids"].long()
        out = torch.zeros(case["T"], case["top"], N, dtype=torch.float64, device="cuda")
        for e in range(E):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            if len(t):
                out[t, j] = x[t] @ _exact_weights(s, slice(e * N, e * N + N)).T
        return out
    step = max(2, (1 << 26) // case["K"] // 2 * 2)
    p = torch.cat([x @ _exact_weights(s, slice(at, min(N, at + step))).T for at in range(0, N, step)], 1)
    if op == "mm":
        return p
    gate, up = p[:, 0::2], p[:, 1::2]
    if case["act"] == "silu":
        return gate * torch.sigmoid(gate) * up
    return 0.5 * gate * (1 + torch.tanh(math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3))) * up
