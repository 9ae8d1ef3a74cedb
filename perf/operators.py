"""The operators around a paged key/value cache held in 8 bits, as a serving loop over the W4A16 projections calls them.

Three operators, each called once per decoding (or speculative-verify, or chunked-prefill) step:

* ``plan``    block tables, slots and positions of the step's tokens from the requests' lengths, blocks taken from a free list;
* ``append``  the step's keys and values written into their slots as e4m3 codes, one power-of-two scale per (block, head);
* ``attend``  causal attention of the step's queries over that cache, grouped heads, optionally a sliding window.

``run`` is either the plain form (elementary torch operations in 32 bits) or, with ``own`` set, the framework's entry points.
Head layouts: (8, 2, 256) is the one of the decode-layer projection set of this repository's benchmark (q 2048 x 2560 and
k/v 512 x 2560, heads of 256); the others are generic.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -64  # the smallest scale of a block is 2**-64


def listed():
    return [
        # plan: eight requests decoding one token each: the smallest call, all launch latency
        dict(name="plan_decode_b8", op="plan", B=8, ctx=4000, new=1, ragged=False, block=64, lens=1),
        # plan: a full batch verifying five drafted tokens per request, small blocks
        dict(name="plan_verify_b200", op="plan", B=200, ctx=16000, new=5, ragged=False, block=16, lens=2),
        # plan: many requests whose prompts are admitted in ragged chunks (about 65k tokens)
        dict(name="plan_chunks_b333", op="plan", B=333, ctx=2000, new=400, ragged=True, block=32, lens=3),
        # append: one new token of each of 48 requests; the decode step's write
        dict(name="append_decode_b48", op="append", B=48, ctx=4000, new=1, ragged=False, block=64, hq=8, hkv=2, dim=256, lens=4),
        # append: nine ragged prompt chunks up to 2000 tokens
        dict(name="append_chunks_b9", op="append", B=9, ctx=1500, new=2000, ragged=True, block=16, hq=32, hkv=8, dim=128, lens=5),
        # attend: one short request, the smallest call
        dict(name="attend_decode_b1", op="attend", B=1, ctx=1000, new=1, ragged=False, block=64, hq=8, hkv=2, dim=256, window=0, lens=6),
        # attend: an ordinary ragged decode batch
        dict(name="attend_decode_b32", op="attend", B=32, ctx=8000, new=1, ragged=True, block=16, hq=32, hkv=8, dim=128, window=0, lens=7),
        # attend: one very long request; the work has to be split along the cache
        dict(name="attend_long_b1", op="attend", B=1, ctx=131071, new=1, ragged=False, block=64, hq=8, hkv=2, dim=256, window=0, lens=8),
        # attend: the largest decode batch (0.5 GB of cache)
        dict(name="attend_decode_b64", op="attend", B=64, ctx=16000, new=1, ragged=True, block=64, hq=8, hkv=2, dim=256, window=0, lens=9),
        # attend: speculative verify, four drafted tokens and the last accepted one
        dict(name="attend_verify_b16", op="attend", B=16, ctx=16000, new=5, ragged=False, block=64, hq=8, hkv=2, dim=256, window=0, lens=10),
        # attend: a sliding-window layer of the same model on long requests
        dict(name="attend_window_b40", op="attend", B=40, ctx=30000, new=3, ragged=True, block=32, hq=8, hkv=2, dim=256, window=1024, lens=11),
        # attend: ragged prompt chunks over what is already cached, seven query heads a key head
        dict(name="attend_chunks_b3", op="attend", B=3, ctx=6000, new=300, ragged=True, block=128, hq=28, hkv=4, dim=128, window=0, lens=12),
    ]


HEADS = ((8, 2, 256), (8, 1, 256), (32, 8, 128), (28, 4, 128), (64, 8, 128), (12, 4, 64), (16, 16, 128))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("plan", "append", "append", "attend", "attend", "attend"))
    case = dict(op=op, block=rng.choice((16, 32, 64, 128)), ragged=rng.random() < 0.7, lens=rng.randrange(1 << 30))
    if op == "plan":
        B = _log(rng, 1, 1000)
        return dict(case, B=B, ctx=_log(rng, 1, 30000), new=_log(rng, 1, max(1, min(2000, 65000 // B))))
    hq, hkv, dim = rng.choice(HEADS)
    case.update(hq=hq, hkv=hkv, dim=dim)
    if op == "append":
        B = _log(rng, 1, 256)
        return dict(case, B=B, ctx=_log(rng, 1, 4000), new=_log(rng, 1, max(1, min(2000, 16000 // B))))
    case["window"] = rng.choice((0, 0, 0, 512, 1000))
    # tokens x key heads x dim up to the largest listed case's, and few enough scores for the plain form
    B, most = _log(rng, 1, 128), 32 * 16000 * 2 * 256
    ctx = _log(rng, 1, max(1, min(131000, most // (B * hkv * dim))))
    new = rng.choice((1, 1, 1, 2, 3, 4, 5, 6, 7, 8, _log(rng, 9, 300)))
    new = max(1, min(new, 11_000_000_000 // (B * hq * dim * (ctx + 300))))
    return dict(case, B=B, ctx=ctx, new=new)


def _lengths(case):
    """(cached, new) of the case's requests: the same for every seed, so that the work is the case's own."""
    r = np.random.RandomState(case["lens"])
    B, ctx, new = case["B"], case["ctx"], case["new"]
    if case["ragged"]:
        return r.randint(0, ctx + 1, B).astype(np.int64), r.randint(1, new + 1, B).astype(np.int64)
    return np.full(B, ctx, np.int64), np.full(B, new, np.int64)


def _ceil(a, b):
    return -(-a // b)


def prepare(case, seed):
    """Lengths, tables and tensors of one step. The order of the requests, the blocks and every value follow the seed."""
    r = np.random.RandomState(seed % (1 << 31))
    g = torch.Generator(device="cuda").manual_seed(seed)
    cached, new = _lengths(case)
    order = r.permutation(len(cached))
    cached, new = cached[order], new[order]
    B, block = case["B"], case["block"]
    total = cached + new
    have, need = _ceil(cached, block), _ceil(total, block)
    max_blocks = int(need.max()) + 3
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1])
    blocks = int(need.sum()) + 5
    ids = r.permutation(blocks)  # blocks are handed out in no order
    state = dict(case=case, B=B, T=T, block=block, max_new=int(new.max()), max_len=int(total.max()))

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).cuda()

    table = np.full((B, max_blocks), -1, np.int64)
    cols = np.arange(max_blocks)[None]
    start = np.concatenate([[0], np.cumsum(have if case["op"] == "plan" else need)])
    held = have if case["op"] == "plan" else need
    at = np.minimum(start[:-1, None] + cols, blocks - 1)
    table = np.where(cols < held[:, None], ids[at], -1)
    state.update(table=dev(table), cu=dev(cu), lens=dev(total))
    if case["op"] == "plan":
        state.update(cached=dev(cached), new=dev(new), free=dev(ids[start[-1]:]), head=dev(np.array([2])))
        return state

    hkv, dim, hq = case["hkv"], case["dim"], case["hq"]
    which = np.repeat(np.arange(B), new)
    pos = np.arange(T) - cu[which] + cached[which]
    state["slots"] = dev(table[which, pos // block] * block + pos % block)

    def cache():
        # about N(0, 1) times a factor of its own for each block and head: layers' keys and values differ in size by place
        size = torch.exp(0.5 * torch.randn(blocks, hkv, 1, 1, device="cuda", generator=g))
        x = torch.randn(blocks, hkv, block, dim, device="cuda", generator=g).mul_(size)
        scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / E4M3_MAX)))
        return x.div_(scale[:, :, None, None]).to(torch.float8_e4m3fn), scale

    (state["k"], state["k_scale"]), (state["v"], state["v_scale"]) = cache(), cache()
    if case["op"] == "append":
        # the key and value columns of one projection's output row, as a fused q/k/v product leaves them
        qkv = torch.randn(T, (hq + 2 * hkv) * dim, device="cuda", generator=g).to(torch.bfloat16)
        state["k_new"] = qkv[:, hq * dim:(hq + hkv) * dim].view(T, hkv, dim)
        state["v_new"] = qkv[:, (hq + hkv) * dim:].view(T, hkv, dim)
    else:
        state["q"] = (1.5 * torch.randn(T, hq, dim, device="cuda", generator=g)).to(torch.bfloat16)
        state["span"] = _span(case, cached, new)
    return state


def _span(case, cached, new):
    """The most tokens that a request's queries reach: the plain form gathers no more."""
    first = np.maximum(cached - case["window"] + 1, 0) if case["window"] else np.zeros_like(cached)
    return int((cached + new - first).max())


# ---- the plain forms ---------------------------------------------------------------------


def _plain_plan(s):
    block, T = s["block"], s["T"]
    cached, new, table, free = s["cached"].long(), s["new"].long(), s["table"], s["free"]
    cu = torch.cat([cached.new_zeros(1), torch.cumsum(new, 0)])
    lens = cached + new
    have, need = (cached + block - 1) // block, (lens + block - 1) // block
    taken = torch.cat([cached.new_zeros(1), torch.cumsum(need - have, 0)]) + s["head"].long()
    col = torch.arange(table.shape[1], device="cuda")[None]
    at = (taken[:-1, None] + col - have[:, None]).clamp(0, free.numel() - 1)
    table = torch.where((col >= have[:, None]) & (col < need[:, None]), free[at], table)
    t = torch.arange(T, device="cuda")
    which = (t[:, None] >= cu[None, 1:]).sum(1)
    pos = t - cu[which] + cached[which]
    slots = table[which, pos // block] * block + pos % block
    return [table, cu.int(), lens.int(), slots.int(), pos.int(), taken[-1:].int()]


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (at least 2**MIN_EXP), by comparisons only."""
    m, e = torch.frexp(amax)  # amax = m 2**e, m in [0.5, 1); 448 = 0.875 * 2**9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp_min(MIN_EXP)
    e = torch.where(amax == 0, torch.full_like(e, MIN_EXP), e)
    return torch.ldexp(torch.ones_like(amax), e)


def _plain_append(s):
    block, B = s["block"], s["B"]
    slots, lead = s["slots"].long(), s["cu"][:-1].long()
    blk, off = slots // block, slots % block
    blk0, off0 = blk[lead], off[lead]  # each request's first touched block, and the rows it already holds
    rows = torch.arange(block, device="cuda")
    kept = rows[None, :] < off0[:, None]
    out = []
    for x, codes, scale in ((s["k_new"], s["k"], s["k_scale"]), (s["v_new"], s["v"], s["v_scale"])):
        x = x.float()
        peak = torch.zeros_like(scale).index_reduce_(0, blk, x.abs().amax(-1), "amax")
        fresh = _pow2_scale(peak[blk])
        # a block that holds earlier tokens keeps its scale unless the new ones need a larger one
        held = torch.zeros_like(scale)
        held[blk0] = torch.where(off0[:, None] > 0, scale[blk0], torch.zeros_like(scale[blk0]))
        old0 = held[blk0]
        now = torch.maximum(fresh, held[blk])
        now0 = now[lead]
        raw = codes.view(torch.uint8)
        old = raw[blk0]
        again = old.view(codes.dtype).float() * (old0 / now0)[:, :, None, None]
        again = again.to(codes.dtype).view(torch.uint8)
        raw[blk0] = torch.where(kept[:, None, :, None], again, old)
        raw[blk, :, off] = (x / now[:, :, None]).to(codes.dtype).view(torch.uint8)
        scale[blk] = now
        out += [codes, scale]
    return out


def _plain_attend(s):
    case, B, T, block, M, span = s["case"], s["B"], s["T"], s["block"], s["max_new"], s["span"]
    hq, hkv, dim, window = case["hq"], case["hkv"], case["dim"], case["window"]
    cu, lens = s["cu"].long(), s["lens"].long()
    new = cu[1:] - cu[:-1]
    cached = lens - new
    first = (cached - window + 1).clamp_min(0) if window else torch.zeros_like(cached)
    tok = first[:, None] + torch.arange(span, device="cuda")[None]  # [B, span] token positions
    exists = tok < lens[:, None]
    safe = torch.where(exists, tok, torch.zeros_like(tok))
    blk = torch.gather(s["table"].long(), 1, safe // block)
    at = blk * block * hkv + safe % block  # row of head 0; head h is h * block rows further
    head = torch.arange(hkv, device="cuda") * block

    def rows(codes, scale):
        x = codes.view(torch.uint8).view(-1, dim)[at[:, None, :] + head[None, :, None]].view(codes.dtype).float()
        return x.mul_(scale[blk].transpose(1, 2)[..., None])  # [B, hkv, span, dim]

    j = torch.arange(M, device="cuda")
    mine = j[None] < new[:, None]
    q = s["q"][torch.where(mine, cu[:-1, None] + j[None], torch.zeros_like(mine, dtype=torch.long))].float()
    q = q.view(B, M, hkv, hq // hkv, dim).permute(0, 2, 1, 3, 4).reshape(B, hkv, M * (hq // hkv), dim)
    score = q @ rows(s["k"], s["k_scale"]).transpose(2, 3)
    score = score.mul_(1.0 / math.sqrt(dim)).view(B, hkv, M, hq // hkv, span)
    at_row = cached[:, None] + j[None]  # [B, M]
    seen = (tok[:, None, :] <= at_row[:, :, None]) & exists[:, None, :]
    if window:
        seen = seen & (tok[:, None, :] > at_row[:, :, None] - window)
    score = score.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = p.view(B, hkv, -1, span) @ rows(s["v"], s["v_scale"])
    o = o.view(B, hkv, M, hq // hkv, dim) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.permute(0, 2, 1, 3, 4).reshape(B * M, hq, dim)
    t = torch.arange(T, device="cuda")
    which = (t[:, None] >= cu[None, 1:]).sum(1)
    return o[which * M + t - cu[which]].to(torch.bfloat16)


# ---- the framework's -----------------------------------------------------------------------


def _own(s):
    from skinny_gemm_gb300 import ops

    op = s["case"]["op"]
    if op == "plan":
        p = ops.kv_plan(s["cached"], s["new"], s["table"], s["free"], s["T"], s["block"], head=s["head"])
        return [s["table"], p.cu, p.lens, p.slots, p.positions, p.head]
    cache = s.get("cache")
    if cache is None:  # the handle that a serving loop keeps for each layer
        cache = s["cache"] = ops.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if op == "append":
        ops.kv_append(s["k_new"], s["v_new"], cache, s["slots"])
        return [s["k"], s["k_scale"], s["v"], s["v_scale"]]
    return ops.kv_attention(s["q"], cache, s["table"], s["cu"], s["lens"], s["max_new"], s["max_len"], window=s["case"]["window"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_plan(state) if op == "plan" else _plain_append(state) if op == "append" else _plain_attend(state)


def work(case):
    cached, new = _lengths(case)
    B, block = case["B"], case["block"]
    total, T = cached + new, int(new.sum())
    fresh = int((_ceil(total, block) - _ceil(cached, block)).sum())
    if case["op"] == "plan":
        # lengths in; the table entry of a started block per request; free blocks in and table entries out; cu, lens, slots, positions
        return dict(bytes=4 * (2 * B + int((cached % block > 0).sum()) + 2 * fresh + 2 * B + 1 + 2 * T), flops=0)
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    if case["op"] == "append":
        touched = int((_ceil(total, block) - cached // block).sum())
        return dict(bytes=2 * T * hkv * dim * 3 + 4 * T + 2 * 2 * 4 * touched * hkv, flops=2 * 3 * T * hkv * dim)
    first = np.maximum(cached - case["window"] + 1, 0) if case["window"] else np.zeros_like(cached)
    tokens = int((total - first).sum())
    blocks = int((_ceil(total, block) - first // block).sum())
    pairs = 0
    for c, n in zip(cached.tolist(), new.tolist()):
        seen = np.arange(c + 1, c + n + 1)
        pairs += int((np.minimum(seen, case["window"]) if case["window"] else seen).sum())
    return dict(bytes=2 * tokens * hkv * dim + blocks * (2 * 4 * hkv + 4) + 2 * 2 * T * hq * dim + 8 * B, flops=4 * pairs * hq * dim)


# ---- the definitions in 64 bits --------------------------------------------------------------


def _round_e4m3(y):
    """y (float64) to the nearest e4m3 value, ties to the even significand."""
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -30))).clamp_min(-6.0)
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    B, block = s["B"], s["block"]
    if case["op"] == "plan":
        return None  # whole numbers only
    hkv, dim, hq = case["hkv"], case["dim"], case["hq"]
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].long()
    if case["op"] == "append":
        out = []
        for x, codes, scale in ((s["k_new"], s["k"], s["k_scale"]), (s["v_new"], s["v"], s["v_scale"])):
            x, codes, scale = x.double(), codes.double(), scale.double()
            for b in range(B):
                new = cu[b + 1] - cu[b]
                at = lens[b] - new
                while at < lens[b]:
                    i, lo = int(table[b, at // block]), at % block
                    n = min(block - lo, lens[b] - at)
                    t = cu[b] + at - (lens[b] - new)
                    part = x[t:t + n].transpose(0, 1)  # [hkv, n, dim]
                    peak = part.abs().amax((1, 2))
                    want = torch.exp2(torch.ceil(torch.log2((peak / E4M3_MAX).clamp_min(2.0 ** MIN_EXP))))
                    if lo:
                        want = torch.maximum(want, scale[i])
                        codes[i, :, :lo] = _round_e4m3(codes[i, :, :lo] * (scale[i] / want)[:, None, None])
                    codes[i, :, lo:lo + n] = _round_e4m3(part / want[:, None, None])
                    scale[i] = want
                    at += n
            out += [codes, scale]
        return out
    if 4.0 * hq * dim * float(s["T"]) * s["span"] > 4e12:
        return None
    out = torch.zeros(s["T"], hq, dim, dtype=torch.float64, device="cuda")
    for b in range(B):
        L, new = lens[b], cu[b + 1] - cu[b]
        lo = max(0, L - new - case["window"] + 1) if case["window"] else 0
        blk = table[b, lo // block:_ceil(L, block)]
        off = lo - lo // block * block
        k = (s["k"].view(torch.uint8)[blk].view(torch.float8_e4m3fn).double() * s["k_scale"][blk].double()[:, :, None, None])
        v = (s["v"].view(torch.uint8)[blk].view(torch.float8_e4m3fn).double() * s["v_scale"][blk].double()[:, :, None, None])
        k = k.transpose(0, 1).reshape(hkv, -1, dim)[:, off:off + L - lo]
        v = v.transpose(0, 1).reshape(hkv, -1, dim)[:, off:off + L - lo]
        key = torch.arange(lo, L, device="cuda")
        row = torch.arange(L - new, L, device="cuda")
        hide = key[None] > row[:, None]
        if case["window"]:
            hide |= key[None] <= row[:, None] - case["window"]
        for h in range(hq):
            z = s["q"][cu[b]:cu[b + 1], h].double() @ k[h * hkv // hq].T / math.sqrt(dim)
            w = torch.softmax(z.masked_fill(hide, -math.inf), -1)
            out[cu[b]:cu[b + 1], h] = w @ v[h * hkv // hq]
    return out
