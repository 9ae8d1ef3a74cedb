"""Microscaled 4-bit products as programs run them: captured, on several streams, in a chain, with waits that run out, and past 2^31."""
import time
import zlib

import numpy as np
import pytest
import torch

import fp4_cases as fc
from skinny_gemm_gb300 import ops

pytestmark = pytest.mark.gpu


def gen(*seed):
    return torch.Generator().manual_seed(zlib.crc32(repr(seed).encode()))


def made(fmt, M, N, K, E=1):
    g = gen(fmt, M, N, K, E)
    codes, byte, factor, _ = fc.weights(g, E, N, K, fmt)
    return fc.activations(g, M, K).cuda(), fc.matrix(ops, codes, byte, factor, E, fmt)


# one of each kernel: rows quantised in the product, split over a cluster, several tiles a CTA, 64 rows, pairs, four and two pairs a tile
CASES = [("nv", 1, 500, 2560), ("mx", 5, 300, 4096), ("nv", 9, 640, 2048), ("nv", 3, 50000, 256), ("mx", 60, 300, 512), ("nv", 100, 1000, 1024), ("nv", 400, 1500, 800),
         ("mx", 70, 300, 4096), ("nv", 300, 2500, 9024)]


@pytest.mark.parametrize("fmt,M,N,K", CASES)
def test_captured_and_replayed(fmt, M, N, K):
    """The first call of all is captured; replays take the inputs that are there then, and graphs of one stream do not share memory."""
    x, w = made(fmt, M, N, K)
    other = x.flip(0).contiguous() * 0.5
    y, z = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    a, b = x.clone(), other.clone()
    g, h = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        ops.fp4_mm(a, w, out=y)
    with torch.cuda.graph(h):
        ops.fp4_mm(b, w, out=z)
    want, want2 = ops.fp4_mm(x, w), ops.fp4_mm(other, w)
    for _ in range(3):
        g.replay()
        h.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(z, want2)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):  # both at once
        with torch.cuda.stream(s):
            g.replay()
        with torch.cuda.stream(t):
            h.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(z, want2)
    a.copy_(other)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want2) and ops.device_status() == 0


@pytest.mark.parametrize("fmt,M,N,K", CASES)
def test_streams(fmt, M, N, K):
    """Calls on several streams at once, with the stream's own workspaces and with given ones."""
    x, w = made(fmt, M, N, K)
    want = ops.fp4_mm(x, w)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty_like(want) for _ in range(6)]
    n = ops.lib().w4a16_fp4_mm_workspace_bytes(M, K, ops.FP4_FORMATS[fmt])
    own = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(4):
        for i, s in enumerate(streams):
            ops.fp4_mm(x, w, out=outs[i], stream=s)
            with torch.cuda.stream(s):
                ops.fp4_mm(x, w, out=outs[3 + i], workspace=own[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and ops.device_status() == 0


def test_routed_captured_and_streams():
    x, w = made("nv", 40, 130, 320, E=6)
    ids = torch.randint(0, 6, (40, 2), generator=gen(1), dtype=torch.int32).cuda()
    want = ops.fp4_mm_id(x, w, ids)
    y = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        ops.fp4_mm_id(x, w, ids, out=y)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty_like(want) for _ in range(3)]
    for _ in range(3):
        g.replay()
        for o, s in zip(outs, streams):
            ops.fp4_mm_id(x, w, ids, out=o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and all(torch.equal(o, want) for o in outs)
    ids.fill_(3)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ops.fp4_mm_id(x, w, ids)) and ops.device_status() == 0


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_weights_written_just_before(fmt, M):
    """Weights quantised, and written again, on the same stream right before the product that reads them."""
    g = gen(fmt, M)
    x = fc.activations(g, M, 512).cuda()
    a, b = (torch.randn(2000, 512, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    wa, wb = ops.fp4_quant(a, fmt), ops.fp4_quant(b, fmt)
    torch.cuda.synchronize()
    ya, yb = ops.fp4_mm(x, wa), ops.fp4_mm(x, wb)
    w = ops.FP4Matrix.empty(2000, 512, format=fmt)
    torch.cuda.synchronize()
    got = []
    for i in range(20):
        ops.fp4_quant(b if i % 2 else a, fmt, out=w)
        got.append(ops.fp4_mm(x, w))
    torch.cuda.synchronize()
    assert all(torch.equal(y, yb if i % 2 else ya) for i, y in enumerate(got))


@pytest.mark.parametrize("T,top,E", [(8, 1, 8), (30, 3, 20), (256, 4, 1024), (256, 4, 1025), (205, 5, 1024)])
def test_routes_and_experts_written_just_before(T, top, E):
    """Ids, activations and experts written on the same stream right before the call that reads them; rows without an expert among
    them."""
    g = gen(T, top, E)
    made_ids = [torch.randint(-1, E, (T, top), generator=g, dtype=torch.int32).cuda() for _ in range(2)]
    made_x = [fc.activations(g, T, 256).cuda() for _ in range(2)]
    made_w = [torch.randn(E, 40, 256, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    want = []
    for i, x, w in zip(made_ids, made_x, made_w):
        want.append(ops.fp4_mm_id(x, ops.fp4_quant(w), i))
        torch.cuda.synchronize()
    each = ops.fp4_dequant(ops.fp4_quant(made_w[1]))[made_ids[1].long().clamp(min=0)].double()
    plain = torch.einsum("tjnk,tk->tjn", each, ops.fp4_dequant(ops.fp4_quant(made_x[1])).double()) * (made_ids[1] >= 0)[..., None]
    assert (want[1].double() - plain).norm() <= 2.0 ** -8 * plain.norm()
    ids, x, w = torch.zeros_like(made_ids[0]), torch.zeros_like(made_x[0]), ops.FP4Matrix.empty(40, 256, E)
    torch.cuda.synchronize()
    for i in range(12):
        ops.fp4_quant(made_w[i % 2], out=w)
        x.copy_(made_x[i % 2])
        ids.copy_(made_ids[i % 2])
        assert torch.equal(ops.fp4_mm_id(x, w, ids), want[i % 2]), i
    got = []
    for i in range(12):
        ids.copy_(made_ids[i % 2])
        x.copy_(made_x[i % 2])
        ops.fp4_quant(made_w[i % 2], out=w)
        got.append(ops.fp4_mm_id(x, w, ids))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(got)) and ops.device_status() == ops.DEVICE_BAD_ID


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_block_of_a_decoder_layer(fmt):
    """A gated feed-forward block, a routed one and the shared quantisation of q, k and v in a row, captured as a step is, against
    float64 of the same chain of roundings."""
    g = gen(fmt, "layer")
    H, F, T, E = 320, 448, 6, 4
    x = fc.activations(g, T, H)
    wg, wu = (torch.randn(F, H, generator=g).div(H ** 0.5).to(torch.bfloat16) for _ in range(2))
    wd = torch.randn(H, F, generator=g).div(F ** 0.5).to(torch.bfloat16)
    we = torch.randn(E, 2 * F, H, generator=g).div(H ** 0.5).to(torch.bfloat16)
    qw = [torch.randn(n, H, generator=g).div(H ** 0.5).to(torch.bfloat16) for n in (256, 64, 64)]
    ids = torch.randint(0, E, (T, 2), generator=g, dtype=torch.int32).cuda()
    up, down = ops.FP4Matrix.gated(wg.cuda(), wu.cuda(), fmt), ops.fp4_quant(wd.cuda(), fmt)
    experts = ops.fp4_quant(we.cuda(), fmt)
    qkv = [ops.fp4_quant(w.cuda(), fmt) for w in qw]
    xd = x.cuda()

    def step():
        q = ops.fp4_quant(xd, fmt)
        heads = [ops.fp4_mm(q, w) for w in qkv]
        h = ops.fp4_gated(xd, up, act="gelu")
        return heads, h, ops.fp4_mm(h, down), ops.fp4_mm_id(xd, experts, ids, act="silu")

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        heads, h, y, routed = step()
    graph.replay()
    torch.cuda.synchronize()
    assert ops.device_status() == 0

    def held(t):
        return fc.values(*fc.quant(t.cpu(), fmt), fmt)

    def inside(got, want, bound):
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= bound).all(), (err / bound).max()

    xv = held(x)
    for got, w in zip(heads, qw):
        inside(got, xv @ held(w).T, fc.product_bound(xv @ held(w).T, xv, held(w)))
    gate, u = xv @ held(wg).T, xv @ held(wu).T
    inside(h, fc.act64(gate, "gelu") * u, fc.gated_bound(gate, u, xv, held(wg), held(wu), "gelu"))
    hv = held(h)  # the chain goes on from the rounded h
    inside(y, hv @ held(wd).T, fc.product_bound(hv @ held(wd).T, hv, held(wd)))
    for t in range(T):
        for j in range(2):
            w = held(we[int(ids[t, j])])
            gate, u = xv[t:t + 1] @ w[0::2].T, xv[t:t + 1] @ w[1::2].T
            inside(routed[t, j][None], fc.act64(gate, "silu") * u, fc.gated_bound(gate, u, xv[t:t + 1], w[0::2], w[1::2], "silu"))


@pytest.mark.parametrize("E", [1, 4096])
def test_many_experts_and_tokens(E):
    """More routed rows than every CTA counts for itself (a launch of its own finds the places), and the most experts."""
    T, top, N, K = (3000, 2, 66, 64) if E == 1 else (1200, 3, 18, 32)
    x, w = made("mx", T, N, K, E)
    ids = torch.randint(0, E, (T, top), generator=gen(E), dtype=torch.int32).cuda()
    ids[5, 0], ids[T - 1, top - 1] = -7, E
    y = ops.fp4_mm_id(x, w, ids)
    assert ops.device_status() == ops.DEVICE_BAD_ID
    xv = fc.values(*fc.quant(x.cpu(), "mx"), "mx")
    wv = ops.fp4_dequant(w).double().cpu().numpy().reshape(E, N, K)
    i = ids.cpu().numpy()
    bad = (i < 0) | (i >= E)
    want = np.einsum("tjnk,tk->tjn", wv[np.where(bad, 0, i)], xv) if E > 1 else np.repeat((xv @ wv[0].T)[:, None], top, 1)
    mass = np.abs(xv).sum(1)[:, None, None] * np.abs(wv).max()
    err = np.abs(y.double().cpu().numpy() - np.where(bad[..., None], 0, want))
    assert (err <= np.abs(want) * 2.0 ** -8 + mass * (1.1 * K * 2.0 ** -23 + 2.0 ** -22) * 1.01 + 2.0 ** -133).all()
    assert not y[torch.from_numpy(bad).cuda()].any()


def test_past_2_31():
    """Outputs and codes whose offsets do not fit 32 bits."""
    M, N, K = 8400, 262144, 32  # 2.2e9 values of y
    x, w = made("mx", M, N, K)
    y = ops.fp4_mm(x, w)
    xv, rows = fc.values(*fc.quant(x.cpu()[-300:], "mx"), "mx"), slice(N - 400, N)
    wv = ops.fp4_dequant(w)[rows].double().cpu().numpy()
    want = xv @ wv.T
    err = np.abs(y[-300:, rows].double().cpu().numpy() - want)
    assert (err <= fc.product_bound(want, xv, wv)).all() and ops.device_status() == 0
    del x, w, y
    torch.cuda.empty_cache()
    N, K = 140000, 32768  # 2.3e9 bytes of codes, a factor of 1
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((ops.fp4_scale_bytes(N, K, "nv"),), 0x30, dtype=torch.uint8, device="cuda")
    w = ops.FP4Matrix(codes, scales, None, N, K)
    x = fc.activations(gen(2), 3, K).cuda()
    y = ops.fp4_mm(x, w)
    xv = fc.values(*fc.quant(x.cpu(), "nv"), "nv")
    c = codes[-200:].cpu().numpy()
    c = np.stack([c & 15, c >> 4], -1).reshape(200, K)
    wv = fc.values(c, np.full((200, K // 16), 0x30, np.uint8), None, "nv")
    want = xv @ wv.T
    err = np.abs(y[:, -200:].double().cpu().numpy() - want)
    assert (err <= fc.product_bound(want, xv, wv)).all() and ops.device_status() == 0


@pytest.mark.parametrize("fmt,M,N,K", CASES)
def test_waits_run_out_and_the_context_survives(fmt, M, N, K, monkeypatch):
    """The first stage of one CTA waits for an arrival that never comes (every copy still lands): all roles give up, the flag is
    raised, and the next call is right."""
    x, w = made(fmt, M, N, K)
    want = ops.fp4_mm(x, w)
    assert ops.device_status() == 0
    monkeypatch.setenv("W4A16_FAULT", "wait")
    ops.lib().w4a16_debug_reload_env()
    try:
        t0 = time.perf_counter()
        ops.fp4_mm(x, w)
        flags = ops.device_status()
        elapsed = time.perf_counter() - t0
    finally:
        monkeypatch.delenv("W4A16_FAULT")
        ops.lib().w4a16_debug_reload_env()
    assert flags == ops.DEVICE_TIMEOUT and elapsed < 20
    for _ in range(3):
        assert torch.equal(ops.fp4_mm(x, w), want)
    assert ops.device_status() == 0


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("M,N,K", [(3, 512, 2048), (30, 512, 320), (9, 40000, 96), (300, 512, 320), (300, 520, 64)])
def test_outputs_at_any_address(M, N, K, act):
    """Outputs that begin at any even address are written whole, and nothing beside them."""
    x, w = made("nv", M, N, K)
    call = (lambda **kw: ops.fp4_mm(x, w, **kw)) if act is None else (lambda **kw: ops.fp4_gated(x, w, act, **kw))
    want = call()
    n = want.numel()
    for shift in (0, 1, 2, 4, 8, 13, 16):
        buf = torch.full((n + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
        out = buf[16 + shift:16 + shift + n].view(want.shape)
        call(out=out)
        assert torch.equal(out, want) and (buf[:16 + shift] == 5).all() and (buf[16 + shift + n:] == 5).all(), shift
    assert ops.device_status() == 0


@pytest.mark.parametrize("setting", ["0", "1"])
def test_launch_settings(setting, monkeypatch):
    """Plain launches, and overlapped ones without early fetches, give the same bits."""
    cases = [made(*c) for c in CASES]
    xe, we = made("nv", 50, 200, 96, E=5)
    ids = torch.randint(0, 5, (50, 3), generator=gen(9), dtype=torch.int32).cuda()
    want = [ops.fp4_mm(x, w) for x, w in cases] + [ops.fp4_mm_id(xe, we, ids)]
    monkeypatch.setenv("W4A16_PDL", setting)
    ops.lib().w4a16_debug_reload_env()
    try:
        got = [ops.fp4_mm(x, w) for x, w in cases] + [ops.fp4_mm_id(xe, we, ids)]
        torch.cuda.synchronize()
    finally:
        monkeypatch.delenv("W4A16_PDL")
        ops.lib().w4a16_debug_reload_env()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and ops.device_status() == 0


def test_between_the_library_s_other_calls():
    """Attention over the paged cache, affine 4-bit products and microscaled ones back to back on one stream, as launches that
    overlap; captured and not: the bits of the calls one by one."""
    from skinny_gemm_gb300 import synth

    H, hq, hkv, dim, T, E = 512, 8, 2, 64, 6, 3
    g = gen("mixed")
    wq = ops.W4Matrix.from_host(synth.make_weights(1, hq * dim, H))
    rand = lambda *s: torch.randn(*s, generator=g).div(s[-1] ** 0.5).to(torch.bfloat16).cuda()  # noqa: E731
    wkv, wo, w13, w2 = ops.fp4_quant(rand(2 * hkv * dim, H)), ops.fp4_quant(rand(H, hq * dim), "mx"), ops.FP4Matrix.gated(rand(1536, H), rand(1536, H)), ops.fp4_quant(rand(H, 1536))
    we = ops.fp4_quant(rand(E, 256, H), "mx")
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    big = torch.randn(200, H, generator=g).to(torch.bfloat16).cuda()
    ids = torch.randint(0, E, (T, 2), generator=g, dtype=torch.int32).cuda()
    cached = torch.tensor([700, 30], dtype=torch.int32, device="cuda")
    new = torch.tensor([4, 2], dtype=torch.int32, device="cuda")
    cache = ops.KVCache.empty(64, hkv, 16, dim)
    free = torch.arange(64, dtype=torch.int32, device="cuda")
    table = torch.full((2, 48), -1, dtype=torch.int32, device="cuda")
    first = ops.kv_plan(torch.zeros_like(cached), cached, table, free, 730, 16)
    ops.kv_append(*(torch.randn(730, hkv, dim, generator=g).to(torch.bfloat16).cuda() for _ in range(2)), cache, first.slots)
    plan = ops.kv_plan(cached, new, table, free, T, 16, head=first.head)
    torch.cuda.synchronize()

    def layer(sync=lambda: None):
        q = ops.mm(x, wq)
        sync()
        kv = ops.fp4_mm(x, wkv).view(T, 2 * hkv, dim)
        sync()
        ops.kv_append(kv[:, :hkv], kv[:, hkv:], cache, plan.slots)
        sync()
        o = ops.kv_attention(q.view(T, hq, dim), cache, table, plan.cu, plan.lens, 4, 768)
        sync()
        y = ops.fp4_mm(o.view(T, -1), wo)
        sync()
        h = ops.fp4_gated(y, w13)
        sync()
        z = ops.fp4_mm(h, w2)
        sync()
        r = ops.fp4_mm_id(z, we, ids)
        sync()
        p = ops.fp4_gated(big, w13)
        sync()
        return q, kv, o, y, h, z, r, p

    want = [t.clone() for t in layer(torch.cuda.synchronize)]
    for _ in range(20):
        got = layer()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer()
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and ops.device_status() == 0


@pytest.mark.parametrize("T,top,E", [(6, 1, 4), (300, 4, 9)])
def test_routed_waits_run_out(T, top, E, monkeypatch):
    x, w = made("nv", T, 200, 320, E)
    ids = torch.randint(0, E, (T, top), generator=gen(T), dtype=torch.int32).cuda()
    want = ops.fp4_mm_id(x, w, ids)
    monkeypatch.setenv("W4A16_FAULT", "wait")
    ops.lib().w4a16_debug_reload_env()
    try:
        ops.fp4_mm_id(x, w, ids)
        flags = ops.device_status()
    finally:
        monkeypatch.delenv("W4A16_FAULT")
        ops.lib().w4a16_debug_reload_env()
    assert flags == ops.DEVICE_TIMEOUT
    assert torch.equal(ops.fp4_mm_id(x, w, ids), want) and ops.device_status() == 0


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_longest_row(fmt):
    """K = 2^30.  Values that the codes hold exactly come back as they were; a product with few that are not zero is exact."""
    K = 1 << 30
    grid = torch.tensor([0.5, -1.5, 2, 0, -4, 1, -3, 6] * 4, dtype=torch.bfloat16, device="cuda")
    x = grid.repeat(K // 32).view(1, K)
    x[0, -32:] = grid.flip(0)
    w = ops.fp4_quant(x, fmt)
    assert torch.equal(ops.fp4_dequant(w), x)
    x.zero_()
    x[0, 6], x[0, K // 2 + 3], x[0, K - 3] = -3.0, 6.0, 4.0  # beside -3, 0 and 2
    # nv takes the 4 alone in its block for 4.125: its scale is e4m3(4 / 6) = 0.6875 (of a power of two; 2/3 lies between 0.625 and
    # that, nearer to it), its code e2m1(4 / 0.6875) = 6.  The -3 has scale 1/2 and comes back whole, and mx's scales are 1.
    assert ops.fp4_mm(x, w).item() == -3.0 * -3 + (4.125 if fmt == "nv" else 4.0) * 2 and ops.device_status() == 0


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_rows_and_values_at_any_sixteen_bytes(fmt):
    """Rows to quantise, and values that come back, at addresses and strides of 16 bytes."""
    x = torch.randn(70, 96, generator=gen(fmt)).to(torch.bfloat16).cuda()
    want = ops.fp4_quant(x, fmt)
    back = ops.fp4_dequant(want)
    for shift in (0, 8, 16, 24):
        wide = torch.full((70 * 104 + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
        rows = wide[shift:shift + 70 * 104].view(70, 104)[:, :96]
        rows.copy_(x)
        w = ops.fp4_quant(rows, fmt)
        assert torch.equal(w.codes, want.codes) and torch.equal(ops.fp4_dequant(w), back), shift
        for M in (3, 70):
            assert torch.equal(ops.fp4_mm(rows[:M], want), ops.fp4_mm(x[:M], want)), (shift, M)
        buf = torch.full((70 * 96 + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
        ops.fp4_dequant(want, out=buf[shift:shift + 70 * 96].view(70, 96))
        assert torch.equal(buf[shift:shift + 70 * 96].view(70, 96), back) and (buf[:shift] == 5).all() and (buf[shift + 70 * 96:] == 5).all()
    assert ops.device_status() == 0


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("T,top,E,N,K", [(5, 2, 6, 130, 320), (100, 1, 3, 300, 4096), (300, 2, 3, 500, 320), (1500, 1, 20, 130, 96)])
def test_one_expert_or_none(fmt, T, top, E, N, K):
    """All rows of one expert, so that tiles which there might be are not there; and no row with an expert at all."""
    x, w = made(fmt, T, N, K, E=E)
    xv, wv = ops.fp4_dequant(ops.fp4_quant(x, fmt)).double(), ops.fp4_dequant(w).double()
    for e in (0, E - 1):
        y = ops.fp4_mm_id(x, w, torch.full((T, top), e, dtype=torch.int32, device="cuda"))
        want = xv @ wv[e].T
        assert ((y.double() - want[:, None]).norm() <= 2.0 ** -8 * want.norm() * top ** 0.5) and ops.device_status() == 0
        assert all(torch.equal(y[:, 0], y[:, j]) for j in range(top))
    out = torch.full((T, top, N), 3.0, dtype=torch.bfloat16, device="cuda")
    for e in (-1, E, 2 ** 31 - 1, -2 ** 31):
        out.fill_(3.0)
        ops.fp4_mm_id(x, w, torch.full((T, top), e, dtype=torch.int32, device="cuda"), out=out)
        assert ops.device_status() == ops.DEVICE_BAD_ID and not out.any()
    one = torch.full((T, top), -1, dtype=torch.int32, device="cuda")
    one[T // 2, 0] = 1
    y = ops.fp4_mm_id(x, w, one)
    assert ops.device_status() == ops.DEVICE_BAD_ID and y[T // 2, 0].any() and not y[:T // 2].any() and not y[T // 2 + 1:].any() and not y[:, 1:].any()


@pytest.mark.parametrize("fmt,M,N,K", [("nv", 300, 2500, 9024), ("mx", 130, 640, 4096), ("nv", 2000, 2600, 512)])
def test_many_rows_on_two_streams_at_once(fmt, M, N, K):
    """Calls that fill the GPU, some as clusters of four pairs, at once on several streams and in replayed graphs."""
    x, w = made(fmt, M, N, K)
    want = ops.fp4_mm(x, w)
    streams = [torch.cuda.Stream() for _ in range(3)]
    graphs, outs = [], [torch.empty_like(want) for _ in range(6)]
    torch.cuda.synchronize()
    for o in outs[3:]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.fp4_mm(x, w, out=o)
        graphs.append(g)
    for _ in range(8):
        for s, o, g in zip(streams, outs, graphs):
            ops.fp4_mm(x, w, out=o, stream=s)
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and ops.device_status() == 0


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("top,E,N,K,act", [(2, 9, 130, 2048, None), (4, 64, 96, 1024, "silu"), (8, 20, 200, 320, None), (1, 3, 514, 4096, "gelu"), (3, 5, 40, 96, None)])
def test_routed_rows_do_not_depend_on_the_batch(fmt, top, E, N, K, act):
    """A few tokens (quantised in the product), more, and tokens 80 bytes further apart: the rows of the one call of them all."""
    x, w = made(fmt, 40, N, K, E=E)
    g = gen(top, E, N)
    ids = torch.randint(0, E, (40, top), generator=g, dtype=torch.int32).cuda()
    want = ops.fp4_mm_id(x, w, ids, act=act)
    wide = torch.full((40, K + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :K] = x
    for T in (1, 2, 3, 4, 5, 8, 10, 11, 16, 17, 32, 33):
        for a in (0, 40 - T):
            y = ops.fp4_mm_id(x[a:a + T], w, ids[a:a + T].contiguous(), act=act)
            assert torch.equal(y, want[a:a + T]), (T, a)
            assert torch.equal(ops.fp4_mm_id(wide[a:a + T, :K], w, ids[a:a + T].contiguous(), act=act), y)
    x2 = x.clone()
    x2[1, 5], x2[2, 7] = float("nan"), float("inf")
    y = ops.fp4_mm_id(x2[:4], w, ids[:4].contiguous(), act=act)
    assert y[1:3].isnan().all() and torch.equal(y[0], want[0]) and torch.equal(y[3], want[3])
    assert ops.device_status() == 0


def test_few_tokens_captured_and_on_streams():
    """One launch a call: replayed while the same runs on other streams, with ids that change between replays."""
    x, w = made("nv", 4, 1536, 2048, E=64)
    ids = torch.randint(0, 64, (4, 8), generator=gen(4), dtype=torch.int32).cuda()
    other = torch.randint(-1, 64, (4, 8), generator=gen(5), dtype=torch.int32).cuda()
    want, want2 = ops.fp4_mm_id(x, w, ids), ops.fp4_mm_id(x, w, other)
    assert (want2[other < 0] == 0).all() and ops.device_status() == ops.DEVICE_BAD_ID
    now, y = ids.clone(), torch.full_like(want, 7.0)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        ops.fp4_mm_id(x, w, now, out=y)
        ops.fp4_mm_id(x, w, now, out=y)
    streams, outs = [torch.cuda.Stream() for _ in range(3)], [torch.empty_like(want) for _ in range(3)]
    torch.cuda.synchronize()
    for i in range(6):
        now.copy_(other if i % 2 else ids)
        for s, o in zip(streams, outs):
            ops.fp4_mm_id(x, w, ids, out=o, stream=s)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want2 if i % 2 else want) and all(torch.equal(o, want) for o in outs)
    ops.device_status()
