"""Refusals of the microscaled 4-bit calls, sizes and layouts (no GPU: nothing is launched)."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch

import fp4_cases as fc
from skinny_gemm_gb300 import ops
from test_kv_devices_cpu import Stream, current, on  # noqa: F401  (fixture)

P, Q, R = 0x100000, 0x40000000, 0x80000000  # stand-in addresses, apart


@pytest.fixture()
def L(monkeypatch):
    monkeypatch.delenv("W4A16_FAULT", raising=False)
    lib = ops.lib()
    lib.w4a16_debug_reload_env()
    return lib


def matrix(rows=128, K=256, experts=1, fmt=1, codes=P, scales=P, row_scale=P):
    return ops.Fp4Struct(codes, scales, row_scale, rows, K, experts, fmt)


def ref(m):
    return ctypes.byref(m)  # (keeps m)


def err(L):
    return L.w4a16_last_error().decode()


@pytest.mark.parametrize("N,K", [(1, 32), (127, 64), (128, 96), (129, 2304), (1000, 16384)])
def test_sizes(L, N, K):
    for name, fmt in ops.FP4_FORMATS.items():
        want = -(-N // 128) * -(-(K // ops.FP4_BLOCK[name]) // 4) * 512
        assert ops.fp4_scale_bytes(N, K, name) == want == L.w4a16_fp4_scale_bytes(N, K, fmt)
        assert fc.tile_index(N, K // ops.FP4_BLOCK[name]).max() < want
        assert len(np.unique(fc.tile_index(N, K // ops.FP4_BLOCK[name]))) == N * K // ops.FP4_BLOCK[name]
        assert L.w4a16_fp4_mm_workspace_bytes(N, K, fmt) >= N * K // 2 + want + 4 * N
        assert L.w4a16_fp4_mm_id_workspace_bytes(N, 2, K, 4, fmt) > 0
    for bad in ((1, 33, 1), (1, 0, 1), (-1, 64, 1), (1, 64, 0), (1, 64, 3), ((1 << 30) + 1, 64, 1)):
        assert L.w4a16_fp4_scale_bytes(*bad) == 0 == L.w4a16_fp4_mm_workspace_bytes(*bad)
    for bad in ((-1, 1, 64, 4, 1), (1, 0, 64, 4, 1), (1, 1025, 64, 4, 1), (1, 1, 64, 0, 1), (1, 1, 64, 4097, 1), (1 << 30, 2, 64, 4, 1)):
        assert L.w4a16_fp4_mm_id_workspace_bytes(*bad) == 0


def test_matrix_refusals(L):
    """What every call checks of a matrix, through fp4_dequant."""
    def call(**kw):
        return L.w4a16_fp4_dequant(ref(matrix(**kw)), Q, None)

    assert L.w4a16_fp4_dequant(None, Q, None) == ops.ERR_NULL
    assert call(fmt=0) == call(fmt=3) == ops.ERR_SHAPE and "format" in err(L)
    assert call(K=0) == call(K=48) == call(K=-32) == ops.ERR_SHAPE and "multiple of 32" in err(L)
    assert call(experts=0) == call(experts=4097) == ops.ERR_EXPERTS
    assert call(rows=-1) == call(rows=1 << 29, experts=4) == ops.ERR_SHAPE
    assert call(codes=None) == call(scales=None) == ops.ERR_NULL
    assert call(codes=P + 8) == call(scales=P + 4) == call(row_scale=P + 2) == ops.ERR_ALIGN
    assert L.w4a16_fp4_dequant(ref(matrix()), None, None) == ops.ERR_NULL
    assert L.w4a16_fp4_dequant(ref(matrix()), Q + 8, None) == ops.ERR_ALIGN
    assert call(rows=0, codes=None, scales=None) == ops.OK
    assert call(codes=Q + 128 * 512 - 16) == call(scales=Q) == call(row_scale=Q + 64) == ops.ERR_SHAPE and "overlaps" in err(L)


def test_quant_refusals(L):
    def call(x=Q, stride=256, **kw):
        return L.w4a16_fp4_quant(x, stride, ref(matrix(**kw)), None)

    assert call(x=None) == ops.ERR_NULL
    assert call(row_scale=None) == ops.ERR_NULL and "row_scale" in err(L)
    assert call(stride=248) == ops.ERR_SHAPE and call(stride=260) == ops.ERR_ALIGN and call(x=Q + 8) == ops.ERR_ALIGN
    assert call(rows=0, x=None) == ops.OK
    for kw in ({"codes": Q + 2 * 127 * 256}, {"scales": Q + 512}, {"row_scale": Q - 4}, {"codes": Q - 128 * 128 + 16}):
        assert call(**kw) == ops.ERR_SHAPE and "overlaps" in err(L)


def test_mm_refusals(L):
    need = L.w4a16_fp4_mm_workspace_bytes(3, 256, 1)

    def call(x=Q, stride=256, y=R, M=3, act=0, ws=P, wn=need, **kw):
        return L.w4a16_fp4_mm(x, stride, ref(matrix(**kw)), y, M, act, ws, wn, None)

    assert call(M=-1) == ops.ERR_SHAPE and call(M=0, x=None, y=None, ws=None, wn=0) == ops.OK
    assert call(x=None) == call(y=None) == call(ws=None) == ops.ERR_NULL
    assert call(wn=need - 1) == ops.ERR_SHAPE and "too small" in err(L)
    assert call(ws=P + 128) == call(y=R + 1) == call(x=Q + 2) == call(stride=257) == ops.ERR_ALIGN
    assert call(stride=128) == ops.ERR_SHAPE
    assert call(act=3) == call(act=-1) == ops.ERR_KERNEL
    assert call(rows=127, act=1) == ops.ERR_SHAPE and "pairs" in err(L)
    assert call(rows=0) == ops.ERR_SHAPE
    assert call(experts=2) == ops.ERR_EXPERTS and "fp4_mm_id" in err(L)
    assert call(y=Q + 2 * 256) == call(y=Q - 2 * 3 * 128 + 2) == call(codes=R) == ops.ERR_SHAPE and "overlaps" in err(L)


def test_mm_q_refusals(L):
    def call(x=None, y=R, act=0, **kw):
        return L.w4a16_fp4_mm_q(ref(x or matrix(rows=5)), ref(matrix(**kw)), y, act, None)

    assert call(x=matrix(rows=5, K=288)) == call(x=matrix(rows=5, fmt=2)) == ops.ERR_SHAPE
    assert call(x=matrix(rows=5, experts=2)) == call(experts=2) == ops.ERR_EXPERTS
    assert call(y=None) == ops.ERR_NULL and call(y=R + 1) == ops.ERR_ALIGN and call(act=9) == ops.ERR_KERNEL
    assert call(x=matrix(rows=0), y=None) == ops.OK
    assert call(x=matrix(rows=5, codes=R)) == call(x=matrix(rows=5, row_scale=R + 4)) == call(scales=R + 16) == ops.ERR_SHAPE and "overlaps" in err(L)


def test_mm_id_refusals(L):
    need = L.w4a16_fp4_mm_id_workspace_bytes(3, 2, 256, 4, 1)

    def call(x=Q, stride=256, ids=P, y=R, T=3, top=2, act=0, ws=P, wn=need, **kw):
        kw.setdefault("experts", 4)
        return L.w4a16_fp4_mm_id(x, stride, ref(matrix(**kw)), ids, y, T, top, act, ws, wn, None)

    assert call(T=-1) == call(top=0) == call(top=1025) == call(T=1 << 30) == ops.ERR_EXPERTS
    assert call(T=0, x=None, ids=None, y=None, ws=None, wn=0) == ops.OK
    assert call(ids=None) == call(y=None) == call(ws=None) == call(x=None) == ops.ERR_NULL
    assert call(ids=P + 2) == call(ws=P + 64) == ops.ERR_ALIGN
    assert call(wn=need - 1) == ops.ERR_SHAPE and call(y=Q) == ops.ERR_SHAPE and call(rows=1, act=2) == ops.ERR_SHAPE


def test_injected_faults(L, monkeypatch):
    for fault, code in (("validate", ops.ERR_SHAPE), ("launch", ops.ERR_CUDA)):
        monkeypatch.setenv("W4A16_FAULT", fault)
        L.w4a16_debug_reload_env()
        m, x = matrix(), matrix(rows=2)
        big = 1 << 30
        assert L.w4a16_fp4_quant(Q, 256, ref(m), None) == code
        assert L.w4a16_fp4_dequant(ref(m), Q, None) == code
        assert L.w4a16_fp4_mm(Q, 256, ref(m), R, 1, 0, P, big, None) == code
        assert L.w4a16_fp4_mm_q(ref(x), ref(m), R, 0, None) == code
        assert L.w4a16_fp4_mm_id(Q, 256, ref(m), P, R, 1, 1, 0, P, big, None) == code
    monkeypatch.delenv("W4A16_FAULT")
    L.w4a16_debug_reload_env()


def u8(where, n):
    return on(where, n, dtype=torch.uint8)


def host_matrix(where=0, N=64, K=64, E=1, fmt="nv"):
    return ops.FP4Matrix(u8(where, E * N * K // 2), u8(where, E * ops.fp4_scale_bytes(N, K, fmt)),
                         on(where, E * N, dtype=torch.float32) if fmt == "nv" else None, N, K, E, fmt)


def test_matrix_arguments(current):  # noqa: F811
    c, s, f = u8(0, 64 * 32), u8(0, 512), on(0, 64, dtype=torch.float32)
    for args in ((c, s, f, 64, 96), (c, u8(0, 511), f, 64, 64), (c, s, on(0, 63, dtype=torch.float32), 64, 64), (c, s, f, 64, 64, 2),
                 (c, s, f, 64, 64, 1, "e5"), (c, s, f, 64, 48), (c, u8(1, 512), f, 64, 64), (c, s, on(1, 64, dtype=torch.float32), 64, 64)):
        with pytest.raises(ValueError):
            ops.FP4Matrix(*args)
    with pytest.raises(ValueError):
        ops.FP4Matrix(torch.zeros(64 * 32, dtype=torch.uint8), s, f, 64, 64)
    with pytest.raises(TypeError):
        ops.FP4Matrix([0], s, f, 64, 64)
    m = host_matrix(E=2)
    assert m.nbytes == 2 * (64 * 32 + 512 + 4 * 64) and m._c.experts == 2


def test_calls_take_one_device(current):  # noqa: F811
    x, other = on(0, 3, 64, dtype=torch.bfloat16), on(1, 3, 64, dtype=torch.bfloat16)
    w, far = host_matrix(0), host_matrix(1)
    for call in (lambda: ops.fp4_mm(other, w), lambda: ops.fp4_mm(x, far), lambda: ops.fp4_mm(host_matrix(1, 3), w), lambda: ops.fp4_quant(other),
                 lambda: ops.fp4_dequant(far), lambda: ops.fp4_mm(x, w, stream=Stream(1)), lambda: ops.fp4_mm(x, w, out=on(1, 3, 64, dtype=torch.bfloat16)),
                 lambda: ops.fp4_mm(x, w, out=on(0, 3, 64, dtype=torch.bfloat16), workspace=u8(1, 4096)),
                 lambda: ops.fp4_quant(x, out=host_matrix(1, 3)), lambda: ops.fp4_gated(other, w),
                 lambda: ops.fp4_mm_id(x, host_matrix(0, E=2), on(1, 3)), lambda: ops.fp4_mm_id(x, host_matrix(1, E=2), on(0, 3))):
        with pytest.raises(ValueError):
            call()


def test_call_arguments(current):  # noqa: F811
    x, w = on(0, 3, 64, dtype=torch.bfloat16), host_matrix(0)
    e = host_matrix(0, E=2)
    for call in (lambda: ops.fp4_mm(x[:, :32], w), lambda: ops.fp4_mm(x.float(), w), lambda: ops.fp4_mm(x.t(), w), lambda: ops.fp4_mm(x, e),
                 lambda: ops.fp4_mm(x, w, out=on(0, 3, 63, dtype=torch.bfloat16)), lambda: ops.fp4_gated(x, w, act=None), lambda: ops.fp4_gated(x, w, act="relu"),
                 lambda: ops.fp4_gated(x, host_matrix(0, N=63)), lambda: ops.fp4_mm(host_matrix(0, N=3, fmt="mx"), w), lambda: ops.fp4_quant(x, format="int4"),
                 lambda: ops.fp4_quant(on(0, 3, 48, dtype=torch.bfloat16)), lambda: ops.fp4_quant(x, out=host_matrix(0, N=4)),
                 lambda: ops.fp4_mm_id(x, e, on(0, 4)), lambda: ops.fp4_mm_id(x, e, on(0, 3, 0)), lambda: ops.fp4_mm_id(x, e, on(0, 3, dtype=torch.int64)),
                 lambda: ops.fp4_mm_id(on(0, 1, 3, 64, dtype=torch.bfloat16), e, on(0, 3)),
                 lambda: ops.FP4Matrix.gated(x, on(0, 4, 64, dtype=torch.bfloat16)), lambda: ops.FP4Matrix.from_rows(u8(0, 64).view(2, 32), u8(0, 8).view(2, 4), format="fp4"),
                 lambda: ops.FP4Matrix.from_rows(u8(0, 64).view(2, 32), u8(0, 6).view(2, 3))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_plain_quantiser_properties(fmt):
    """The tests' own 64-bit quantiser: codes of values that it can hold are those values, errors are half a step."""
    g = torch.Generator().manual_seed(5)
    x = fc.activations(g, 40, 192)
    codes, byte, factor = fc.quant(x, fmt)
    v = fc.values(codes, byte, factor, fmt)
    again = fc.values(*fc.quant(torch.from_numpy(v).to(torch.bfloat16), fmt), fmt)
    assert np.array_equal(v, again) or fmt == "nv"  # (nv: a block's largest code may be 4 afterwards)
    b = np.abs(x.double().numpy()).reshape(40, -1, fc.BLOCK[fmt]).max(-1).repeat(fc.BLOCK[fmt], 1)
    # the widest step is 2 of 6 (nv, whose scale is off by 2^-4 more) or of 4 (mx, past 6 cut to it: a quarter)
    assert (np.abs(v - x.double().numpy()) <= b * (0.25 if fmt == "mx" else 1 / 6 + 0.08) + 1e-30).all()
