"""Python binding of libw4a16.so: argument marshalling only.

Every computation runs in the library's CUDA kernels.  PyTorch supplies the
device memory, the current CUDA stream and the output allocation; there is
no CPU or PyTorch fallback, and a missing or unbuildable library raises.

Names follow the C ABI in ``include/w4a16.h``: ``mm``, ``mm_group``,
``mm_id``, ``unpack``, ``dequant``, ``get_plan``, ``device_status``; and in
``include/stq1.h`` for the STQ1_0 ternary format: ``stq1_mm``,
``stq1_mm_id``, ``stq1_get_rows``, ``stq1_get_plan`` over an ``STQ1Matrix``
(repacked on the device by ``stq1_pack``).  Between a layer's q/k/v and o
projections: ``kv_plan``, ``kv_append`` and ``kv_attention`` over a ``KVCache``
(paged keys and values in 8 bits).  Microscaled 4-bit floating point on both
operands: ``fp4_quant``, ``fp4_dequant``, ``fp4_mm``, ``fp4_gated`` and
``fp4_mm_id`` over an ``FP4Matrix``.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import threading
from dataclasses import dataclass

import torch

from . import _build

GROUP = 64

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_EXPERTS, ERR_CUDA, ERR_KERNEL, ERR_DEVICE = 0, -1, -2, -3, -4, -5, -6, -7
KERNELS = {"auto": 0, "simt": 1, "tc": 2, "vanilla": 3, "tc_stream": 4, "tc_tile": 5, "tc_prefill": 6}
KERNEL_NAMES = {v: k for k, v in KERNELS.items()}
DEVICE_BAD_ID, DEVICE_TIMEOUT, DEVICE_KV_RANGE = 1, 2, 4

EXPORTS = ("w4a16_mm", "w4a16_mm_ws", "w4a16_mm_g", "w4a16_workspace_bytes", "w4a16_mm_kernel", "w4a16_mm_noalloc", "w4a16_mm_group", "w4a16_mm_argmax", "w4a16_embed", "w4a16_expand_groups",
           "w4a16_mm_id", "w4a16_mm_id_kernel", "w4a16_unpack", "w4a16_dequant", "w4a16_get_plan", "w4a16_device_status", "w4a16_last_error",
           "w4a16_debug_reload_env", "w4a16_version",
           "w4a16_kv_plan", "w4a16_kv_append", "w4a16_kv_attention", "w4a16_kv_attention_workspace_bytes",
           "w4a16_fp4_scale_bytes", "w4a16_fp4_quant", "w4a16_fp4_dequant", "w4a16_fp4_mm_workspace_bytes", "w4a16_fp4_mm",
           "w4a16_fp4_mm_q", "w4a16_fp4_mm_id_workspace_bytes", "w4a16_fp4_mm_id",
           "stq1_packed_bytes", "stq1_pack", "stq1_mm", "stq1_mm_id", "stq1_get_rows", "stq1_get_plan")
MAX_GROUP = 8
STQ1_BLOCK_WEIGHTS, STQ1_BLOCK_BYTES = 256, 42


class W4A16Error(RuntimeError):
    """A library call failed; ``status`` is the w4a16_status code."""

    def __init__(self, status: int, message: str):
        super().__init__(f"w4a16 status {status}: {message}")
        self.status = status


class W4A16ValueError(W4A16Error, ValueError):
    pass


class Plan(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("ksplit", ctypes.c_int), ("slice_k", ctypes.c_int),
                ("rows_per_tile", ctypes.c_int), ("units", ctypes.c_int), ("threads", ctypes.c_int),
                ("grid_x", ctypes.c_int), ("smem_bytes", ctypes.c_int), ("workspace_bytes", ctypes.c_int)]

    def as_dict(self) -> dict:
        d = {f: getattr(self, f) for f, _ in self._fields_}
        d["kernel"] = KERNEL_NAMES.get(self.kernel, self.kernel)
        return d


class Stq1Plan(ctypes.Structure):
    _fields_ = [("ksplit", ctypes.c_int), ("blocks_per_slice", ctypes.c_int), ("rows_per_pass", ctypes.c_int)]


class Item(ctypes.Structure):
    """w4a16_mm_item: one projection of a w4a16_mm_group call (device pointers)."""
    _fields_ = [("x", ctypes.c_void_p), ("Wq", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("biases", ctypes.c_void_p), ("y", ctypes.c_void_p), ("N", ctypes.c_int)]


class KvCacheStruct(ctypes.Structure):
    """w4a16_kv_cache (device pointers)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("blocks", ctypes.c_int), ("heads", ctypes.c_int),
                ("block", ctypes.c_int), ("dim", ctypes.c_int)]


class Fp4Struct(ctypes.Structure):
    """w4a16_fp4 (device pointers)."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("row_scale", ctypes.c_void_p),
                ("rows", ctypes.c_int), ("K", ctypes.c_int), ("experts", ctypes.c_int), ("format", ctypes.c_int)]


_lock = threading.Lock()
_lib: ctypes.CDLL | None = None


def library_path() -> str:
    return _build.CUDA_LIB


def lib() -> ctypes.CDLL:
    """Open libw4a16.so (building it in-tree if it is missing or stale)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.build_cuda()
            L = ctypes.CDLL(path)
            P, i, z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            L.w4a16_mm.argtypes = [P, P, P, P, P, i, i, i, P]
            L.w4a16_mm_ws.argtypes = [P, P, P, P, P, i, i, i, P, z, P]
            L.w4a16_mm_g.argtypes = [P, P, P, P, P, i, i, i, i, P, z, P]
            L.w4a16_workspace_bytes.argtypes = [i, i]
            L.w4a16_workspace_bytes.restype = z
            L.w4a16_mm_kernel.argtypes = [P, P, P, P, P, i, i, i, i, P]
            L.w4a16_mm_noalloc.argtypes = [P, P, P, P, P, i, i, i, P]
            L.w4a16_mm_group.argtypes = [ctypes.POINTER(Item), i, i, i, P]
            L.w4a16_mm_argmax.argtypes = [P, P, P, P, P, P, i, i, i, P, z, P]
            L.w4a16_embed.argtypes = [P, P, P, P, P, i, i, i, P]
            L.w4a16_expand_groups.argtypes = [P, P, i, i, i, P]
            L.w4a16_mm_id.argtypes = [P, P, P, P, P, P, i, i, i, i, P]
            L.w4a16_mm_id_kernel.argtypes = [P, P, P, P, P, P, i, i, i, i, i, P]
            L.w4a16_unpack.argtypes = [P, P, i, i, P]
            L.w4a16_dequant.argtypes = [P, P, P, P, i, i, P]
            L.w4a16_get_plan.argtypes = [i, i, i, ctypes.POINTER(Plan)]
            L.w4a16_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_int)]
            ll, f = ctypes.c_int64, ctypes.c_float
            L.w4a16_kv_plan.argtypes = [P] * 10 + [i] * 5 + [P]
            L.w4a16_kv_append.argtypes = [P, ll, P, ll, P, P, i, P]
            L.w4a16_kv_attention.argtypes = [P, ll, P, P, P, P, P] + [i] * 7 + [f, P, z, P, P]
            L.w4a16_kv_attention_workspace_bytes.argtypes = [i] * 8
            L.w4a16_kv_attention_workspace_bytes.restype = z
            L.w4a16_fp4_scale_bytes.argtypes = [i, i, i]
            L.w4a16_fp4_quant.argtypes = [P, ll, P, P]
            L.w4a16_fp4_dequant.argtypes = [P, P, P]
            L.w4a16_fp4_mm_workspace_bytes.argtypes = [i, i, i]
            L.w4a16_fp4_mm.argtypes = [P, ll, P, P, i, i, P, z, P]
            L.w4a16_fp4_mm_q.argtypes = [P, P, P, i, P]
            L.w4a16_fp4_mm_id_workspace_bytes.argtypes = [i, i, i, i, i]
            L.w4a16_fp4_mm_id.argtypes = [P, ll, P, P, P, i, i, i, P, z, P]
            for f in ("w4a16_fp4_scale_bytes", "w4a16_fp4_mm_workspace_bytes", "w4a16_fp4_mm_id_workspace_bytes"):
                getattr(L, f).restype = z
            L.stq1_packed_bytes.argtypes = [i, i]
            L.stq1_packed_bytes.restype = ctypes.c_size_t
            L.stq1_pack.argtypes = [P, P, i, i, P]
            L.stq1_mm.argtypes = [P, P, P, i, i, i, P]
            L.stq1_mm_id.argtypes = [P, P, P, P, i, i, i, i, P]
            L.stq1_get_rows.argtypes = [P, P, P, i, i, i, P]
            L.stq1_get_plan.argtypes = [i, i, ctypes.POINTER(Stq1Plan)]
            for f in ("w4a16_mm", "w4a16_mm_ws", "w4a16_mm_g", "w4a16_mm_kernel", "w4a16_mm_noalloc", "w4a16_mm_group", "w4a16_mm_argmax",
                      "w4a16_embed", "w4a16_expand_groups", "w4a16_mm_id", "w4a16_mm_id_kernel", "w4a16_unpack", "w4a16_dequant",
                      "w4a16_get_plan", "w4a16_device_status", "w4a16_kv_plan", "w4a16_kv_append", "w4a16_kv_attention",
                      "w4a16_fp4_quant", "w4a16_fp4_dequant", "w4a16_fp4_mm", "w4a16_fp4_mm_q", "w4a16_fp4_mm_id",
                      "stq1_pack", "stq1_mm", "stq1_mm_id", "stq1_get_rows",
                      "stq1_get_plan"):
                getattr(L, f).restype = ctypes.c_int
            L.w4a16_last_error.restype = ctypes.c_char_p
            L.w4a16_version.restype = ctypes.c_char_p
            L.w4a16_debug_reload_env.restype = None
            _lib = L
    return _lib


def _raise(rc: int) -> None:
    if rc == OK:
        return
    msg = (lib().w4a16_last_error() or b"").decode()
    if rc in (ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_EXPERTS, ERR_KERNEL):
        raise W4A16ValueError(rc, msg)
    raise W4A16Error(rc, msg)


def _stream_ptr(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _empty(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """What a call on ``stream`` (None: the current one) writes and returns: memory of
    that stream, as the current one may still be busy with its own, and not given back
    before the current one is done with it either."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    now = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if now != stream:
        t.record_stream(now)
    return t


def _dev_tensor(t: torch.Tensor, dtype: torch.dtype, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


# ---- workspaces (include/w4a16.h "Workspace") --------------------------------------------
#
# The library allocates nothing; this binding is its caller and owns the
# workspaces: one zeroed block per (device, stream), made with torch on the
# first call on that stream outside graph capture (a call captured before
# one exists runs without a workspace, which gives the same bits).

_ws_lock = threading.Lock()
_ws_cache: dict = {}


def workspace_bytes(N: int, K: int) -> int:
    return int(lib().w4a16_workspace_bytes(N, K))


def _capturing() -> bool:
    try:
        return bool(torch.cuda.is_current_stream_capturing())
    except Exception:
        return False


def workspace(stream=None, create: bool = True):
    """The zeroed workspace of the current device and `stream` (uint8 tensor),
    or None when there is none yet and one cannot be made now."""
    s = stream if stream is not None else torch.cuda.current_stream()
    key = (s.device.index if s.device.index is not None else torch.cuda.current_device(), int(s.cuda_stream))
    with _ws_lock:
        ws = _ws_cache.get(key)
        if ws is None and create and not _capturing():
            n = int(lib().w4a16_workspace_bytes(512, 512))
            ws = torch.zeros(n, dtype=torch.uint8, device=f"cuda:{key[0]}")
            torch.cuda.current_stream(ws.device).synchronize()
            _ws_cache[key] = ws
        return ws


def _ws_args(ws):
    if ws is None:
        return None, 0
    _dev_tensor(ws, torch.uint8, "workspace")
    return ws.data_ptr(), ws.numel()


def _g64(w, what: str) -> None:
    if w.group != GROUP:
        raise ValueError(f"{what} takes group-64 tables; expand group {w.group} with W4Matrix.from_group")


def _kernel_id(kernel) -> int:
    if kernel is None:
        return 0
    if isinstance(kernel, str):
        if kernel not in KERNELS:
            raise ValueError(f"unknown kernel {kernel!r}; one of {sorted(KERNELS)}")
        return KERNELS[kernel]
    return int(kernel)


@dataclass
class W4Matrix:
    """Packed W4A16 weights on the GPU.

    Wq: int32 [.., N, K/8] (bit pattern of the uint32 words, eight codes each,
    low nibble first); scales, biases: bfloat16 [.., N, K/group] (group 64,
    or 128 for a single matrix read natively by ``mm``).  With E > 1 the
    leading dimension stacks E experts.
    """

    Wq: torch.Tensor
    scales: torch.Tensor
    biases: torch.Tensor
    N: int
    K: int
    E: int = 1
    group: int = GROUP

    def __post_init__(self):
        lead = () if self.E == 1 else (self.E,)
        if self.group not in (GROUP, 128) or (self.group != GROUP and self.E != 1):
            raise ValueError(f"group {self.group}: 64, or 128 for a single matrix")
        if tuple(self.Wq.shape) != lead + (self.N, self.K // 8):
            raise ValueError(f"Wq shape {tuple(self.Wq.shape)} does not match N={self.N}, K={self.K}, E={self.E}")
        for name in ("scales", "biases"):
            t = getattr(self, name)
            if tuple(t.shape) != lead + (self.N, self.K // self.group):
                raise ValueError(f"{name} shape {tuple(t.shape)} does not match N={self.N}, K={self.K}, "
                                 f"group={self.group}")
        _dev_tensor(self.Wq, torch.int32, "Wq")
        _dev_tensor(self.scales, torch.bfloat16, "scales")
        _dev_tensor(self.biases, torch.bfloat16, "biases")

    @classmethod
    def from_host(cls, host, device="cuda") -> "W4Matrix":
        """From numpy arrays (``synth.HostW4``: uint32 codes, bf16 bit patterns)."""
        wq = torch.from_numpy(host.Wq.view("int32")).to(device)
        s = torch.from_numpy(host.scales.view("int16")).view(torch.bfloat16).to(device)
        b = torch.from_numpy(host.biases.view("int16")).view(torch.bfloat16).to(device)
        return cls(wq, s, b, host.N, host.K, host.E)

    @classmethod
    def from_group(cls, Wq: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor, N: int, K: int,
                   group: int, stream=None) -> "W4Matrix":
        """A table quantized with `group` codes per scale and bias (a multiple
        of 64, e.g. the book's 128): scales/biases bf16 [N][K/group] expanded
        once on the device through ``w4a16_expand_groups``.  The stream is
        synchronised after the expansion: the tensor-core calls may fetch
        weights before earlier kernels on their stream finish (the
        overlapped-launch contract of include/w4a16.h)."""
        _dev_tensor(scales, torch.bfloat16, "scales")
        _dev_tensor(biases, torch.bfloat16, "biases")
        if scales.numel() != N * (K // group) or biases.numel() != N * (K // group):
            raise ValueError(f"scales and biases must hold N * K / group = {N * (K // group)} values")
        out = []
        for t in (scales, biases):
            d = _empty((N, K // GROUP), torch.bfloat16, t.device, stream)
            _raise(lib().w4a16_expand_groups(t.data_ptr(), d.data_ptr(), N, K, group, _stream_ptr(stream)))
            out.append(d)
        (stream if stream is not None else torch.cuda.current_stream()).synchronize()
        return cls(Wq, out[0], out[1], N, K)

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.Wq, self.scales, self.biases))


def mm(x: torch.Tensor, w: W4Matrix, out: torch.Tensor | None = None, kernel=None, stream=None,
       workspace="auto") -> torch.Tensor:
    """y[..., N] = x[..., K] W^T (leading dims flatten into M) through
    ``w4a16_mm_ws`` with this stream's workspace (``workspace="auto"``), a
    given uint8 workspace tensor, or ``w4a16_mm`` (``workspace=None``); an
    explicit ``kernel`` goes through ``w4a16_mm_kernel`` without one."""
    if w.E != 1:
        raise ValueError("mm takes a single matrix; use mm_id for stacked experts")
    _dev_tensor(x, torch.bfloat16, "x")
    if x.shape[-1] != w.K:
        raise ValueError(f"x has K={x.shape[-1]}, weights have K={w.K}")
    if w.group != GROUP and kernel not in (None, "auto", 0):
        raise ValueError("group-128 tables run on their own kernel; no kernel selection")
    M = x.numel() // w.K
    if out is None:
        out = _empty((*x.shape[:-1], w.N), torch.bfloat16, x.device, stream)
    _dev_tensor(out, torch.bfloat16, "out")
    if out.numel() != M * w.N:
        raise ValueError("out has the wrong number of elements")
    L = lib()
    k = _kernel_id(kernel)
    args = (x.data_ptr(), w.Wq.data_ptr(), w.scales.data_ptr(), w.biases.data_ptr(), out.data_ptr(), M, w.N, w.K)
    if w.group != GROUP:
        ws = globals()["workspace"](stream) if isinstance(workspace, str) else workspace
        rc = L.w4a16_mm_g(*args, w.group, *_ws_args(ws), _stream_ptr(stream))
    elif k != 0:
        rc = L.w4a16_mm_kernel(*args, k, _stream_ptr(stream))
    else:
        ws = globals()["workspace"](stream) if isinstance(workspace, str) else workspace
        if ws is None:
            rc = L.w4a16_mm(*args, _stream_ptr(stream))
        else:
            rc = L.w4a16_mm_ws(*args, *_ws_args(ws), _stream_ptr(stream))
    _raise(rc)
    return out


def mm_argmax(x: torch.Tensor, w: W4Matrix, idx: torch.Tensor | None = None, val: torch.Tensor | None = None,
              stream=None, workspace="auto"):
    """(idx, val) through ``w4a16_mm_argmax``: for every row of x (leading dims
    flatten into M) the index of the largest output of ``mm(x, w)`` and that
    output (ties to the smallest index), without writing the outputs.

    idx is int32 [..], val bf16 [..]; pass ``val=False`` to skip the values.
    The call needs a workspace: this stream's (``"auto"``; make one call on
    the stream before capturing it into a CUDA graph) or a given one."""
    _g64(w, "mm_argmax")
    if w.E != 1:
        raise ValueError("mm_argmax takes a single matrix")
    _dev_tensor(x, torch.bfloat16, "x")
    if x.shape[-1] != w.K:
        raise ValueError(f"x has K={x.shape[-1]}, weights have K={w.K}")
    M = x.numel() // w.K
    if idx is None:
        idx = _empty(x.shape[:-1], torch.int32, x.device, stream)
    _dev_tensor(idx, torch.int32, "idx")
    if idx.numel() != M:
        raise ValueError("idx must have one element per row")
    if val is None:
        val = _empty(x.shape[:-1], torch.bfloat16, x.device, stream)
    if val is not False:
        _dev_tensor(val, torch.bfloat16, "val")
        if val.numel() != M:
            raise ValueError("val must have one element per row")
    vp = val.data_ptr() if val is not False else None
    ws = globals()["workspace"](stream) if isinstance(workspace, str) else workspace
    if ws is None and M > 0:
        raise ValueError("mm_argmax needs a workspace: call it once on this stream before graph capture, "
                         "or pass workspace=")
    rc = lib().w4a16_mm_argmax(x.data_ptr(), w.Wq.data_ptr(), w.scales.data_ptr(), w.biases.data_ptr(), idx.data_ptr(),
                               vp, M, w.N, w.K, *_ws_args(ws), _stream_ptr(stream))
    _raise(rc)
    return idx, (val if val is not False else None)


def embed(ids: torch.Tensor, w: W4Matrix, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rows ids of the packed table w (N rows of width K), dequantized to bf16
    [..., K] through ``w4a16_embed``; ids int32 on the device."""
    _g64(w, "embed")
    if w.E != 1:
        raise ValueError("embed takes a single table")
    _dev_tensor(ids, torch.int32, "ids")
    T = ids.numel()
    if out is None:
        out = _empty((*ids.shape, w.K), torch.bfloat16, ids.device, stream)
    _dev_tensor(out, torch.bfloat16, "out")
    if out.numel() != T * w.K:
        raise ValueError("out has the wrong number of elements")
    rc = lib().w4a16_embed(w.Wq.data_ptr(), w.scales.data_ptr(), w.biases.data_ptr(), ids.data_ptr(), out.data_ptr(),
                           T, w.N, w.K, _stream_ptr(stream))
    _raise(rc)
    return out


def mm_group(xs, ws, outs=None, stream=None) -> list:
    """[mm(x, w) for x, w in zip(xs, ws)] through one ``w4a16_mm_group`` call.

    The projections must share K and the number of activation rows M; each
    result equals ``mm(x, w)`` bit for bit."""
    xs, ws = list(xs), list(ws)
    if not 1 <= len(xs) == len(ws) <= MAX_GROUP:
        raise ValueError(f"need 1..{MAX_GROUP} (x, w) pairs")
    K = ws[0].K
    M = xs[0].numel() // K if K else 0
    if outs is None:
        outs = [_empty((*x.shape[:-1], w.N), torch.bfloat16, x.device, stream) for x, w in zip(xs, ws)]
    items = (Item * len(xs))()
    for i, (x, w, y) in enumerate(zip(xs, ws, outs)):
        if w.E != 1:
            raise ValueError("mm_group takes single matrices")
        _g64(w, "mm_group")
        _dev_tensor(x, torch.bfloat16, "x")
        _dev_tensor(y, torch.bfloat16, "out")
        if w.K != K or x.shape[-1] != K or x.numel() != M * K:
            raise ValueError("every item must have the same K and the same number of rows")
        if y.numel() != M * w.N:
            raise ValueError("out has the wrong number of elements")
        items[i] = Item(x.data_ptr(), w.Wq.data_ptr(), w.scales.data_ptr(), w.biases.data_ptr(), y.data_ptr(), w.N)
    _raise(lib().w4a16_mm_group(items, len(xs), M, K, _stream_ptr(stream)))
    return outs


def mm_id(x: torch.Tensor, w: W4Matrix, ids: torch.Tensor, out: torch.Tensor | None = None, kernel=None,
          stream=None) -> torch.Tensor:
    """y[t] = W[ids[t]] x[t] through ``w4a16_mm_id``; x [T, K], ids int32 [T] on the GPU."""
    _g64(w, "mm_id")
    _dev_tensor(x, torch.bfloat16, "x")
    _dev_tensor(ids, torch.int32, "ids")
    if x.dim() != 2 or x.shape[1] != w.K:
        raise ValueError("x must be [T, K]")
    T = x.shape[0]
    if ids.numel() != T:
        raise ValueError("ids must hold one expert id per token")
    if out is None:
        out = _empty((T, w.N), torch.bfloat16, x.device, stream)
    _dev_tensor(out, torch.bfloat16, "out")
    L = lib()
    rc = L.w4a16_mm_id_kernel(x.data_ptr(), w.Wq.data_ptr(), w.scales.data_ptr(), w.biases.data_ptr(),
                              ids.data_ptr(), out.data_ptr(), T, w.N, w.K, w.E, _kernel_id(kernel),
                              _stream_ptr(stream))
    _raise(rc)
    return out


def unpack(w: W4Matrix, stream=None) -> torch.Tensor:
    """Codes q[N][K] as uint8 through ``w4a16_unpack`` (bit-exact debug path)."""
    q = _empty((w.N, w.K), torch.uint8, w.Wq.device, stream)
    _raise(lib().w4a16_unpack(w.Wq.data_ptr(), q.data_ptr(), w.N, w.K, _stream_ptr(stream)))
    return q


def dequant(w: W4Matrix, stream=None) -> torch.Tensor:
    """fp32 weights fma(q, s, b) [N][K] through ``w4a16_dequant``."""
    _g64(w, "dequant")
    out = _empty((w.N, w.K), torch.float32, w.Wq.device, stream)
    _raise(lib().w4a16_dequant(w.Wq.data_ptr(), w.scales.data_ptr(), w.biases.data_ptr(), out.data_ptr(),
                               w.N, w.K, _stream_ptr(stream)))
    return out


def get_plan(N: int, K: int, kernel=None) -> dict:
    p = Plan()
    _raise(lib().w4a16_get_plan(N, K, _kernel_id(kernel), ctypes.byref(p)))
    return p.as_dict()


def device_status(stream=None) -> int:
    """Synchronise and return (then clear) the device flags; raises on CUDA errors only."""
    flags = ctypes.c_int(0)
    rc = lib().w4a16_device_status(_stream_ptr(stream), ctypes.byref(flags))
    if rc not in (OK, ERR_DEVICE):
        _raise(rc)
    if flags.value & DEVICE_TIMEOUT and (_kv_counter_cache or _kv_capture_sets):
        _kv_reset_counters(torch.cuda.current_device())
    return flags.value


# ---- STQ1_0 ternary matrices (include/stq1.h) -------------------------------------------

@dataclass
class STQ1Matrix:
    """An STQ1_0 matrix (or E stacked experts) repacked on the GPU for the
    stq1 kernels: ``packed`` uint8 [E * stq1_packed_bytes(N, K)]."""

    packed: torch.Tensor
    N: int
    K: int
    E: int = 1

    @classmethod
    def from_blocks(cls, blocks: torch.Tensor, N: int, K: int, E: int = 1, stream=None) -> "STQ1Matrix":
        """From the page's 42-byte blocks, uint8 [.., N, K/256, 42] on the GPU."""
        _dev_tensor(blocks, torch.uint8, "blocks")
        per = stq1_packed_bytes(N, K)
        if per == 0:
            raise ValueError(f"STQ1_0 needs N >= 1 and K a multiple of 256 in 256..32768 (N={N}, K={K})")
        if blocks.numel() != E * N * (K // STQ1_BLOCK_WEIGHTS) * STQ1_BLOCK_BYTES:
            raise ValueError("blocks must hold E * N * K/256 blocks of 42 bytes")
        packed = _empty((E * per,), torch.uint8, blocks.device, stream)
        src = blocks.reshape(E, -1)
        for e in range(E):
            _raise(lib().stq1_pack(src[e].data_ptr(), packed.data_ptr() + e * per, N, K, _stream_ptr(stream)))
        return cls(packed, N, K, E)

    @classmethod
    def from_host(cls, blocks, N: int, K: int, E: int = 1, device="cuda") -> "STQ1Matrix":
        """From a numpy uint8 array of blocks (``synth.make_stq1``)."""
        return cls.from_blocks(torch.from_numpy(blocks.reshape(-1).copy()).to(device), N, K, E)

    @property
    def nbytes(self) -> int:
        """Bytes of the weights in the page's format (42 per 256 weights)."""
        return self.E * self.N * (self.K // STQ1_BLOCK_WEIGHTS) * STQ1_BLOCK_BYTES


def stq1_packed_bytes(N: int, K: int) -> int:
    return int(lib().stq1_packed_bytes(N, K))


def stq1_mm(x: torch.Tensor, w: STQ1Matrix, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[..., N] = x[..., K] W^T (float32) through ``stq1_mm``."""
    if w.E != 1:
        raise ValueError("stq1_mm takes a single matrix; use stq1_mm_id for stacked experts")
    _dev_tensor(x, torch.float32, "x")
    if x.shape[-1] != w.K:
        raise ValueError(f"x has K={x.shape[-1]}, weights have K={w.K}")
    M = x.numel() // w.K
    if out is None:
        out = _empty((*x.shape[:-1], w.N), torch.float32, x.device, stream)
    _dev_tensor(out, torch.float32, "out")
    if out.numel() != M * w.N:
        raise ValueError("out has the wrong number of elements")
    _raise(lib().stq1_mm(x.data_ptr(), w.packed.data_ptr(), out.data_ptr(), M, w.N, w.K, _stream_ptr(stream)))
    return out


def stq1_mm_id(x: torch.Tensor, w: STQ1Matrix, ids: torch.Tensor, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """y[t] = W[ids[t]] x[t] (float32) through ``stq1_mm_id``; x [T, K], ids int32 [T]."""
    _dev_tensor(x, torch.float32, "x")
    _dev_tensor(ids, torch.int32, "ids")
    if x.dim() != 2 or x.shape[1] != w.K:
        raise ValueError("x must be [T, K]")
    T = x.shape[0]
    if ids.numel() != T:
        raise ValueError("ids must hold one expert id per token")
    if out is None:
        out = _empty((T, w.N), torch.float32, x.device, stream)
    _dev_tensor(out, torch.float32, "out")
    _raise(lib().stq1_mm_id(x.data_ptr(), w.packed.data_ptr(), ids.data_ptr(), out.data_ptr(), T, w.N, w.K, w.E,
                            _stream_ptr(stream)))
    return out


def stq1_get_rows(ids: torch.Tensor, w: STQ1Matrix, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rows ids of W as float32 [..., K] through ``stq1_get_rows``."""
    if w.E != 1:
        raise ValueError("stq1_get_rows takes a single matrix")
    _dev_tensor(ids, torch.int32, "ids")
    T = ids.numel()
    if out is None:
        out = _empty((*ids.shape, w.K), torch.float32, ids.device, stream)
    _dev_tensor(out, torch.float32, "out")
    if out.numel() != T * w.K:
        raise ValueError("out has the wrong number of elements")
    _raise(lib().stq1_get_rows(w.packed.data_ptr(), ids.data_ptr(), out.data_ptr(), T, w.N, w.K,
                               _stream_ptr(stream)))
    return out


def stq1_get_plan(N: int, K: int) -> dict:
    p = Stq1Plan()
    _raise(lib().stq1_get_plan(N, K, ctypes.byref(p)))
    return {f: getattr(p, f) for f, _ in p._fields_}


# ---- paged key/value cache in 8 bits (include/w4a16.h "Paged key/value cache") --------------

KV_BLOCKS, KV_DIMS, KV_MAX_GROUP, KV_COUNTERS = (16, 32, 64, 128), (64, 128, 256), 32, 512


@dataclass(frozen=True)
class KVCache:
    """Keys and values of one layer: e4m3 codes ``k``, ``v`` (torch.float8_e4m3fn
    [blocks, heads, block, dim]) with one power-of-two scale per (block, head)
    ``k_scale``, ``v_scale`` (float32 [blocks, heads]).  ``kv_append`` fills
    blocks; their first contents do not matter (``empty`` leaves them unset)."""

    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    def __post_init__(self):
        for name in ("k", "v"):
            t = _dev_tensor(getattr(self, name), torch.float8_e4m3fn, name)
            if t.dim() != 4 or t.shape != self.k.shape:
                raise ValueError(f"{name} must be [blocks, heads, block, dim] (got {tuple(t.shape)})")
        for name, n in zip(("blocks", "heads", "block", "dim"), self.k.shape):
            object.__setattr__(self, name, n)
        if self.block not in KV_BLOCKS or self.dim not in KV_DIMS:
            raise ValueError(f"block {self.block} must be one of {KV_BLOCKS}, dim {self.dim} one of {KV_DIMS}")
        for name in ("k_scale", "v_scale"):
            t = _dev_tensor(getattr(self, name), torch.float32, name)
            if t.shape != (self.blocks, self.heads):
                raise ValueError(f"{name} must be [blocks, heads] (got {tuple(t.shape)})")
        if any(t.device != self.k.device for t in (self.v, self.k_scale, self.v_scale)):
            raise ValueError("the cache's tensors must be on one device")
        c = KvCacheStruct(self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(),
                          self.blocks, self.heads, self.block, self.dim)
        object.__setattr__(self, "_c", c)
        object.__setattr__(self, "_ptr", ctypes.addressof(c))
        object.__setattr__(self, "_dev", self.k.get_device())

    @classmethod
    def empty(cls, blocks: int, heads: int, block: int, dim: int, device="cuda") -> "KVCache":
        k, v = (torch.empty(blocks, heads, block, dim, dtype=torch.float8_e4m3fn, device=device) for _ in range(2))
        ks, vs = (torch.empty(blocks, heads, dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.k, self.v, self.k_scale, self.v_scale))


@dataclass
class KVPlan:
    """One step's rows (int32, on the device): ``cu`` [B + 1] first row of each
    request, ``lens`` [B] lengths after the step, ``slots`` and ``positions``
    [T], ``head`` [1] free-list entries taken so far."""

    cu: torch.Tensor
    lens: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor
    head: torch.Tensor

    @classmethod
    def empty(cls, B: int, T: int, device="cuda", stream=None) -> "KVPlan":
        """Unset; for a call on ``stream`` (None: the current one)."""
        flat = _empty((2 * B + 2 * T + 2,), torch.int32, device, stream)
        return cls(*torch.unsafe_split_with_sizes(flat, (B + 1, B, T, T, 1)))  # (whole numbers: nothing to differentiate)


def _on_device(t: torch.Tensor, name: str, dev: int) -> None:
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, other tensors of the call on cuda:{dev}")


def _i32(t: torch.Tensor, name: str, n: int | None = None, dev: int | None = None) -> int:
    """The address of a contiguous int32 CUDA tensor of n elements on device dev (None: any)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.is_cuda and t.is_contiguous()):
        _dev_tensor(t, torch.int32, name)
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} must have {n} elements (got {t.numel()})")
    if dev is not None and t.get_device() != dev:
        _on_device(t, name, dev)
    return t.data_ptr()


def _stream_on(stream, dev: int) -> int:
    """The stream of a call whose tensors are on device dev: the current device's, or one given."""
    if stream is None:
        if torch._C._cuda_getDevice() != dev:
            raise ValueError(f"the call's tensors are on cuda:{dev}, which is not the current device")
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev or torch._C._cuda_getDevice() != dev:
        raise ValueError(f"the call's tensors are on cuda:{dev}; the stream, or the current device, is another's")
    return stream.cuda_stream


def _kv_rows(t: torch.Tensor, name: str, heads: int, dim: int) -> int:
    """The token stride of a bf16 CUDA tensor [T, heads, dim] whose rows are dense
    (the tokens may be further apart: columns of a fused projection)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.is_cuda):
        raise ValueError(f"{name} must be a bfloat16 CUDA tensor")
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be [T, {heads}, {dim}] (got {tuple(shape)})")
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != dim and heads > 1):
        raise ValueError(f"{name}: each token's heads * dim values must be contiguous")
    return s0 if shape[0] > 1 else heads * dim


def kv_plan(cached: torch.Tensor, new: torch.Tensor, table: torch.Tensor, free: torch.Tensor, T: int, block: int,
            head: torch.Tensor | None = None, out: KVPlan | None = None, stream=None) -> KVPlan:
    """Block tables, slots and positions of a step through ``w4a16_kv_plan``.

    cached, new: int32 [B] tokens of each request in the cache and joining it;
    table: int32 [B, max_blocks], its entries for the new blocks written in
    place; free: int32 block ids to take from, beginning at entry ``head``
    (int32 [1] on the device; None is 0; the plan's ``head`` is the next one).
    T rows: the sum of ``new``, or more (the rest get slot -1).  ``out``: a plan
    to write; its arrays overlap nothing else, but its ``lens`` may be ``cached``
    (lengths advanced in place)."""
    tp = _i32(table, "table")
    if table.dim() != 2:
        raise ValueError("table must be [B, max_blocks]")
    B, max_blocks = table.shape
    dev = table.get_device()
    if out is None:
        if T < 0:
            raise ValueError("T must not be negative")
        out = KVPlan.empty(B, T, table.device, stream)
        cu = out.cu.data_ptr()  # the arrays lie one after another
        lens = cu + 4 * (B + 1)
        slots = lens + 4 * B
        outs = (cu, lens, slots, slots + 4 * T, slots + 8 * T)
    else:
        outs = (_i32(out.cu, "cu", B + 1, dev), _i32(out.lens, "lens", B, dev), _i32(out.slots, "slots", T, dev),
                _i32(out.positions, "positions", T, dev), _i32(out.head, "head_out", 1, dev))
    rc = lib().w4a16_kv_plan(_i32(cached, "cached", B, dev), _i32(new, "new", B, dev), tp, _i32(free, "free", None, dev),
                             None if head is None else _i32(head, "head", 1, dev), *outs, B, T, block, max_blocks,
                             free.numel(), _stream_on(stream, dev))
    if rc:
        _raise(rc)
    return out


def kv_append(k: torch.Tensor, v: torch.Tensor, cache: KVCache, slots: torch.Tensor, stream=None) -> None:
    """Write keys and values k, v (bf16 [T, heads, dim]; tokens may be strided)
    into ``slots`` (int32 [T], a plan's) of ``cache`` through ``w4a16_kv_append``."""
    ks, vs = _kv_rows(k, "k", cache.heads, cache.dim), _kv_rows(v, "v", cache.heads, cache.dim)
    T = k.shape[0]
    if v.shape[0] != T:
        raise ValueError("k and v must have the same number of tokens")
    dev = cache._dev
    _on_device(k, "k", dev)
    _on_device(v, "v", dev)
    rc = lib().w4a16_kv_append(k.data_ptr(), ks, v.data_ptr(), vs, _i32(slots, "slots", T, dev), cache._ptr, T,
                               _stream_on(stream, dev))
    if rc:
        _raise(rc)


KV_CAPTURE_SETS = 1024  # counters for captured calls, per device (2 MB)
_kv_counter_cache: dict = {}
_kv_capture_sets: dict = {}


def _kv_counters(raw_stream: int, device: torch.device):
    """(tensor, address) of zeroed counters of a call on the current stream: the stream's, kept here as
    its workspace is; for a captured call, whose graph may be replayed beside that
    stream, a set of its own.  Those are made with the device's first call outside
    capture and handed out once; without one left, the graph zeroes a set from its
    own memory."""
    key = (device.index, raw_stream)
    if _capturing():
        with _ws_lock:
            sets = _kv_capture_sets.get(device.index)
            if sets is not None and sets[1] < KV_CAPTURE_SETS:
                sets[1] += 1
                return sets[0], sets[0].data_ptr() + 4 * KV_COUNTERS * (sets[1] - 1)
        t = torch.zeros(KV_COUNTERS, dtype=torch.int32, device=device)
        return t, t.data_ptr()
    c = _kv_counter_cache.get(key)
    if c is None:
        zeros = torch.zeros(KV_COUNTERS, dtype=torch.int32, device=device)
        with _ws_lock:
            if device.index not in _kv_capture_sets:
                _kv_capture_sets[device.index] = [torch.zeros(KV_CAPTURE_SETS * KV_COUNTERS, dtype=torch.int32, device=device), 0]
            torch.cuda.current_stream(device).synchronize()
            c = _kv_counter_cache.setdefault(key, (zeros, zeros.data_ptr()))
    return c


def _kv_reset_counters(dev: int) -> None:
    """After a wait ran out on device dev, the current one: a call there may have left counters behind.  Other
    devices' calls may be running; their counters are as they should be."""
    torch.cuda.synchronize()
    for t in [c[0] for key, c in _kv_counter_cache.items() if key[0] == dev] + [s[0] for i, s in _kv_capture_sets.items() if i == dev]:
        t.zero_()
    torch.cuda.synchronize()


KV_WORKSPACE_KEPT = 64 << 20  # larger workspaces are not kept between calls
_kv_ws_cache: dict = {}


def _kv_workspace(n: int, raw_stream: int, device: torch.device):
    """(tensor, address) of n bytes for a call on the current stream: the stream's
    own, kept here and grown when a call needs more, or (large, or under graph
    capture) one for this call, whose memory comes back in the stream's order.  It
    needs no initial contents."""
    key = (device.index, raw_stream)
    kept = _kv_ws_cache.get(key)
    if kept is not None and kept[2] >= n and not _capturing():
        return kept
    t = torch.empty(n, dtype=torch.uint8, device=device)
    kept = (t, t.data_ptr(), n)
    if n <= KV_WORKSPACE_KEPT and not _capturing():
        _kv_ws_cache[key] = kept
    return kept


@functools.lru_cache(maxsize=1024)
def _kv_attention_bytes(*sizes: int) -> int:
    return int(lib().w4a16_kv_attention_workspace_bytes(*sizes))


def kv_attention_workspace_bytes(B: int, T: int, q_heads: int, cache: KVCache, max_new: int, max_len: int,
                                 window: int = 0) -> int:
    return _kv_attention_bytes(B, T, q_heads, cache.heads, cache.dim, max_new, max_len, window)


def kv_attention(q: torch.Tensor, cache: KVCache, table: torch.Tensor, cu: torch.Tensor, lens: torch.Tensor,
                 max_new: int, max_len: int, scale: float | None = None, window: int = 0,
                 out: torch.Tensor | None = None, stream=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Causal attention of q (bf16 [T, q_heads, dim]; tokens may be strided) over
    ``cache`` through ``w4a16_kv_attention``: bf16 [T, q_heads, dim].

    table, cu, lens: a plan's; max_new, max_len: the caller's bounds on the
    requests' new tokens and lengths; scale: 1 / sqrt(dim) by default; window:
    tokens that a row sees, itself included (0: all).  The workspace is this
    stream's, kept by this module, unless one (uint8) is given."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [T, q_heads, dim]")
    T, hq, dim = q.shape
    qs = _kv_rows(q, "q", hq, cache.dim)
    tp = _i32(table, "table")
    if table.dim() != 2:
        raise ValueError("table must be [B, max_blocks]")
    B, max_blocks = table.shape
    dev, di = q.device, cache._dev
    _on_device(q, "q", di)
    _on_device(table, "table", di)
    cup, lp = _i32(cu, "cu", B + 1, di), _i32(lens, "lens", B, di)
    raw = _stream_on(stream, di)
    if out is None:
        out = _empty((T, hq, dim), torch.bfloat16, dev, stream)
    else:
        _dev_tensor(out, torch.bfloat16, "out")
        _on_device(out, "out", di)
        if out.shape != q.shape:
            raise ValueError(f"out must be {tuple(q.shape)}")
    wn = _kv_attention_bytes(B, T, hq, cache.heads, dim, max_new, max_len, window) if workspace is None else 0
    with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):  # the call's stream is the current one
        counters, cp = _kv_counters(raw, dev)  # (both tensors are held until the launch: neither may get the other's memory)
        if wn:
            workspace, wp, _ = _kv_workspace(wn, raw, dev)
        else:
            wp, wn = _ws_args(workspace)
    if workspace is not None:
        _on_device(workspace, "workspace", di)
    rc = lib().w4a16_kv_attention(q.data_ptr(), qs, cache._ptr, tp, cup, lp,
                                  out.data_ptr(), B, T, hq, max_blocks, max_new, max_len, window,
                                  1.0 / math.sqrt(dim) if scale is None else scale, wp, wn, cp, raw)
    if rc:
        _raise(rc)
    return out


# ---- microscaled 4-bit floating point (include/w4a16.h "Microscaled 4-bit floating point") ----

FP4_FORMATS, FP4_BLOCK = {"nv": 1, "mx": 2}, {"nv": 16, "mx": 32}
FP4_ACTS = {None: 0, "silu": 1, "gelu": 2}


def fp4_scale_bytes(N: int, K: int, format: str) -> int:
    """Bytes of the scales of one expert's N rows of K codes."""
    if format not in FP4_FORMATS:
        raise ValueError(f"unknown format {format!r}; one of {sorted(FP4_FORMATS)}")
    b = 4 * FP4_BLOCK[format]
    return -(-N // 128) * -(-K // b) * 512


class FP4Matrix:
    """A matrix of e2m1 codes with block scales on the GPU: ``codes`` uint8 [E * N, K / 2],
    two a byte, low nibble first; ``scales`` uint8 [E * fp4_scale_bytes(N, K, format)], in
    the order of include/w4a16.h; ``row_scale`` float32 [E * N] (format "nv"; None: 1).

    ``fp4_quant`` makes one from bf16 rows, ``gated`` from gate and up rows of a
    feed-forward block, ``from_rows`` from scales in row order (a checkpoint's)."""

    __slots__ = ("N", "K", "E", "format", "_codes", "_scales", "_row_scale", "_flat", "_c", "_ptr", "_dev", "_device")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, row_scale: torch.Tensor | None, N: int, K: int,
                 E: int = 1, format: str = "nv"):
        n = fp4_scale_bytes(N, K, format)
        if K <= 0 or K % 32 or N < 0 or E < 1:
            raise ValueError(f"N = {N}, K = {K} (a positive multiple of 32), E = {E}")
        dev = _dev_tensor(codes, torch.uint8, "codes").get_device()
        _dev_tensor(scales, torch.uint8, "scales")
        if codes.numel() != E * N * (K // 2):
            raise ValueError(f"codes must hold E * N * K / 2 = {E * N * (K // 2)} bytes")
        if scales.numel() != E * n:
            raise ValueError(f"scales must hold E * fp4_scale_bytes = {E * n} bytes")
        _on_device(scales, "scales", dev)
        if row_scale is not None:
            _dev_tensor(row_scale, torch.float32, "row_scale")
            if row_scale.numel() != E * N:
                raise ValueError("row_scale must have one factor per row")
            _on_device(row_scale, "row_scale", dev)
        self.N, self.K, self.E, self.format = N, K, E, format
        self._codes, self._scales, self._row_scale, self._flat = codes, scales, row_scale, None
        self._device, self._dev = codes.device, dev
        self._c = Fp4Struct(codes.data_ptr(), scales.data_ptr(), None if row_scale is None else row_scale.data_ptr(), N, K, E,
                            FP4_FORMATS[format])
        self._ptr = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, N: int, K: int, E: int = 1, format: str = "nv", device="cuda", stream=None) -> "FP4Matrix":
        """Unset; for a call on ``stream`` (None: the current one)."""
        n = E * fp4_scale_bytes(N, K, format)
        if K <= 0 or K % 32 or N < 0 or E < 1:
            raise ValueError(f"N = {N}, K = {K} (a positive multiple of 32), E = {E}")
        # scales (a multiple of 512 bytes) and codes in one block of memory; their tensors are made when asked for
        flat = _empty((n + E * N * (K // 2),), torch.uint8, device, stream)
        f = _empty((E * N,), torch.float32, device, stream) if format == "nv" else None
        self, at = cls.__new__(cls), flat.data_ptr()
        self.N, self.K, self.E, self.format = N, K, E, format
        self._flat, self._codes, self._scales, self._row_scale = flat, None, None, f
        self._device, self._dev = flat.device, flat.get_device()
        self._c = Fp4Struct(at + n, at, None if f is None else f.data_ptr(), N, K, E, FP4_FORMATS[format])
        self._ptr = ctypes.addressof(self._c)
        return self

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            self._scales = self._flat[:self.E * fp4_scale_bytes(self.N, self.K, self.format)]
        return self._scales

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            n = self.E * fp4_scale_bytes(self.N, self.K, self.format)
            self._codes = self._flat[n:].view(self.E * self.N, self.K // 2)
        return self._codes

    @property
    def row_scale(self) -> torch.Tensor | None:
        return self._row_scale

    @classmethod
    def gated(cls, gate: torch.Tensor, up: torch.Tensor, format: str = "nv", stream=None) -> "FP4Matrix":
        """Gate and up weights (bf16 [F, K], or [E, F, K]) quantised into the one matrix of
        2 F rows that ``fp4_gated`` takes: row 2 i is gate's row i, row 2 i + 1 up's."""
        if gate.shape != up.shape or gate.dim() not in (2, 3):
            raise ValueError("gate and up must both be [F, K] or [E, F, K]")
        if stream is None:
            return fp4_quant(torch.stack((gate, up), -2).flatten(-3, -2), format)
        _stream_on(stream, gate.get_device())
        with torch.cuda.stream(stream):  # the interleaved rows are the call's own: made, read and given back in its order
            both = torch.stack((gate, up), -2).flatten(-3, -2)
        return fp4_quant(both, format, stream=stream)

    @classmethod
    def from_rows(cls, codes: torch.Tensor, scales: torch.Tensor, row_scale: torch.Tensor | float | None = None,
                  format: str = "nv") -> "FP4Matrix":
        """From codes uint8 [N, K / 2] or [E, N, K / 2] and scale bytes uint8 [.., N, K / block]
        in row order; row_scale [.., N], or one number (of Python, or a tensor of one) for all rows."""
        E, N, K = (1 if codes.dim() == 2 else codes.shape[0]), codes.shape[-2], 2 * codes.shape[-1]
        fp4_scale_bytes(N, K, format)
        nb = K // FP4_BLOCK[format]
        if tuple(scales.shape) != tuple(codes.shape[:-1]) + (nb,) or scales.dtype is not torch.uint8:
            raise ValueError(f"scales must be uint8 {tuple(codes.shape[:-1]) + (nb,)}")
        rows, cols = -(-N // 128) * 128, -(-nb // 4) * 4
        full = torch.zeros(E, rows, cols, dtype=torch.uint8, device=scales.device)
        full[:, :N, :nb] = scales.view(E, N, nb)
        tiled = full.view(E, rows // 128, 4, 32, cols // 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(-1).contiguous()
        if row_scale is not None:
            row_scale = torch.as_tensor(row_scale, dtype=torch.float32, device=codes.device).expand(codes.shape[:-1]).reshape(-1).contiguous()
        return cls(codes.reshape(E * N, K // 2), tiled, row_scale, N, K, E, format)

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.codes, self.scales, self.row_scale) if t is not None)

    def __repr__(self) -> str:
        return f"FP4Matrix(N={self.N}, K={self.K}, E={self.E}, format={self.format!r}, device={self._device})"


def _fp4_x(x: torch.Tensor, K: int, dev: int | None):
    """(rows, row stride) of bf16 activations [.., K]: dense rows, which may be apart where x is [M, K]."""
    if not (isinstance(x, torch.Tensor) and x.dtype is torch.bfloat16 and x.is_cuda):
        _dev_tensor(x, torch.bfloat16, "x")
    shape = x.shape
    if not shape or shape[-1] != K:
        raise ValueError(f"x must be [.., {K}] (got {tuple(shape)})")
    if dev is not None and x.get_device() != dev:
        _on_device(x, "x", dev)
    if x.is_contiguous():
        return shape[0] if len(shape) == 2 else x.numel() // K, K
    if len(shape) != 2 or x.stride(1) != 1:
        raise ValueError("x must be contiguous, or [M, K] with contiguous rows")
    return shape[0], x.stride(0) if shape[0] > 1 else K


def fp4_quant(x: torch.Tensor, format: str = "nv", out: FP4Matrix | None = None, stream=None) -> FP4Matrix:
    """Rows of x (bf16 [.., K]; [M, K] rows may be strided) as e2m1 codes and block scales
    through ``w4a16_fp4_quant``.  A contiguous [E, N, K] is E experts of N rows."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1 or format not in FP4_FORMATS:
        raise ValueError(f"x must be a tensor [.., K], format one of {sorted(FP4_FORMATS)}")
    K = x.shape[-1]
    if K <= 0 or K % 32:
        raise ValueError(f"K = {K} must be a positive multiple of 32")
    M, stride = _fp4_x(x, K, None)
    dev = x.get_device()
    raw = _stream_on(stream, dev)
    if out is None:
        E = max(x.shape[0], 1) if x.dim() == 3 else 1
        out = FP4Matrix.empty(M // E, K, E, format, x.device, stream)
    elif (out.N * out.E, out.K, out.format) != (M, K, format):
        raise ValueError(f"out must have {M} rows of {K} codes, format {format}")
    elif out._dev != dev:
        raise ValueError(f"out is on cuda:{out._dev}, x on cuda:{dev}")
    rc = (_lib or lib()).w4a16_fp4_quant(x.data_ptr(), stride, out._ptr, raw)
    if rc:
        _raise(rc)
    return out


def fp4_dequant(w: FP4Matrix, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values of w as bf16 [N, K] (or [E, N, K]) through ``w4a16_fp4_dequant``."""
    shape = (w.N, w.K) if w.E == 1 else (w.E, w.N, w.K)
    raw = _stream_on(stream, w._dev)
    if out is None:
        out = _empty(shape, torch.bfloat16, w._device, stream)
    else:
        _fp4_out(out, shape, w._dev)
    rc = (_lib or lib()).w4a16_fp4_dequant(w._ptr, out.data_ptr(), raw)
    if rc:
        _raise(rc)
    return out


def _fp4_out(out: torch.Tensor, shape, dev: int) -> None:
    _dev_tensor(out, torch.bfloat16, "out")
    _on_device(out, "out", dev)
    if out.numel() != math.prod(shape):
        raise ValueError(f"out must be {tuple(shape)}")


@functools.lru_cache(maxsize=1024)
def _fp4_mm_bytes(M: int, K: int, format: int) -> int:
    return int((_lib or lib()).w4a16_fp4_mm_workspace_bytes(M, K, format))


@functools.lru_cache(maxsize=1024)
def _fp4_mm_id_bytes(*sizes: int) -> int:
    return int((_lib or lib()).w4a16_fp4_mm_id_workspace_bytes(*sizes))


def _fp4_act(w: FP4Matrix, act) -> int:
    if act is None:
        return 0
    if act not in FP4_ACTS:
        raise ValueError(f"unknown activation {act!r}; one of {list(FP4_ACTS)}")
    if w.N % 2:
        raise ValueError(f"N = {w.N}: gate and up rows come in pairs")
    return FP4_ACTS[act]


def _fp4_space(need: int, workspace, raw: int, stream, w: FP4Matrix):
    """(tensor, address, bytes) of a call's workspace: the stream's own, or the given one."""
    if workspace is not None:
        _on_device(workspace, "workspace", w._dev)
        return (workspace, *_ws_args(workspace))
    if stream is None:
        return _kv_workspace(need, raw, w._device)
    with torch.cuda.stream(stream):  # the call's stream is the current one
        return _kv_workspace(need, raw, w._device)


def _fp4_product(x, w: FP4Matrix, act, out, stream, workspace):
    if w.E != 1:
        raise ValueError("stacked experts: use fp4_mm_id")
    a = _fp4_act(w, act)
    cols = w.N if a == 0 else w.N // 2
    dev = w._dev
    raw = _stream_on(stream, dev)
    quantised = isinstance(x, FP4Matrix)
    if quantised:
        M = x.N
        lead = (M,)
        if x.K != w.K or x.format != w.format or x.E != 1:
            raise ValueError(f"x has K={x.K}, format {x.format}, E={x.E}; weights have K={w.K}, format {w.format}")
        if x._dev != dev:
            raise ValueError(f"x is on cuda:{x._dev}, w on cuda:{dev}")
    else:
        M, stride = _fp4_x(x, w.K, dev)
        lead = x.shape[:-1]
    if out is None:
        out = _empty((*lead, cols), torch.bfloat16, w._device, stream)
    else:
        _fp4_out(out, (M, cols), dev)
    if quantised:
        rc = (_lib or lib()).w4a16_fp4_mm_q(x._ptr, w._ptr, out.data_ptr(), a, raw)
    else:
        keep, ws, wn = _fp4_space(_fp4_mm_bytes(M, w.K, FP4_FORMATS[w.format]), workspace, raw, stream, w)
        rc = (_lib or lib()).w4a16_fp4_mm(x.data_ptr(), stride, w._ptr, out.data_ptr(), M, a, ws, wn, raw)
    if rc:
        _raise(rc)
    return out


def fp4_mm(x, w: FP4Matrix, out: torch.Tensor | None = None, stream=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[.., N] = x'[.., K] W^T in bf16 through ``w4a16_fp4_mm``: x bf16 (leading dims
    flatten into rows; [M, K] rows may be strided), quantised row by row in w's format;
    or an ``FP4Matrix`` already (``w4a16_fp4_mm_q``).  The workspace is this stream's,
    kept by this module, unless one (uint8) is given."""
    return _fp4_product(x, w, None, out, stream, workspace)


def fp4_gated(x, w: FP4Matrix, act: str = "silu", out: torch.Tensor | None = None, stream=None,
              workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The first half of a gated feed-forward block: act(x' G^T) * (x' U^T), bf16 [.., N / 2],
    over the interleaved rows of ``FP4Matrix.gated``; act "silu" or "gelu" (tanh form)."""
    if act is None:
        raise ValueError("fp4_gated needs an activation; fp4_mm has none")
    return _fp4_product(x, w, act, out, stream, workspace)


def fp4_mm_id(x: torch.Tensor, w: FP4Matrix, ids: torch.Tensor, act: str | None = None, out: torch.Tensor | None = None,
              stream=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[t, j] = W[ids[t, j]] x'[t] through ``w4a16_fp4_mm_id``: x bf16 [T, K], ids int32 [T, top]
    (or [T]), y bf16 [T, top, N] (or [T, N]); with an ``act``, the gated form of each
    expert, [.., N / 2].  An id outside 0..E-1 gives a row of zeros and raises DEVICE_BAD_ID."""
    a = _fp4_act(w, act)
    T, stride = _fp4_x(x, w.K, w._dev)
    if x.dim() != 2:
        raise ValueError("x must be [T, K]")
    ip = _i32(ids, "ids", None, w._dev)
    if ids.dim() not in (1, 2) or ids.shape[0] != T or ids.dim() == 2 and ids.shape[1] < 1:
        raise ValueError(f"ids must be [{T}, top] or [{T}]")
    top = ids.shape[1] if ids.dim() == 2 else 1
    shape = (*ids.shape, w.N if a == 0 else w.N // 2)
    raw = _stream_on(stream, w._dev)
    if out is None:
        out = _empty(shape, torch.bfloat16, w._device, stream)
    else:
        _fp4_out(out, shape, w._dev)
    keep, ws, wn = _fp4_space(_fp4_mm_id_bytes(T, top, w.K, w.E, FP4_FORMATS[w.format]), workspace, raw, stream, w)
    rc = (_lib or lib()).w4a16_fp4_mm_id(x.data_ptr(), stride, w._ptr, ip, out.data_ptr(), T, top, a, ws, wn, raw)
    if rc:
        _raise(rc)
    return out


def version() -> str:
    return lib().w4a16_version().decode()
