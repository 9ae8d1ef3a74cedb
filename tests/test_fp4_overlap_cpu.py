"""Memory that a microscaled 4-bit product would write while it still reads it is refused (no GPU: nothing is launched)."""
import pytest

from skinny_gemm_gb300 import ops
from test_fp4_cpu import L, err, matrix, ref  # noqa: F401  (fixture)

W, X, IDS, Y, WS = (i << 30 for i in range(1, 6))  # stand-in addresses, apart


@pytest.fixture()
def launches(L, monkeypatch):  # noqa: F811
    """Calls that pass all checks fail at their launch."""
    monkeypatch.setenv("W4A16_FAULT", "launch")
    L.w4a16_debug_reload_env()
    yield L
    monkeypatch.delenv("W4A16_FAULT")
    L.w4a16_debug_reload_env()


def weights(experts=1):
    return matrix(experts=experts, codes=W, scales=W + (1 << 20), row_scale=W + (1 << 21))


@pytest.mark.parametrize("act", [0, 1])
def test_mm_id(launches, act):
    T, top, N, K = 6, 3, 128, 256
    need = launches.w4a16_fp4_mm_id_workspace_bytes(T, top, K, 4, 1)
    y_bytes = 2 * T * top * (N // 2 if act else N)

    def call(ids=IDS, y=Y, ws=WS, x=X):
        return launches.w4a16_fp4_mm_id(x, K, ref(weights(4)), ids, y, T, top, act, ws, need, None)

    assert call() == ops.ERR_CUDA
    for at in (0, y_bytes - 4, 4 - 4 * T * top):
        assert call(ids=Y + at) == ops.ERR_SHAPE and "y overlaps ids" in err(launches)
    for at in (y_bytes, -4 * T * top):
        assert call(ids=Y + at) == ops.ERR_CUDA
    for at in (0, need - 2, 2 - y_bytes):
        assert call(y=WS + at) == ops.ERR_SHAPE and "y overlaps the workspace" in err(launches)
    assert call(y=WS + need) == call(y=WS - y_bytes) == ops.ERR_CUDA
    for at in (0, need - 16, 16 - 2 * T * K):
        assert call(x=WS + at) == ops.ERR_SHAPE and "x overlaps the workspace" in err(launches)
    assert call(x=WS - 2 * T * K) == ops.ERR_CUDA


@pytest.mark.parametrize("M", [1, 40, 300])
def test_mm(launches, M):
    N, K = 128, 256
    need = launches.w4a16_fp4_mm_workspace_bytes(M, K, 1)

    def call(y=Y, ws=WS, x=X, stride=K):
        return launches.w4a16_fp4_mm(x, stride, ref(weights()), y, M, 0, ws, need, None)

    assert call() == ops.ERR_CUDA
    for at in (0, need - 2, 2 - 2 * M * N):
        assert call(y=WS + at) == ops.ERR_SHAPE and "y overlaps the workspace" in err(launches)
    assert call(y=WS + need) == call(y=WS - 2 * M * N) == ops.ERR_CUDA
    for at in (0, need - 16, 16 - 2 * M * K):
        assert call(x=WS + at) == ops.ERR_SHAPE and "x overlaps the workspace" in err(launches)
    assert call(x=WS - 2 * M * K) == ops.ERR_CUDA
    if M > 1:  # rows that are further apart reach further
        assert call(x=WS - 2 * M * K, stride=2 * K) == ops.ERR_SHAPE
