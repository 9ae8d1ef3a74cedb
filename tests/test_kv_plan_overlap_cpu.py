"""w4a16_kv_plan refuses arrays that overlap what it writes (no GPU: the addresses are never dereferenced)."""
import pytest

from skinny_gemm_gb300 import ops

B, T, WIDE, FREE = 3, 5, 4, 9
SIZES = dict(cached=B, fresh=B, table=B * WIDE, free=FREE, head=1, cu=B + 1, lens=B, slots=T, positions=T, head_out=1)
WRITTEN = ("table", "cu", "lens", "slots", "positions", "head_out")


@pytest.fixture()
def L(monkeypatch):
    monkeypatch.delenv("W4A16_FAULT", raising=False)
    lib = ops.lib()
    lib.w4a16_debug_reload_env()
    return lib


def _places():
    """Disjoint addresses, one array right behind another."""
    at, out = 0x10000, {}
    for name, n in SIZES.items():
        out[name] = at
        at += 4 * n
    return out


def _refused(L, places):
    """True where the call refuses an overlap (without a GPU it fails later, with another code, where it does not)."""
    rc = L.w4a16_kv_plan(*(places[n] for n in SIZES), B, T, 16, WIDE, FREE, None)
    said = L.w4a16_last_error().decode()
    return rc == ops.ERR_SHAPE and ("overlap" in said or "head_out must not be head" in said)


@pytest.fixture(autouse=True)
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake addresses")


def test_neighbours_are_fine(L):
    assert not _refused(L, _places())


@pytest.mark.parametrize("one", WRITTEN)
@pytest.mark.parametrize("two", list(SIZES))
def test_overlaps(L, one, two):
    if one == two:
        return
    for shift in (0, 4 * (SIZES[two] - 1), -4 * (SIZES[one] - 1)):  # the same place, the last element, the first
        p = _places()
        p[two] = 0x80000
        p[one] = p[two] + shift
        in_place = (one, two) in (("lens", "cached"), ("cached", "lens")) and shift == 0
        assert _refused(L, p) != in_place, (one, two, shift)
    for shift in (4 * SIZES[two], -4 * SIZES[one]):
        p = _places()
        p[two] = 0x80000
        p[one] = p[two] + shift
        assert not _refused(L, p), (one, two, shift)


def test_no_requests(L):
    """Empty arrays overlap nothing."""
    p = _places()
    p["cached"] = p["fresh"] = p["table"] = p["lens"] = p["slots"]
    rc = L.w4a16_kv_plan(*(p[n] for n in SIZES), 0, T, 16, WIDE, FREE, None)
    assert rc != ops.ERR_SHAPE
