"""The line of tiles of the paged attention (csrc/kv_line.cuh), built for the host: whole numbers against plain loops."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "skinny_gemm_gb300", "csrc")
SOURCE = r"""
#include "kv_line.cuh"
using namespace w4a16;
extern "C" int tiles(int TQ, int window, int base, int fresh, int rt) {
  Line p{};
  p.TQ = TQ;
  p.window = window;
  return tiles_before(p, Req{0, fresh, base}, rt);
}
// Row tiles of a step's accepted requests; -1: refused.
extern "C" long long row_tiles_of(const int* cu, const int* lens, int B, int T, int TQ, int max_new, int max_len) {
  Line p{cu, lens, B, TQ, T, 0, T, max_new, max_len, 0};
  long long n = 0;
  bool bad = false, back = false;
  for (int b = 0; b < B; ++b) {
    back |= steps_back(RawReq(p, b));
    n += row_tiles(p, load_req(p, b, &bad));
  }
  return back ? -1 : n;
}
// The rows t0 .. t0 + n - 1 of a step: each row's position, -1 where no request has it, -2 where two have it.
extern "C" void positions(const int* cu, const int* lens, int B, int all, int t0, int n, int max_new, int max_len, int* pos) {
  Line p{cu, lens, B, 1, all, t0, n, max_new, max_len, 0};
  bool bad = false;
  for (int t = 0; t < n; ++t) pos[t] = -1;
  for (int b = 0; b < B; ++b) {
    const Req r = load_req(p, b, &bad);
    for (int j = 0; j < r.fresh; ++j) pos[r.c0 + j] = pos[r.c0 + j] == -1 ? r.base + j : -2;
  }
}
extern "C" long long most(int B, int T, int TQ, int max_new) { return most_row_tiles(B, T, TQ, max_new); }
"""
TOP = 2 ** 31 - 1


@pytest.fixture(scope="module")
def line(tmp_path_factory):
    d = tmp_path_factory.mktemp("line")
    src, lib = d / "line.cpp", d / "line.so"
    src.write_text(SOURCE)
    # (-fwrapv: an overflow gives what the device gives)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    L = ctypes.CDLL(str(lib))
    for f in (L.row_tiles_of, L.most):
        f.restype = ctypes.c_longlong
    return L


def _tiles(TQ, window, base, fresh, rt):
    """Tiles of the row tiles before rt: from the first token that their first row sees to their last row's own."""
    n = 0
    for i in range(rt):
        last = base + min((i + 1) * TQ, fresh) - 1
        first = max(0, base + i * TQ - window + 1) if window else 0
        n += last // 128 - first // 128 + 1
    return n


def _check(line, TQ, window, base, fresh):
    n = -(-fresh // TQ)
    for rt in sorted({0, 1, 2, n // 3, n // 2, n - 1, n} & set(range(n + 1))):
        assert line.tiles(TQ, window, base, fresh, rt) == _tiles(TQ, window, base, fresh, rt), (TQ, window, base, fresh, rt)


@pytest.mark.parametrize("TQ", [1, 2, 3, 4, 5, 6, 8, 12, 24, 32])
def test_tiles_before(line, TQ):
    r = np.random.RandomState(TQ)
    for _ in range(200):
        fresh = int(r.randint(1, 700))
        base = int(r.choice([0, 1, 127, 128, int(r.randint(0, 5000))]))
        window = int(r.choice([0, 1, 2, 100, 128, 129, int(r.randint(1, 6000)), 10 ** 9]))
        _check(line, TQ, window, base, fresh)


@pytest.mark.parametrize("TQ", [1, 8, 32])
@pytest.mark.parametrize("window", [TOP, TOP - 1, TOP - 7, TOP - 8, TOP - 31, TOP - 40, 2 ** 30])
def test_windows_up_to_the_largest_number(line, TQ, window):
    """A window near 2^31 ("no limit"), from an empty cache on and near the longest request (within 2^31 tiles, as the
    call checks)."""
    for base, fresh in ((0, 300), (0, 9), (1, 64), (5, 700), (TQ, 300), (TOP - 400, 3 * TQ), (TOP - 3 * TQ, 3 * TQ)):
        _check(line, TQ, window, base, fresh)


def _row_tiles(line, cu, lens, T, TQ, max_new, max_len):
    a, b = ((ctypes.c_int * len(x))(*x) for x in (cu, lens))
    return line.row_tiles_of(a, b, len(lens), T, TQ, max_new, max_len)


def test_no_step_has_more_row_tiles_than_its_arrays_are_made_for(line):
    """Any offsets: requests accepted by themselves, bounds that do not hold, offsets out of range or stepping back."""
    r = np.random.RandomState(1)
    for _ in range(4000):
        B, T, TQ = int(r.randint(1, 40)), int(r.randint(1, 50)), int(r.choice([1, 2, 3, 8, 32]))
        max_new, max_len = int(r.randint(1, 20)), 100
        cu = np.sort(r.randint(-3, T + 4, B + 1)) if r.rand() < 0.6 else r.randint(-3, T + 4, B + 1)
        lens = r.randint(-2, 110, B)
        n = _row_tiles(line, [int(x) for x in cu], [int(x) for x in lens], T, TQ, max_new, max_len)
        assert n <= line.most(B, T, TQ, min(max_new, T)), (cu, lens, T, TQ, max_new)
        assert (n == -1) == bool(np.any(np.diff(cu) < 0))
    assert _row_tiles(line, [0, 1, 0, 1, 0, 1], [1024] * 5, 1, 4, 1, 1024) == -1
    assert _row_tiles(line, [0, 2] * 11, [384] * 21, 2, 8, 2, 384) == -1


def test_a_launch_of_some_of_the_rows(line):
    """Rows keep their positions however the call's rows are divided over launches."""
    r = np.random.RandomState(2)
    for _ in range(500):
        B = int(r.randint(1, 12))
        cu = np.concatenate([[0], np.cumsum(r.randint(0, 9, B))])
        T = int(cu[-1] + r.randint(0, 4))
        lens = np.diff(cu) + r.randint(-1, 200, B)
        max_new, max_len = int(r.randint(1, 10)), 150
        want = [-1] * T
        for b in range(B):
            n = int(cu[b + 1] - cu[b])
            if n <= min(max_new, lens[b]) and lens[b] <= max_len:
                want[cu[b]:cu[b + 1]] = range(lens[b] - n, lens[b])
        per = int(r.randint(1, T + 2))
        got, a, b = [], *((ctypes.c_int * len(x))(*(int(v) for v in x)) for x in (cu, lens))
        for t0 in range(0, T, per):
            n = min(per, T - t0)
            pos = (ctypes.c_int * n)()
            line.positions(a, b, B, T, t0, n, max_new, max_len, pos)
            got += list(pos)
        assert got == want
