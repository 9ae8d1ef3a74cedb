// kv_line.cuh -- the line of tiles that kv_attention.cu cuts over its CTAs: which
// requests take part, their row tiles and the tiles of those.  Whole numbers
// only, the same on the device and on the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define KV_LINE_FN __host__ __device__
#define KV_LINE KV_LINE_FN __forceinline__
#define KV_LINE_CALL KV_LINE_FN __noinline__
#else
#include <algorithm>
#define KV_LINE_FN
#define KV_LINE inline
#define KV_LINE_CALL inline
#endif

namespace w4a16 {

#ifndef __CUDACC__
using std::max;
using std::min;
#endif

constexpr int kTile = 128;  // tokens per tile (the M of the MMAs)

struct Line {
  const int32_t* cu;
  const int32_t* lens;
  int B, TQ;   // TQ tokens per row tile
  int all;     // rows of the call
  int t0, T;   // this launch's rows: the first, and how many
  int max_new, max_len, window;
};

// A request's part of the launch: its row tiles and their ranges of 128-token
// tiles.  (Rows of a request do not depend on one another, so a part is a request
// with fewer new tokens.)
struct Req {
  int c0, fresh, base;  // first row from t0 on, new tokens (0: nothing to do), tokens before them
};

struct RawReq {
  int c0, c1, len;
  KV_LINE RawReq(const Line& p, int b) : c0(0), c1(0), len(0) {
    if (b < p.B) c0 = p.cu[b], c1 = p.cu[b + 1], len = p.lens[b];
  }
};

KV_LINE Req check_req(const Line& p, const RawReq& w, bool* bad) {
  Req r{0, 0, 0};
  const int c0 = w.c0, c1 = w.c1, len = w.len;
  const bool ok = c0 >= 0 && c0 <= c1 && c1 <= p.all && c1 - c0 <= p.max_new && c1 - c0 <= len && len <= p.max_len;
  if (!ok) {
    if (c1 != c0) *bad = true;
    return r;
  }
  const int a = max(c0, p.t0), e = min(c1, p.t0 + p.T);
  if (a < e) r = Req{a - p.t0, e - a, len - (c1 - a)};
  return r;
}

// Offsets that step back anywhere make requests overlap, each of them valid by
// itself, and a line longer than the call's arrays are made for: such a step is
// refused as a whole.
KV_LINE bool steps_back(const RawReq& w) { return w.c1 < w.c0; }

// The most row tiles of a step whose offsets do not step back.
inline int64_t most_row_tiles(int B, int T, int TQ, int max_new) {
  const int64_t reqs = T < B ? T : B, each = reqs * (((int64_t)max_new + TQ - 1) / TQ), by_rows = reqs + (int64_t)T / TQ;
  return by_rows < each ? by_rows : each;
}

KV_LINE Req load_req(const Line& p, int b, bool* bad) { return check_req(p, RawReq(p, b), bad); }

KV_LINE int row_tiles(const Line& p, const Req& r) {
  return r.fresh <= p.TQ ? (r.fresh > 0) : (r.fresh + p.TQ - 1) / p.TQ;
}
KV_LINE int first_tile(const Line& p, const Req& r, int rt) {
  return p.window > 0 ? max(0, r.base + rt * p.TQ - p.window + 1) / kTile : 0;
}
KV_LINE int last_tile(const Line& p, const Req& r, int rt) {
  return (r.base + min((rt + 1) * p.TQ, r.fresh) - 1) / kTile;
}

// sum over 0 <= i < n of floor((b + i a) / m), for sums below 2^32: whole
// parts are taken out, then the lattice points under the line are counted
// along the other axis, as in Euclid's algorithm (Graham, Knuth and Patashnik,
// Concrete Mathematics, section 3.5, has such floor sums).
KV_LINE_CALL uint32_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  uint32_t s = 0;
  while (n > 0) {
    const uint32_t qa = a / m, qb = b / m;
    if (qa) s += (uint32_t)((uint64_t)n * (n - 1) / 2) * qa;
    s += n * qb;
    a -= qa * m;
    b -= qb * m;
    const uint32_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y - n * m;
    const uint32_t t = a;
    a = m;
    m = t;
  }
  return s;
}

// Tiles of the row tiles before rt (of one key head).
inline KV_LINE_FN int tiles_before(const Line& p, const Req& r, int rt) {
  const int n = row_tiles(p, r);
  if (rt <= 0) return 0;
  if (rt == 1) return last_tile(p, r, 0) - first_tile(p, r, 0) + 1;
  int s = rt + (int)floor_sum(rt == n ? n - 1 : rt, kTile, p.TQ, r.base + p.TQ - 1);
  if (rt == n) s += last_tile(p, r, n - 1);
  if (p.window > 0) {
    // first token of row tile i: max(0, x + i TQ), above 0 from i0 on at the earliest (a window may be as long as
    // numbers go, so -x + TQ needs the 32nd bit)
    const int x = r.base - p.window + 1;
    const uint32_t u = (uint32_t)x, tq = (uint32_t)p.TQ, i0 = x >= 0 ? 0 : (0u - u + tq - 1) / tq;
    if (i0 < (uint32_t)rt) s -= (int)floor_sum((uint32_t)rt - i0, kTile, tq, u + i0 * tq);
  }
  return s;
}

// The cut of `total` tiles into grid ranges that differ by at most one tile.
struct Cut {
  int per, rem;
  KV_LINE Cut(int total, int grid) : per(total / grid), rem(total - per * grid) {}
  KV_LINE int begin(int c) const { return c * per + min(c, rem); }
  KV_LINE int owner(int x) const {
    const int big = rem * (per + 1);
    return x < big ? x / (per + 1) : rem + (x - big) / max(per, 1);
  }
};

}  // namespace w4a16
