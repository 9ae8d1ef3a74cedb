// kv_attention.cu -- attention over the paged 8-bit key/value cache
// (w4a16_kv_attention; the formulas are those of include/w4a16.h "Paged
// key/value cache").
//
// Mathematics.  The bytes of K and V go to the tensor cores as they lie in
// the cache; what is not e4m3 is split into e4m3 terms instead:
//   * a bf16 query has 8 significant bits, an e4m3 value 4, so with a power
//     of two e per row, q / e = hi + lo / 16 exactly (to 2^-22 of the row's
//     largest element), and K q = e (K hi + K lo / 16);
//   * the weights p = exp(z - max) <= 1 enter as 256 p = hi + lo / 16, two
//     terms again: rounded to 8 significant bits, as a bf16 P would be.
// S^T = K [hi | lo]^T puts a cached token on each TMEM lane and the query
// rows (and their second terms) on the columns, so a few query rows fill the
// MMA's N and not its 128-row M; O^T = V^T [hi | lo] takes V as it lies too (an
// M-major operand).  With z in log2 units, a token's V scale vs joins its
// weight before the maximum is taken (z + log2 vs), so the terms stay in
// e4m3's range whatever the blocks' scales; the row sum takes p / vs.
//
// Split.  A tile is 128 tokens at a fixed position; a group eight tiles.  A
// tile gives (maximum m, sum l, O) per row; a group folds its tiles in order,
// a row its groups in eight interleaved chains joined as a tree
// (kv_combine_kernel).  All tiles of the call form one line (request, row
// tile, key head, tile) cut into equal ranges, one per CTA: a group that lies
// in one range is folded in registers and written as one partial result, one
// that a cut divides is written tile by tile and folded by the combine kernel
// with the same operations.  So the cut follows the load and the bits do not.
//
// Bound: HBM.  A 128-token tile of heads of 256 is 64 KB; one CTA has one to
// two tiles in flight, two CTAs an SM where shared memory allows.
//
// CTA: six warps.
//   warps 0-3  a thread per token: scores from TMEM, mask, maximum, weights
//              into shared memory; then a thread per output column (TMEM lane
//              again): O from TMEM folded into registers
//   warp 4     work list, block table, TMA of K and V blocks, scales
//   warp 5     tensor memory, MMA issue (lane 0)
// Every wait is bounded: one that gives up raises W4A16_DEVICE_TIMEOUT, the
// roles leave their loops, copies and MMAs in flight are waited for (bounded)
// and the tensor memory is freed.
#include <cuda.h>
#include <cuda_fp8.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "kv.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace w4a16 {
namespace {

using namespace ptx;

constexpr int kTile = 128;      // tokens per tile (the M of the MMAs)
constexpr int kGroupTiles = 8;  // tiles per group
constexpr int kChains = 8;      // interleaved chains over a row's groups
constexpr int kThreads = 192;
constexpr int kDescs = 4;       // tile descriptors in flight
constexpr int kSms = 152;
constexpr float kLog2e = 1.4426950408889634f;

// flags of a tile descriptor
constexpr int kNewSeg = 1;     // another (request, row tile, head) than the tile before
constexpr int kEnd = 2;        // no tile: the CTA's range is done
constexpr int kBadBlock = 4;   // some needed block is not in the cache
constexpr int kGroupBegin = 8; // first tile of a group folded here
constexpr int kGroupEnd = 16;  // its last tile
constexpr int kPart = 32;      // tile of a group that a cut divides
constexpr int kTail = 64;      // ... at this CTA's end (else at its beginning)

struct Desc {
  int flags, h, j0, tile;      // key head, first token of the row tile in its request
  int base, fresh, c0, gi;     // tokens before the step, new tokens, first row, group slot
  int pad[8];
  float ks[8], vs[8];          // scales of the tile's blocks (0: no such block)
};
static_assert(sizeof(Desc) == 128, "two 64-byte halves");

template <int D, int RP>
struct Geo {
  static constexpr int kPanels = D <= 128 ? 1 : D / 128;       // 128-byte column panels of K and V
  static constexpr int kPanelBytes = D <= 128 ? kTile * D : kTile * 128;
  static constexpr int kSlot = kTile * D;
  static constexpr int kQ = kPanels * 2 * RP * 128;
  static constexpr int kP = kTile * 2 * RP;
  // two CTAs an SM where three K/V tiles, the queries and two weight tiles fit in half of it
  static constexpr int kCtas = D == 256 && RP > 8 ? 1 : 2;
  static constexpr int kSlots = D == 256 ? (RP == 8 ? 3 : RP == 16 ? 6 : 5) : D == 128 ? (RP > 16 ? 5 : 6) : 8;
  static constexpr int kBars = 2 * kSlots + 2 * kDescs + 2 * 2 + 2 + 2 + 1 + 1;
  static constexpr int kRows = RP * 4 * (2 * 4 * 2 + 2 * 4 + 3);  // maxima, sums (two tiles x four warps), factors, limits
  static constexpr int kSmem = kSlots * kSlot + kQ + 2 * kP + kDescs * (int)sizeof(Desc) + kRows + 8 * kBars + 16 + 1024;
  static constexpr uint32_t kTmem = RP == 8 ? 64 : RP == 16 ? 128 : 256;  // S twice, O once
  static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
};

struct Params {
  const uint16_t* q;
  int64_t q_stride;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  const int32_t* cu;
  const int32_t* lens;
  uint16_t* out;
  int B, T, q_heads, heads, G, TQ;  // G query heads per key head, TQ tokens per row tile
  int blocks, shift, max_blocks, max_new, max_len, window;
  float qk_scale;  // scale * log2(e)
  int gmax;        // group slots per row
  int grid;
  // workspace
  int64_t* starts;  // [B + 1] tiles before each request
  float* g_acc;     // [gmax][T][q_heads][D]
  float2* g_ml;     // [gmax][T][q_heads]
  float* t_acc;     // [grid][2 * kGroupTiles][RP][D]
  float2* t_ml;     // [grid][2 * kGroupTiles][RP]
  int* flags;
};

struct Maps {
  CUtensorMap k, v;
};

// ---- the line of tiles -----------------------------------------------------------------------

// One request of the step: its row tiles and their ranges of 128-token tiles.
struct Req {
  int c0, fresh, base;  // first row, new tokens (0: nothing to do), tokens before them
};

__device__ __forceinline__ Req load_req(const Params& p, int b, bool* bad) {
  Req r{0, 0, 0};
  if (b >= p.B) return r;
  const int c0 = p.cu[b], c1 = p.cu[b + 1], len = p.lens[b];
  const bool ok = c0 >= 0 && c0 <= c1 && c1 <= p.T && c1 - c0 <= p.max_new && c1 - c0 <= len && len <= p.max_len;
  if (!ok) {
    if (c1 != c0) *bad = true;
    return r;
  }
  r.c0 = c0;
  r.fresh = c1 - c0;
  r.base = len - r.fresh;
  return r;
}

__device__ __forceinline__ int row_tiles(const Params& p, const Req& r) { return (r.fresh + p.TQ - 1) / p.TQ; }
__device__ __forceinline__ int first_tile(const Params& p, const Req& r, int rt) {
  return p.window > 0 ? max(0, r.base + rt * p.TQ - p.window + 1) / kTile : 0;
}
__device__ __forceinline__ int last_tile(const Params& p, const Req& r, int rt) {
  return (r.base + min((rt + 1) * p.TQ, r.fresh) - 1) / kTile;
}

// sum over 0 <= i < n of floor((b + i a) / m), all >= 0: whole parts are
// taken out, then the lattice points under the line are counted along the
// other axis, as in Euclid's algorithm.
__device__ inline int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t s = 0;
  while (n > 0) {
    s += n * (n - 1) / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const int64_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const int64_t t = a;
    a = m;
    m = t;
  }
  return s;
}

// Tiles of the row tiles before rt (of one key head).
__device__ inline int64_t tiles_before(const Params& p, const Req& r, int rt) {
  const int n = row_tiles(p, r);
  if (rt <= 0) return 0;
  if (rt == 1) return last_tile(p, r, 0) - first_tile(p, r, 0) + 1;
  int64_t s = rt + floor_sum(rt == n ? n - 1 : rt, kTile, p.TQ, r.base + p.TQ - 1);
  if (rt == n) s += last_tile(p, r, n - 1);
  if (p.window > 0) {
    const int x = r.base - p.window + 1;  // first token of row tile i: max(0, x + i TQ)
    const int i0 = x >= 0 ? 0 : min(rt, (-x + p.TQ - 1) / p.TQ);
    s -= floor_sum(rt - i0, kTile, p.TQ, max(0, x + i0 * p.TQ));
  }
  return s;
}

// ---- shared pieces -----------------------------------------------------------------------------

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {  // a in the low byte
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3)));
}

// a, b as hi + lo / 16 (each two codes)
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = e4m3x2(a, b);
  const float2 h = from_e4m3x2(hi);
  lo = e4m3x2(__fmul_rn(__fsub_rn(a, h.x), 16.f), __fmul_rn(__fsub_rn(b, h.y), 16.f));
}

// One step of a fold: the running (m, l) takes in (mt, lt); al and be are
// what the running and the new accumulators are multiplied by.  An empty
// side (m = -inf) leaves the other as it is, bit for bit.
__device__ __forceinline__ void fold_ml(float& m, float& l, float mt, float lt, float& al, float& be) {
  const float top = fmaxf(m, mt), ref = top == -INFINITY ? 0.f : top;
  al = exp2f(m - ref);
  be = exp2f(mt - ref);
  l = __fmaf_rn(l, al, __fmul_rn(lt, be));
  m = top;
}

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Barrier of the four softmax warps; returns whether any thread came with `fail`.
__device__ __forceinline__ bool softmax_sync(bool fail) {
  uint32_t any;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.or.pred q, 1, 128, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(any)
      : "r"((uint32_t)fail)
      : "memory");
  return any != 0;
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[N]) {
  static_assert(N % 8 == 0, "columns");
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    float t[8];
    tmem_ld8(addr + i, t);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[i + k] = t[k];
  }
}

// ---- the kernel -----------------------------------------------------------------------------------

template <int D, int RP>
__global__ void __launch_bounds__(kThreads, Geo<D, RP>::kCtas)
    kv_attention_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  using X = Geo<D, RP>;
  constexpr int NS = X::kSlots, NP = X::kPanels;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_mem = base + NS * X::kSlot;
  uint8_t* p_mem = q_mem + X::kQ;
  Desc* descs = reinterpret_cast<Desc*>(p_mem + 2 * X::kP);
  float* s_max = reinterpret_cast<float*>(descs + kDescs);  // [2][4][RP]
  float* s_sum = s_max + 2 * 4 * RP;                        // [2][4][RP]
  float2* s_ab = reinterpret_cast<float2*>(s_sum + 2 * 4 * RP);  // [4][RP]
  float* s_qf = reinterpret_cast<float*>(s_ab + 4 * RP);    // [RP] score factor of a row
  int2* s_lim = reinterpret_cast<int2*>(s_qf + RP);         // [RP] first and last token a row sees
  uint64_t* bar_mem = reinterpret_cast<uint64_t*>(s_lim + RP);
  const uint32_t slots = smem_u32(base), q_s = smem_u32(q_mem), p_s = smem_u32(p_mem), bars = smem_u32(bar_mem);
  auto full = [&](int i) { return bars + 8u * i; };                   // slot: copies landed
  auto empty = [&](int i) { return bars + 8u * (NS + i); };           // slot: MMAs done with it
  auto d_full = [&](int i) { return bars + 8u * (2 * NS + i); };      // descriptor and scales written
  auto d_free = [&](int i) { return bars + 8u * (2 * NS + kDescs + i); };
  auto s_full = [&](int i) { return bars + 8u * (2 * NS + 2 * kDescs + i); };
  auto s_free = [&](int i) { return bars + 8u * (2 * NS + 2 * kDescs + 2 + i); };
  auto p_full = [&](int i) { return bars + 8u * (2 * NS + 2 * kDescs + 4 + i); };
  const uint32_t o_full = bars + 8u * (2 * NS + 2 * kDescs + 6), o_free = o_full + 8, q_full = o_full + 16;
  const uint32_t drained = o_full + 24;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bar_mem + X::kBars);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(d_full(i), 33);
      mbar_init(d_free(i), 5);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(s_free(i), 4);
      mbar_init(p_full(i), 4);
    }
    mbar_init(o_full, 1);
    mbar_init(o_free, 4);
    mbar_init(q_full, 4);
    mbar_init(drained, 1);
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(s_tmem), X::kTmem);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *s_tmem;
  const uint32_t s_col = tmem, o_col = tmem + 4 * RP;
  auto give_up = [&]() {
    atomicOr(p.flags, W4A16_DEVICE_TIMEOUT);
    *s_abort = 1;
  };
  auto wait_warp = [&](uint32_t bar, uint32_t parity) -> bool {  // all lanes; the same answer for all
    const bool ok = __all_sync(0xffffffffu, mbar_wait_parked(bar, parity)) && !*s_abort;
    return __all_sync(0xffffffffu, ok);
  };
  pdl_launch_dependents();
  pdl_wait();
  int loads = 0;  // producer: slots requested

  if (warp == 4) {
    // ---- work list and copies ----
    const int nb = kTile >> p.shift, block = 1 << p.shift;  // blocks per tile
    bool bad = false;
    int64_t total = 0;
    Req mine{0, 0, 0};
    int64_t mine_end = 0;  // inclusive prefix of this lane's request
    auto scan = [&](int b0) {  // loads 32 requests; their inclusive prefix of tiles after `total`
      mine = load_req(p, b0 + lane, &bad);
      int64_t n = mine.fresh > 0 ? tiles_before(p, mine, row_tiles(p, mine)) * p.heads : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, n, d);
        if (lane >= d) n += o;
      }
      mine_end = total + n;
    };
    int b0 = 0;
    for (; b0 < p.B; b0 += 32) {
      scan(b0);
      if (blockIdx.x == 0 && b0 + lane < p.B) p.starts[b0 + lane + 1] = mine_end;
      total = __shfl_sync(0xffffffffu, mine_end, 31);
    }
    if (blockIdx.x == 0 && lane == 0) p.starts[0] = 0;
    if (bad && blockIdx.x == 0) atomicOr(p.flags, W4A16_DEVICE_KV_RANGE);
    const int64_t all = total;
    const int64_t beg = all * blockIdx.x / p.grid, end = all * (blockIdx.x + 1) / p.grid;
    // the request of `beg`
    if (p.B > 32) {
      total = 0;
      for (b0 = 0; b0 < p.B; b0 += 32) {
        scan(b0);
        const int64_t e = __shfl_sync(0xffffffffu, mine_end, 31);
        if (e > beg) break;
        total = e;
      }
    } else {
      b0 = 0;
      total = 0;
    }
    int b = 0, rt = 0, h = 0, tile = 0, t_first = 0, t_last = -1;
    int64_t x = beg;   // position on the line
    int64_t seg0 = 0;  // position of the segment's first tile
    Req r{0, 0, 0};
    auto take = [&](int bl) {  // request b0 + bl becomes the current one
      b = b0 + bl;
      r.c0 = __shfl_sync(0xffffffffu, mine.c0, bl);
      r.fresh = __shfl_sync(0xffffffffu, mine.fresh, bl);
      r.base = __shfl_sync(0xffffffffu, mine.base, bl);
    };
    auto enter = [&]() {
      t_first = first_tile(p, r, rt);
      t_last = last_tile(p, r, rt);
    };
    if (beg < end) {
      const unsigned past = __ballot_sync(0xffffffffu, mine_end > beg);
      const int bl = __ffs(past) - 1;
      const int64_t start = bl > 0 ? __shfl_sync(0xffffffffu, mine_end, bl > 0 ? bl - 1 : 0) : total;
      take(bl);
      int64_t off = beg - start;
      int lo = 0, hi = row_tiles(p, r);
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tiles_before(p, r, mid) * p.heads <= off) lo = mid;
        else hi = mid;
      }
      rt = lo;
      if (rt > 0) off -= tiles_before(p, r, rt) * p.heads;
      enter();
      const int n = t_last - t_first + 1;
      h = (int)(off / n);
      tile = t_first + (int)(off % n);
      seg0 = beg - (tile - t_first);
    }
    // block id of lane l for a tile: -2 not needed, -1 (or any bad id) not in the cache
    auto load_id = [&](int bb, const Req& rr, int row_tile, int tl) {
      const int lo = p.window > 0 ? max(0, rr.base + row_tile * p.TQ - p.window + 1) : 0;
      const int hi = rr.base + min((row_tile + 1) * p.TQ, rr.fresh) - 1;
      const int j = tl * nb + lane;
      if (lane >= nb || (j + 1) * block <= lo || j * block > hi) return -2;
      return j < p.max_blocks ? p.table[(int64_t)bb * p.max_blocks + j] : -1;
    };
    int id = beg < end ? load_id(b, r, rt, tile) : -2;
    bool fresh_seg = true, ok = true;
    int t = 0;
    for (; x < end && ok; ++x, ++t) {
      // this tile's descriptor
      const int ds = t % kDescs;
      const int ch = h, crt = rt, ctile = tile;
      const Req cr = r;
      const int64_t g_lo = max(seg0, x - (ctile % kGroupTiles)), g_hi = min(seg0 + t_last - t_first, x - ctile % kGroupTiles + kGroupTiles - 1);
      const bool whole = g_lo >= beg && g_hi < end;
      int fl = fresh_seg ? kNewSeg : 0;
      if (whole) fl |= (x == g_lo ? kGroupBegin : 0) | (x == g_hi ? kGroupEnd : 0);
      else fl |= kPart | (g_lo >= beg ? kTail : 0);
      const bool valid = id >= 0 && id < p.blocks;
      const unsigned need = __ballot_sync(0xffffffffu, id != -2), have = __ballot_sync(0xffffffffu, valid);
      if (need != have) fl |= kBadBlock;
      if (t >= kDescs && !(ok = wait_warp(d_free(ds), ((t / kDescs) - 1) & 1))) break;
      Desc& de = descs[ds];
      if (lane == 0) {
        de.flags = fl;
        de.h = ch;
        de.j0 = crt * p.TQ;
        de.tile = ctile;
        de.base = cr.base;
        de.fresh = cr.fresh;
        de.c0 = cr.c0;
        de.gi = ctile / kGroupTiles - first_tile(p, cr, 0) / kGroupTiles;
        if (need != have) atomicOr(p.flags, W4A16_DEVICE_KV_RANGE);
      }
      if (lane < nb) {
        if (valid) {
          cp_async4(smem_u32(&de.ks[lane]), p.k_scale + (int64_t)id * p.heads + ch);
          cp_async4(smem_u32(&de.vs[lane]), p.v_scale + (int64_t)id * p.heads + ch);
        } else {
          de.ks[lane] = 0.f;
          de.vs[lane] = 0.f;
        }
      }
      __syncwarp();
      cp_async_arrive(d_full(ds));
      if (lane == 0) mbar_arrive(d_full(ds));
      // the next tile, its block ids requested before this one's slots are waited for
      const bool same = tile < t_last;
      if (x + 1 < end) {
        if (same) {
          ++tile;
        } else {
          seg0 = x + 1;
          if (++h == p.heads) {
            h = 0;
            if (++rt == row_tiles(p, r)) {
              rt = 0;
              int bl = b - b0;
              for (;;) {  // the next request with new tokens (there is one: x + 1 < all)
                const unsigned later = __ballot_sync(0xffffffffu, mine.fresh > 0 && lane > bl);
                if (later) {
                  take(__ffs(later) - 1);
                  break;
                }
                b0 += 32;
                if (b0 >= p.B) break;
                mine = load_req(p, b0 + lane, &bad);
                bl = -1;
              }
            }
          }
          enter();
          tile = t_first;
        }
      }
      const int next_id = x + 1 < end ? load_id(b, r, rt, tile) : -2;
      // lane (block, panel): one copy each of K, then of V
      const int nv = __popc(have);
      const int src = lane / NP, panel = lane % NP;
      const int nth = src < nv ? __fns(have, 0, src + 1) : 0;
      const int my_id = __shfl_sync(0xffffffffu, id, nth & 31);
      const int row = (my_id * p.heads + ch) << p.shift;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int slot = loads % NS;
        if (loads >= NS && !(ok = wait_warp(empty(slot), ((loads / NS) - 1) & 1))) break;
        if (lane == 0) mbar_expect_tx(full(slot), (uint32_t)(nv * block * D));
        __syncwarp();
        if (lane < nv * NP)
          tma_load_2d(slots + slot * X::kSlot + panel * X::kPanelBytes + nth * block * (D <= 128 ? D : 128),
                      kv ? &maps.v : &maps.k, panel * 128, row, full(slot));
        ++loads;
      }
      id = next_id;
      fresh_seg = !same;
    }
    if (!ok) {
      if (lane == 0) give_up();
    } else {  // the end mark
      const int ds = t % kDescs;
      if (t < kDescs || wait_warp(d_free(ds), ((t / kDescs) - 1) & 1)) {
        if (lane == 0) descs[ds].flags = kEnd;
        __syncwarp();
        cp_async_arrive(d_full(ds));
        if (lane == 0) mbar_arrive(d_full(ds));
      } else if (lane == 0) {
        give_up();
      }
    }
  } else if (warp == 5) {
    // ---- MMA issue: S of tile t, then O of tile t - 1 ----
    if (lane == 0) {
      constexpr uint32_t id_s = umma_idesc_e4m3(128, 2 * RP, false, false);
      constexpr uint32_t id_o = umma_idesc_e4m3(128, 2 * RP, true, true);
      bool ok = true;
      int seg = 0;
      auto issue_o = [&](int t) {  // O = V^T P^T of tile t
        const int slot = (2 * t + 1) % NS;
        ok = mbar_wait_parked(p_full(t & 1), (t >> 1) & 1) && mbar_wait_parked(full(slot), ((2 * t + 1) / NS) & 1) &&
             (t == 0 || mbar_wait_parked(o_free, (t - 1) & 1)) && !*s_abort;
        if (!ok) return;
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < NP; ++c)
#pragma unroll
          for (int k = 0; k < kTile / 32; ++k) {
            const uint32_t va = slots + slot * X::kSlot + c * X::kPanelBytes + k * 32 * (D < 128 ? D : 128);
            // heads of 64: the MMA's rows 64 .. 127 repeat whatever lies 512 bytes on, and nobody reads them
            const uint64_t ad = D < 128 ? umma_desc(va, 512, 512, 4) : umma_desc(va, 1024, 1024, 2);
            const uint64_t bd = umma_desc(p_s + (t & 1) * X::kP + k * 512, 128, 2048, 0);
            umma_f8(o_col + c * 2 * RP, ad, bd, id_o, k > 0);
          }
        umma_commit(o_full);
        umma_commit(empty(slot));
      };
      int t = 0;
      for (;; ++t) {
        const int ds = t % kDescs;
        ok = mbar_wait_parked(d_full(ds), (t / kDescs) & 1) && !*s_abort;
        if (!ok) break;
        const int fl = descs[ds].flags;
        mbar_arrive(d_free(ds));
        if (fl & kEnd) break;
        if (t > 0 && (fl & kNewSeg)) issue_o(t - 1);  // the queries of a new segment come after the old one's last O
        if (!ok) break;
        const int slot = (2 * t) % NS;
        if (fl & kNewSeg) ok = mbar_wait_parked(q_full, seg++ & 1);
        ok = ok && mbar_wait_parked(full(slot), ((2 * t) / NS) & 1) &&
             (t < 2 || mbar_wait_parked(s_free(t & 1), ((t >> 1) - 1) & 1)) && !*s_abort;
        if (!ok) break;
        tc_fence_after_sync();
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const uint32_t ka = slots + slot * X::kSlot + (k / 4) * X::kPanelBytes + (k % 4) * 32;
          const uint64_t ad = D < 128 ? umma_desc(ka, 16, 512, 4) : umma_desc(ka, 16, 1024, 2);
          const uint64_t bd = umma_desc(q_s + (k / 4) * 2 * RP * 128 + (k % 4) * 32, 16, 1024, 2);
          umma_f8(s_col + (t & 1) * 2 * RP, ad, bd, id_s, k > 0);
        }
        umma_commit(s_full(t & 1));
        umma_commit(empty(slot));
        if (t > 0 && !(fl & kNewSeg)) issue_o(t - 1);
        if (!ok) break;
      }
      if (ok && t > 0) issue_o(t - 1);
      if (!ok) give_up();
    }
  } else {
    // ---- softmax and fold: thread = token of the tile, then = output column ----
    const uint32_t lane_col = (uint32_t)(32 * warp) << 16;
    float acc[NP][RP];
#pragma unroll
    for (int c = 0; c < NP; ++c)
#pragma unroll
      for (int i = 0; i < RP; ++i) acc[c][i] = 0.f;
    float m_run = -INFINITY, l_run = 0.f;  // lane r of every warp: row r
    bool fail = false;
    // the tile whose O is not folded yet
    struct {
      int flags, h, j0, tile, fresh, c0, gi;
    } prev = {kEnd, 0, 0, 0, 0, 0, 0};
    uint32_t poison[NP];  // rows (bits) of that tile that see a NaN in this thread's column
#pragma unroll
    for (int c = 0; c < NP; ++c) poison[c] = 0;

    // O of tile t: into the accumulators, or out to the workspace
    auto fold = [&](int t) {
      if (!wait_warp(o_full, t & 1)) fail = true;
      if (softmax_sync(fail)) {  // (also: every warp's sums of the tile are written)
        fail = true;
        return;
      }
      tc_fence_after_sync();
      const int par = t & 1;
      float mt = -INFINITY, lt = 0.f;
      if (lane < RP) {
        const float* sm = s_max + par * 4 * RP + lane;
        const float* sl = s_sum + par * 4 * RP + lane;
        mt = fmaxf(fmaxf(sm[0], sm[RP]), fmaxf(sm[2 * RP], sm[3 * RP]));
        lt = __fadd_rn(__fadd_rn(sl[0], sl[RP]), __fadd_rn(sl[2 * RP], sl[3 * RP]));
      }
      const bool part = prev.flags & kPart;
      if (prev.flags & kGroupBegin) {
        m_run = -INFINITY;
        l_run = 0.f;
#pragma unroll
        for (int c = 0; c < NP; ++c)
#pragma unroll
          for (int i = 0; i < RP; ++i) acc[c][i] = 0.f;
      }
      if (!part) {
        float al, be;
        fold_ml(m_run, l_run, mt, lt, al, be);
        if (lane < RP) s_ab[warp * RP + lane] = make_float2(al, be);
        __syncwarp();
      }
      const int rows = min(p.TQ, prev.fresh - prev.j0) * p.G;
      const int part_slot = blockIdx.x * 2 * kGroupTiles + (prev.flags & kTail ? kGroupTiles : 0) + prev.tile % kGroupTiles;
#pragma unroll
      for (int c = 0; c < NP; ++c) {
#pragma unroll
        for (int i0 = 0; i0 < RP; i0 += 8) {
          float hi[8], lo[8];
          tmem_ld8(o_col + c * 2 * RP + i0 + lane_col, hi);
          tmem_ld8(o_col + c * 2 * RP + RP + i0 + lane_col, lo);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            // weights were 256 p = hi + lo / 16
            float o = __fmul_rn(__fmaf_rn(lo[i], 0.0625f, hi[i]), 0.00390625f);
            if ((poison[c] >> (i0 + i)) & 1) o = __uint_as_float(0x7FC00000u);
            if (part) {
              const int d = c * 128 + 32 * warp + lane;
              if (i0 + i < rows && (D >= 128 || d < D))
                p.t_acc[((int64_t)part_slot * RP + i0 + i) * D + d] = o;
            } else {
              const float2 ab = s_ab[warp * RP + i0 + i];
              acc[c][i0 + i] = __fmaf_rn(acc[c][i0 + i], ab.x, __fmul_rn(o, ab.y));
            }
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
      if (part) {
        if (warp == 0 && lane < rows) p.t_ml[(int64_t)part_slot * RP + lane] = make_float2(mt, lt);
      } else if (prev.flags & kGroupEnd) {
        const int64_t row0 = ((int64_t)prev.gi * p.T + prev.c0 + prev.j0) * p.q_heads + prev.h * p.G;
        int j = 0, g = 0;
#pragma unroll
        for (int i = 0; i < RP; ++i) {
          if (i < rows) {
            const int64_t row = row0 + (int64_t)j * p.q_heads + g;
#pragma unroll
            for (int c = 0; c < NP; ++c) {
              const int d = c * 128 + 32 * warp + lane;
              if (D >= 128 || d < D) p.g_acc[row * D + d] = acc[c][i];
            }
          }
          if (++g == p.G) {
            g = 0;
            ++j;
          }
        }
        if (warp == 0 && lane < rows)
          p.g_ml[row0 + (int64_t)(lane / p.G) * p.q_heads + lane % p.G] = make_float2(m_run, l_run);
      }
    };

    int t = 0;
    for (;; ++t) {
      const int ds = t % kDescs, par = t & 1;
      if (!wait_warp(d_full(ds), (t / kDescs) & 1)) fail = true;
      if (softmax_sync(fail)) {
        fail = true;
        break;
      }
      const Desc& de = descs[ds];
      const int fl = de.flags;
      if (fl & kEnd) break;
      const int base_tok = de.base, j0 = de.j0, fresh = de.fresh, c0 = de.c0, h = de.h, tile = de.tile, gi = de.gi;
      const int toks = min(p.TQ, fresh - j0);
      if (fl & kNewSeg) {
        if (t > 0) {
          fold(t - 1);
          if (fail) break;
        }
        // query rows as e4m3 terms: 128 / RP threads a row
        constexpr int TPR = 128 / RP, CPT = (D / 8 + TPR - 1) / TPR;
        const int r = tid / TPR, c = tid % TPR;
        const int j = r / p.G, g = r - j * p.G;
        const bool live = j < toks;
        uint4 v[CPT];
        uint32_t peak = 0;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          v[i] = make_uint4(0, 0, 0, 0);
          const int ch = c + i * TPR;
          if (live && ch < D / 8)
            v[i] = ld_nc_v4(p.q + (int64_t)(c0 + j0 + j) * p.q_stride + (int64_t)(h * p.G + g) * D + 8 * ch);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t u = word_of(v[i], w) & 0x7FFF7FFFu;
            peak = max(peak, max(u & 0xFFFF, u >> 16));
          }
        }
#pragma unroll
        for (int d = TPR / 2; d; d >>= 1) peak = max(peak, __shfl_xor_sync(0xffffffffu, peak, d));
        // largest element into (224, 448]: 448 = 1.75 * 2^8
        const int e = min(max((int)(peak >> 7) - 127 - 8 + ((peak & 127) > 96 ? 1 : 0), -120), 120);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          const int ch = c + i * TPR;
          if (ch < D / 8) {
            float f[8];
            widen8(v[i], f);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) split2(__fmul_rn(f[2 * w], inv), __fmul_rn(f[2 * w + 1], inv), hi[w], lo[w]);
            // K-major, 128-byte swizzle: row n of panel ch / 16
            auto at = [&](int n) {
              return q_mem + (ch / 16) * 2 * RP * 128 + n * 128 + ((((ch % 16) >> 1) ^ (n & 7)) << 4) + (ch & 1) * 8;
            };
            *reinterpret_cast<uint2*>(at(r)) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
            *reinterpret_cast<uint2*>(at(RP + r)) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
          }
        }
        if (c == 0) {
          const float unit = __uint_as_float((uint32_t)(127 + e) << 23);
          // a row with a NaN or an infinity is NaN as a whole
          s_qf[r] = peak >= 0x7F80 ? __uint_as_float(0x7FC00000u) : __fmul_rn(unit, p.qk_scale);
          const int pos = base_tok + j0 + j;
          s_lim[r] = live ? make_int2(p.window > 0 ? pos - p.window + 1 : 0, pos) : make_int2(0, -1);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        if (softmax_sync(false)) {
          fail = true;
          break;
        }
      }
      // token of this thread
      const int tok = tile * kTile + tid;
      const int blk = tid >> p.shift;
      const float ks = de.ks[blk], vs = de.vs[blk];
      const int pos0 = base_tok + j0, pos1 = pos0 + toks - 1;  // positions of the first and last row
      const bool masked = tile * kTile + kTile - 1 > pos0 || (p.window > 0 && tile * kTile < pos1 - p.window + 1);
      const bool fix = masked || (fl & kBadBlock);
      const bool dead = ks == 0.f || tok > pos1 || (p.window > 0 && tok < pos0 - p.window + 1);
      const float lv = dead ? 0.f : log2f(vs), iv = dead ? 0.f : __frcp_rn(vs);
      if (!wait_warp(s_full(par), (t >> 1) & 1)) fail = true;
      tc_fence_after_sync();
      float s[RP];
      {
        float lo[RP];
        tmem_ld<RP>(s_col + par * 2 * RP + lane_col, s);
        tmem_ld<RP>(s_col + par * 2 * RP + RP + lane_col, lo);
        tmem_wait_ld();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free(par));
#pragma unroll
        for (int i = 0; i < RP; ++i)
          s[i] = __fmaf_rn(__fmul_rn(__fmaf_rn(lo[i], 0.0625f, s[i]), s_qf[i]), ks, lv);
      }
      if (fix) {
#pragma unroll
        for (int i = 0; i < RP; ++i) {
          const int2 lim = s_lim[i];
          if (dead || tok < lim.x || tok > lim.y) s[i] = -INFINITY;
        }
      }
#pragma unroll
      for (int i = 0; i < RP; ++i) {
        const float m = warp_max(s[i]);
        if (lane == i) s_max[(par * 4 + warp) * RP + i] = m;
      }
      // V rows that no row sees (stale shared memory, unset blocks) become
      // zeros; NaN codes that only some rows see are taken out of V and put
      // into those rows' results
      bool nan_code = false;
      uint8_t* v_row = base + ((2 * t + 1) % NS) * X::kSlot;
      const bool partly = masked && !dead && (tok > pos0 || (p.window > 0 && tok < pos1 - p.window + 1));
      constexpr int kRowB = D < 128 ? D : 128, kCh = kRowB / 16;
      if (fix) {
        if (!wait_warp(full((2 * t + 1) % NS), ((2 * t + 1) / NS) & 1)) fail = true;
        if (dead || partly) {
#pragma unroll
          for (int c = 0; c < NP; ++c)
#pragma unroll
            for (int i = 0; i < kCh; ++i) {
              uint4* w = reinterpret_cast<uint4*>(v_row + c * X::kPanelBytes + tid * kRowB + ((i + tid) % kCh) * 16);
              if (dead) {
                *w = make_uint4(0, 0, 0, 0);
              } else {
                const uint4 u = *w;
                const uint32_t any = (((u.x & 0x7F7F7F7Fu) + 0x01010101u) | ((u.y & 0x7F7F7F7Fu) + 0x01010101u) |
                                      ((u.z & 0x7F7F7F7Fu) + 0x01010101u) | ((u.w & 0x7F7F7F7Fu) + 0x01010101u)) &
                                     0x80808080u;
                nan_code |= any != 0;
              }
            }
        }
      }
      if (softmax_sync(fail)) {
        fail = true;
        break;
      }
      uint32_t taint[NP];
#pragma unroll
      for (int c = 0; c < NP; ++c) taint[c] = 0;
      if (masked && toks > 1) {
        if (softmax_sync(nan_code)) {
          // (rare) this thread's columns: which tokens hold NaN, which rows see one
#pragma unroll
          for (int c = 0; c < NP; ++c) {
            uint32_t hit[4] = {0, 0, 0, 0};
            if (tid < kRowB)
              for (int k = 0; k < kTile; ++k) {
                const int sw = D < 128 ? (k >> 1) & 3 : k & 7;
                const uint8_t code = v_row[c * X::kPanelBytes + k * kRowB + (((tid >> 4) ^ sw) << 4) + (tid & 15)];
                if ((code & 0x7F) == 0x7F) hit[k >> 5] |= 1u << (k & 31);
              }
            for (int i = 0; i < RP; ++i) {
              const int lo = s_lim[i].x - tile * kTile, hi = s_lim[i].y - tile * kTile;
              bool sees = false;
              for (int k = 0; k < kTile; ++k) sees |= k >= lo && k <= hi && ((hit[k >> 5] >> (k & 31)) & 1);
              if (sees) taint[c] |= 1u << i;
            }
          }
          softmax_sync(false);
          if (nan_code) {
#pragma unroll 1
            for (int c = 0; c < NP; ++c)
              for (int i = 0; i < kRowB; ++i) {
                uint8_t& code = v_row[c * X::kPanelBytes + tid * kRowB + i];
                if ((code & 0x7F) == 0x7F) code = 0;
              }
          }
        }
      }
      // weights, their sums, and their two terms
      uint32_t hi[RP / 2], lo[RP / 2];
#pragma unroll
      for (int i = 0; i < RP; i += 4) {
        const float* sm = s_max + par * 4 * RP + i;
        float4 mx = *reinterpret_cast<const float4*>(sm);
#pragma unroll
        for (int w = 1; w < 4; ++w) {
          const float4 o = *reinterpret_cast<const float4*>(sm + w * RP);
          mx.x = fmaxf(mx.x, o.x);
          mx.y = fmaxf(mx.y, o.y);
          mx.z = fmaxf(mx.z, o.z);
          mx.w = fmaxf(mx.w, o.w);
        }
        s[i + 0] = exp2f(s[i + 0] - (mx.x == -INFINITY ? 0.f : mx.x));
        s[i + 1] = exp2f(s[i + 1] - (mx.y == -INFINITY ? 0.f : mx.y));
        s[i + 2] = exp2f(s[i + 2] - (mx.z == -INFINITY ? 0.f : mx.z));
        s[i + 3] = exp2f(s[i + 3] - (mx.w == -INFINITY ? 0.f : mx.w));
      }
#pragma unroll
      for (int i = 0; i < RP; i += 2)
        split2(__fmul_rn(s[i], 256.f), __fmul_rn(s[i + 1], 256.f), hi[i / 2], lo[i / 2]);
      {
        // row n of the weights: n % 16 within 16-byte rows of tokens, n / 16 2048 bytes apart; hi rows, then lo
        uint32_t w[RP / 2];
#pragma unroll
        for (int i = 0; i < RP / 4; ++i) {
          w[i] = hi[2 * i] | hi[2 * i + 1] << 16;
          w[RP / 4 + i] = lo[2 * i] | lo[2 * i + 1] << 16;
        }
        uint8_t* dst = p_mem + par * X::kP + tid * 16;
#pragma unroll
        for (int i = 0; i < RP / 8; ++i)
          *reinterpret_cast<uint4*>(dst + i * 2048) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      }
      fence_proxy_async();
      // row sums of p / vs over the warp: halves exchanged, so that lane r ends with row r's (the same tree for every RP)
#pragma unroll
      for (int i = 0; i < RP; ++i) s[i] = __fmul_rn(s[i], iv);
      {
        int off = 16;
#pragma unroll
        for (int n = RP; n > 1; n >>= 1, off >>= 1) {
          const bool up = lane & off;
#pragma unroll
          for (int i = 0; i < n / 2; ++i) {
            const float give = up ? s[i] : s[i + n / 2], keep = up ? s[i + n / 2] : s[i];
            s[i] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, off));
          }
        }
#pragma unroll
        for (; off; off >>= 1) s[0] = __fadd_rn(s[0], __shfl_xor_sync(0xffffffffu, s[0], off));
        constexpr int kRep = 32 / RP;  // lanes with the same row
        if (lane % kRep == 0) s_sum[(par * 4 + warp) * RP + lane / kRep] = s[0];
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(p_full(par));
        mbar_arrive(d_free(ds));
      }
      if (t > 0 && !(fl & kNewSeg)) {
        fold(t - 1);
        if (fail) break;
      }
      prev.flags = fl;
      prev.h = h;
      prev.j0 = j0;
      prev.tile = tile;
      prev.fresh = fresh;
      prev.c0 = c0;
      prev.gi = gi;
#pragma unroll
      for (int c = 0; c < NP; ++c) poison[c] = taint[c];
    }
    if (!fail && t > 0) fold(t - 1);
    if (fail && lane == 0) give_up();
  }

  // ---- teardown: copies and MMAs in flight land before memory is released ----
  __syncthreads();
  if (*s_abort) {
    if (warp == 4) asm volatile("cp.async.wait_all;" ::: "memory");
    if (warp == 4 && lane == 0)
      for (int i = max(0, loads - NS); i < loads; ++i) mbar_wait_parked(full(i % NS), (i / NS) & 1);
    if (warp == 5 && lane == 0) {  // one more commit covers every MMA issued
      umma_commit(drained);
      mbar_wait_parked(drained, 0);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, X::kTmem);
  }
}

// ---- combine -----------------------------------------------------------------------------------
//
// A row's groups, in eight interleaved chains (group i in chain i % 8), then
// ((0+1)+(2+3))+((4+5)+(6+7)).  WIDE: a thread set per chain (long caches, few
// rows); otherwise each thread runs all chains of four columns (many rows of
// few groups).  Reads what the attention kernel wrote a moment ago (L2).

struct State {
  float m, l;
  float4 a;
};

__device__ __forceinline__ void fold_state(State& s, float m, float l, const float4& a) {
  float al, be;
  fold_ml(s.m, s.l, m, l, al, be);
  s.a.x = __fmaf_rn(s.a.x, al, __fmul_rn(a.x, be));
  s.a.y = __fmaf_rn(s.a.y, al, __fmul_rn(a.y, be));
  s.a.z = __fmaf_rn(s.a.z, al, __fmul_rn(a.z, be));
  s.a.w = __fmaf_rn(s.a.w, al, __fmul_rn(a.w, be));
}

template <int D, int RP, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 2 * D : 256) kv_combine_kernel(const __grid_constant__ Params p) {
  constexpr int kLanes = D / 4, kSets = WIDE ? kChains : 256 / kLanes;  // thread sets: chains, or rows
  __shared__ float s_m[kSets][kLanes], s_l[kSets][kLanes];
  __shared__ float4 s_a[WIDE ? kSets : 1][kLanes];
  const int set = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
  const int64_t row = WIDE ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * kSets + set;
  pdl_launch_dependents();
  pdl_wait();
  const State none{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  State out = none;
  if (row < (int64_t)p.T * p.q_heads) {
    const int t = (int)(row / p.q_heads), hq = (int)(row % p.q_heads);
    // the request of row t: the last b with cu[b] <= t
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    bool bad = false;
    const Req r = load_req(p, lo, &bad);
    const int j = t - r.c0;
    if (j >= 0 && j < r.fresh) {
      const int rt = j / p.TQ, h = hq / p.G;
      const int tf = first_tile(p, r, rt), tl = last_tile(p, r, rt);
      const int64_t total = p.starts[p.B];
      const int64_t seg0 = p.starts[lo] + (rt ? tiles_before(p, r, rt) * p.heads : 0) + (int64_t)h * (tl - tf + 1);
      const int g0 = first_tile(p, r, 0) / kGroupTiles;  // slot 0
      const int rr = (j - rt * p.TQ) * p.G + hq % p.G;   // row within the row tile
      auto owner = [&](int64_t x) { return ((x + 1) * p.grid - 1) / total; };  // the CTA whose range holds tile x
      State st[WIDE ? 1 : kChains];
#pragma unroll
      for (int i = 0; i < (WIDE ? 1 : kChains); ++i) st[i] = none;
      auto take = [&](int g, State& s) {  // one group
        const int ta = max(tf, g * kGroupTiles), tb = min(tl, g * kGroupTiles + kGroupTiles - 1);
        const int64_t xa = seg0 + ta - tf, oa = owner(xa), ob = owner(seg0 + tb - tf);
        if (oa == ob) {
          const int64_t at = ((int64_t)(g - g0) * p.T + t) * p.q_heads + hq;
          const float2 ml = p.g_ml[at];
          fold_state(s, ml.x, ml.y, *reinterpret_cast<const float4*>(p.g_acc + at * D + 4 * c));
        } else {
          State gs = none;
          for (int k = ta; k <= tb; ++k) {
            const int64_t o = owner(xa + k - ta);
            // at the owner's end unless the group began in an earlier range
            const int64_t at = ((o * 2 + (o == oa ? 1 : 0)) * kGroupTiles + k % kGroupTiles) * RP + rr;
            const float2 ml = p.t_ml[at];
            fold_state(gs, ml.x, ml.y, *reinterpret_cast<const float4*>(p.t_acc + at * D + 4 * c));
          }
          fold_state(s, gs.m, gs.l, gs.a);
        }
      };
      const int ga = tf / kGroupTiles, gb = tl / kGroupTiles;
      if (WIDE) {
        for (int g = ga + ((set - ga) & (kChains - 1)); g <= gb; g += kChains) take(g, st[0]);
        out = st[0];
      } else {
        for (int gg = ga & ~(kChains - 1); gg <= gb; gg += kChains)
#pragma unroll
          for (int i = 0; i < kChains; ++i)
            if (gg + i >= ga && gg + i <= gb) take(gg + i, st[i]);
#pragma unroll
        for (int n = 1; n < kChains; n <<= 1)
#pragma unroll
          for (int i = 0; i + n < (WIDE ? 1 : kChains); i += 2 * n) fold_state(st[i], st[i + n].m, st[i + n].l, st[i + n].a);
        out = st[0];
      }
    }
  }
  if (WIDE) {
    s_m[set][c] = out.m;
    s_l[set][c] = out.l;
    s_a[set][c] = out.a;
    __syncthreads();
    if (set != 0) return;
    State st[kChains];
#pragma unroll
    for (int i = 0; i < kChains; ++i) st[i] = State{s_m[i][c], s_l[i][c], s_a[i][c]};
#pragma unroll
    for (int n = 1; n < kChains; n <<= 1)
#pragma unroll
      for (int i = 0; i + n < kChains; i += 2 * n) fold_state(st[i], st[i + n].m, st[i + n].l, st[i + n].a);
    out = st[0];
  }
  if (row < (int64_t)p.T * p.q_heads) {
    const bool any = out.l != 0.f;  // (NaN: yes)
    uint2 w;
    w.x = (uint32_t)f32_to_bf16_bits(any ? __fdiv_rn(out.a.x, out.l) : 0.f) |
          (uint32_t)f32_to_bf16_bits(any ? __fdiv_rn(out.a.y, out.l) : 0.f) << 16;
    w.y = (uint32_t)f32_to_bf16_bits(any ? __fdiv_rn(out.a.z, out.l) : 0.f) |
          (uint32_t)f32_to_bf16_bits(any ? __fdiv_rn(out.a.w, out.l) : 0.f) << 16;
    *reinterpret_cast<uint2*>(p.out + row * D + 4 * c) = w;
  }
}

// ---- host side -----------------------------------------------------------------------------------

struct Layout {
  int RP, TQ, gmax, grid;
  size_t starts, g_acc, g_ml, t_acc, t_ml, bytes;
};

int ctas_per_sm(int dim, int RP) { return dim == 256 && RP > 8 ? 1 : 2; }

Layout make_layout(int B, int T, int q_heads, int heads, int dim, int max_new, int max_len, int window) {
  Layout y;
  const int G = q_heads / heads;
  if (max_new > T) max_new = T;
  const int64_t rows = (int64_t)G * max_new;
  y.RP = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
  if (y.RP < G) y.RP = G <= 16 ? 16 : 32;
  y.TQ = y.RP / G;
  int64_t groups = ((int64_t)max_len + kTile * kGroupTiles - 1) / (kTile * kGroupTiles);
  if (window > 0) {
    const int64_t span = ((int64_t)window + max_new - 2) / (kTile * kGroupTiles) + 2;
    if (span < groups) groups = span;
  }
  y.gmax = (int)groups;
  // no more CTAs than tiles
  const int64_t per = ((int64_t)max_len + kTile - 1) / kTile;
  const int64_t most = (int64_t)(T < B ? T : B) * heads * (((int64_t)max_new + y.TQ - 1) / y.TQ) * per;
  const int full = kSms * ctas_per_sm(dim, y.RP);
  y.grid = most < full ? (int)most : full;
  auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
  y.starts = 0;
  y.g_acc = up(8 * ((size_t)B + 1));
  y.g_ml = y.g_acc + up((size_t)y.gmax * T * q_heads * dim * 4);
  y.t_acc = y.g_ml + up((size_t)y.gmax * T * q_heads * 8);
  y.t_ml = y.t_acc + up((size_t)y.grid * 2 * kGroupTiles * y.RP * dim * 4);
  y.bytes = y.t_ml + up((size_t)y.grid * 2 * kGroupTiles * y.RP * 8);
  return y;
}

std::mutex g_attr_mu;
bool g_attr[64][9] = {};

template <int D, int RP>
cudaError_t run(const KvAttentionArgs& a, const Layout& y, const Params& p, int pdl, cudaStream_t s) {
  using X = Geo<D, RP>;
  static_assert(X::kCtas == (D == 256 && RP > 8 ? 1 : 2), "ctas_per_sm");
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(g_attr_mu);
    bool& done = g_attr[dev][(D == 64 ? 0 : D == 128 ? 3 : 6) + (RP == 8 ? 0 : RP == 16 ? 1 : 2)];
    if (!done) {
      if (cudaError_t e = cudaFuncSetAttribute(kv_attention_kernel<D, RP>, cudaFuncAttributeMaxDynamicSharedMemorySize, X::kSmem))
        return e;
      done = true;
    }
  }
  Maps maps;
  const int64_t rows = (int64_t)a.cache.blocks * a.cache.heads * a.cache.block;
  const auto sw = D < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  const int inner = D < 128 ? D : 128;
  if (cudaError_t e = encode_map_2d(&maps.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.cache.k, D, rows, D, inner, a.cache.block, sw)) return e;
  if (cudaError_t e = encode_map_2d(&maps.v, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.cache.v, D, rows, D, inner, a.cache.block, sw)) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl > 0 ? 1 : 0;
  cfg.stream = s;
  cfg.gridDim = dim3((unsigned)y.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)X::kSmem;
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, kv_attention_kernel<D, RP>, maps, p)) return e;
  const int64_t out_rows = (int64_t)a.T * a.q_heads;
  cfg.dynamicSmemBytes = 0;
  // few rows of many groups: a thread set per chain; else a thread runs all chains
  if (y.gmax > kChains && out_rows <= 4096) {
    cfg.gridDim = dim3((unsigned)out_rows);
    cfg.blockDim = dim3(2 * D);
    return cudaLaunchKernelEx(&cfg, kv_combine_kernel<D, RP, true>, p);
  }
  constexpr int kRowsPer = 256 / (D / 4);
  cfg.gridDim = dim3((unsigned)((out_rows + kRowsPer - 1) / kRowsPer));
  cfg.blockDim = dim3(256);
  return cudaLaunchKernelEx(&cfg, kv_combine_kernel<D, RP, false>, p);
}

template <int D>
cudaError_t run_d(const KvAttentionArgs& a, const Layout& y, const Params& p, int pdl, cudaStream_t s) {
  switch (y.RP) {
    case 8: return run<D, 8>(a, y, p, pdl, s);
    case 16: return run<D, 16>(a, y, p, pdl, s);
    default: return run<D, 32>(a, y, p, pdl, s);
  }
}

}  // namespace

size_t kv_attention_workspace(int B, int T, int q_heads, int kv_heads, int dim, int max_new, int max_len, int window) {
  return make_layout(B, T, q_heads, kv_heads, dim, max_new, max_len, window).bytes;
}

cudaError_t launch_kv_attention(const KvAttentionArgs& a, int pdl, cudaStream_t s) {
  const Layout y = make_layout(a.B, a.T, a.q_heads, a.cache.heads, a.cache.dim, a.max_new, a.max_len, a.window);
  uint8_t* w = static_cast<uint8_t*>(a.ws);
  Params p;
  p.q = a.q;
  p.q_stride = a.q_stride;
  p.k_scale = a.cache.k_scale;
  p.v_scale = a.cache.v_scale;
  p.table = a.table;
  p.cu = a.cu;
  p.lens = a.lens;
  p.out = a.out;
  p.B = a.B;
  p.T = a.T;
  p.q_heads = a.q_heads;
  p.heads = a.cache.heads;
  p.G = a.q_heads / a.cache.heads;
  p.TQ = y.TQ;
  p.blocks = a.cache.blocks;
  p.shift = __builtin_ctz((unsigned)a.cache.block);
  p.max_blocks = a.max_blocks;
  p.max_new = a.max_new < a.T ? a.max_new : a.T;
  p.max_len = a.max_len;
  p.window = a.window;
  p.qk_scale = a.scale * kLog2e;
  p.gmax = y.gmax;
  p.grid = y.grid;
  p.starts = reinterpret_cast<int64_t*>(w + y.starts);
  p.g_acc = reinterpret_cast<float*>(w + y.g_acc);
  p.g_ml = reinterpret_cast<float2*>(w + y.g_ml);
  p.t_acc = reinterpret_cast<float*>(w + y.t_acc);
  p.t_ml = reinterpret_cast<float2*>(w + y.t_ml);
  p.flags = a.flags;
  switch (a.cache.dim) {
    case 64: return run_d<64>(a, y, p, pdl, s);
    case 128: return run_d<128>(a, y, p, pdl, s);
    default: return run_d<256>(a, y, p, pdl, s);
  }
}

}  // namespace w4a16
