// fp4_pair.cu -- the product of microscaled 4-bit matrices for many activation
// rows: tiles of 256 rows of x by up to 256 rows of W on pairs of SMs.
//
// The arithmetic is fp4_mm.cu's.  Here x is the MMA's M: a tensor-memory lane
// is a row of x and the columns run along y's row, so that a thread holds
// neighbours of y (stores of 32 bytes; gate and up of a pair side by side).
// tcgen05.mma.cta_group::2 multiplies 256 rows of x (128 in each CTA) with TN
// rows of W (half of them in each CTA's shared memory): a CTA takes 38 KB from
// L2 for each 128 x 256 x 256 products, half of what one alone would.
//
// CTA: fourteen warps, persistent over tiles.
//   warp 0     TMA producer of this CTA's x and W rows and their scales
//   warp 1     leader: scales from shared to tensor memory of both CTAs, MMAs
//              and commits; the other CTA: passes "stage landed" on
//   warps 2-13 epilogue: 32 lanes x a third of the columns each
// Few tiles and a long K: clusters of two or four pairs share a tile (SPLIT).
// Tensor memory: two accumulators of 256 columns that share 160 (mx: 128), beside
// three sets of scales of 48 columns (mx: five of 24).  A set is written again
// when the MMAs that read it are done; with two sets the MMAs waited for the
// copies.  The epilogue takes the shared columns into registers first, and lets
// the next tile's MMAs go when it has them.
// Waits are bounded as in fp4_mm.cu; the two CTAs leave together.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "fp4.cuh"
#include "fp4_mm.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace w4a16 {
namespace {

using namespace ptx;

constexpr int kXTile = 128 * 128;  // 16 KB: this CTA's 128 rows of x
constexpr int kWTile = 128 * 128;  // its half of W's rows (up to 128)
constexpr int kEpi = 12;  // epilogue warps, three for each 32 lanes
constexpr int kThreads = 32 * (2 + kEpi);
// Tensor memory's columns: two accumulators of 256, the second from kAccStep on, then the scale sets (a stage's atoms of
// x's scales, 4 columns each, and of W's, 8).
template <int FMT>
struct Geo {
  static constexpr int kAtoms = FMT == W4A16_FP4_MX ? 2 : 4;  // of a stage
  static constexpr int kXScale = kAtoms * kFp4Atom, kWScale = 2 * kXScale;
  static constexpr int kStage = kXTile + kWTile + kXScale + kWScale;
  static constexpr int kStages = 5;
  static constexpr int kBars = 2 * kStages + 7;
  static constexpr int kSmem = kStages * kStage + kEpi * 384 + kBars * 8 + 16;
  static constexpr int kSet = 12 * kAtoms;
  static constexpr int kSets = FMT == W4A16_FP4_MX ? 5 : 3;
  static constexpr int kAccStep = FMT == W4A16_FP4_MX ? 128 : 96;
  static constexpr int kSetsAt = kAccStep + 256;
  static constexpr int kShared = 8 - kAccStep / 32;  // 32s of columns that both accumulators have
  static_assert(kSetsAt + kSets * kSet <= 512 && kShared <= 6, "the SM's tensor memory");
  // Of an SM's 256 KB the L1 gets what shared memory's 196 or 228 KB leave, and the next call's quantiser needs it (4096 x
  // 10240 x 2560, nv: 49.7 us, with 1 KB more 51.6; mx with six stages 46.3, with five 45.1, though 8192 x 16384 x 16384 takes
  // 583 and with six 575).
  static_assert(kSmem + 1024 <= 196 * 1024, "a CTA's shared memory, with the system's 1 KB");
};

struct Maps {
  CUtensorMap w;  // u8 [experts * N][K / 2], box 128 bytes x TN / 2 rows, 128-byte swizzle
  CUtensorMap x;  // u8 [x rows][K / 2], box 128 bytes x 128 rows
  CUtensorMap ws;  // scales, boxes of two row tiles
  CUtensorMap xs;  // ... of one
};

struct PairParams {
  Fp4MmParams p;
  int tn;       // rows of W per tile: 128, 192 or 256
  int n_tiles;  // tiles along W's rows
};

// (a, b) times (x, y) and f, two products at a time.
__device__ __forceinline__ void mul2(float& a, float& b, float x, float y, float f) {
  asm("{ .reg .b64 p, q, r; mov.b64 p, {%0, %1}; mov.b64 q, {%2, %3}; mov.b64 r, {%4, %4};\n"
      "mul.rn.f32x2 q, q, r; mul.rn.f32x2 p, p, q; mov.b64 {%0, %1}, p; }"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y), "f"(f));
}

// Which tile a pair's unit is: sixteen activation tiles by all of W's, then the next sixteen, so that the pairs at work at
// a time share what they read (8192 x 16384 x 16384 with 4 / 8 / 16: 641 / 596 / 586 us).
__device__ __forceinline__ void unit_tile(int64_t u, int x_tiles, int n_tiles, int& xt, int& nt) {
  const int64_t per = 16LL * n_tiles;
  const int g = (int)(u / per), r = (int)(u % per);
  const int wide = min(16, x_tiles - 16 * g);
  xt = 16 * g + r % wide;
  nt = r / wide;
}

// A thread's row of a tile.
struct Rows {
  int64_t m, expert, cols;  // row and columns of y
  float fx;
  int n0;  // the tile's first row of W
  bool mine, factors;
  bool plain;  // all factors of x and W that an epilogue warp has of the tile have products that are normal numbers
  Rows() = default;
  __device__ __forceinline__ Rows(const Fp4MmParams& p, const PairParams& pp, int64_t u, int x_tiles, int r) {
    int xt, nt;
    unit_tile(u, x_tiles, pp.n_tiles, xt, nt);
    n0 = nt * pp.tn;
    expert = 0;
    int place = xt * 256, count = p.M - place;
    if (p.tiles) {
      expert = p.tiles[xt].expert;
      place = p.tiles[xt].place;
      count = p.tiles[xt].count;
    }
    mine = r < count;
    m = mine ? (p.row ? p.row[place + r] : place + r) : 0;
    fx = mine && p.xf ? p.xf[place + r] : 1.0f;
    cols = p.act == W4A16_FP4_LINEAR ? p.N : p.N / 2;
    factors = p.wf || p.xf;
    plain = true;
  }
  __device__ __forceinline__ float wf(const Fp4MmParams& p, int n) const { return !p.wf ? 1.0f : n < p.N ? p.wf[expert * p.N + n] : 1.0f; }
  // lo, hi: the least and the largest of those factors' magnitudes, as bits, that this lane holds.  Whole warps, and one answer
  // for them: what follows has instructions that a warp executes together.
  __device__ __forceinline__ void span(uint32_t lo, uint32_t hi) {
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    plain = __all_sync(0xffffffffu, fp4_normal(__uint_as_float(lo) * fx) && fp4_normal(__uint_as_float(hi) * fx));
  }
};

// 32 sums of a thread's row, from row n0 of W on, to y; wf: W's factors for them.  A lane stores 32 bytes of its row at a
// time: whole sectors.  (4096 x 10240 x 2560, us: 45 so, 62 in stores of 16 bytes, 50 turned through shared memory to 64
// bytes a row.)
__device__ __forceinline__ void put32(const Fp4MmParams& p, const Rows& row, const float* wf, int n0, float (&v)[32]) {
  if (row.factors) {
    if (__builtin_expect(row.plain, 1)) {
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 f = *reinterpret_cast<const float4*>(wf + j);
        mul2(v[j], v[j + 1], f.x, f.y, row.fx);
        mul2(v[j + 2], v[j + 3], f.z, f.w, row.fx);
      }
    } else {
      // (a loop over a copy: unrolled three times, its instructions cost all other calls 0.1 to 0.3 us)
      float u[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) u[j] = v[j];
#pragma unroll 1
      for (int j = 0; j < 32; ++j) u[j] = fp4_scaled(u[j], wf[j], row.fx);
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = u[j];
    }
  }
  const bool linear = p.act == W4A16_FP4_LINEAR;
  uint32_t o[16];
  if (linear) {
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] = fp4_bf16x2(v[2 * j], v[2 * j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      o[j] = fp4_bf16x2(fp4_activate(v[4 * j], p.act) * v[4 * j + 1], fp4_activate(v[4 * j + 2], p.act) * v[4 * j + 3]);
  }
  if (!row.mine) return;
  uint16_t* y = p.y + row.m * row.cols + (linear ? n0 : n0 / 2);
  const bool whole = n0 + 32 <= p.N;
  if (whole && p.vec == 32) {
    // (past the L1, which has little room here: 4096 x 10240 x 2560, nv, 48.2 us, else 49.8)
    st_past_v8(y, o);
    if (linear) st_past_v8(y + 16, o + 8);
  } else if (whole && p.vec == 16) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (linear || j < 2) *reinterpret_cast<uint4*>(y + 8 * j) = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
  } else {
    const int left = (linear ? p.N - n0 : (p.N - n0) / 2);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if (linear || j < 8) {
        if (2 * j < left) y[2 * j] = (uint16_t)o[j];
        if (2 * j + 1 < left) y[2 * j + 1] = (uint16_t)(o[j] >> 16);
      }
    }
  }
}

// SPLIT: clusters of p.split pairs share a tile's K, one tile each.  Each pair's partial sums go to the pairs that add them
// up, every split-th 32 of the columns to one, through distributed shared memory in the stages' place; they are added in
// the order of K.
template <int FMT, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) fp4_pair_kernel(const __grid_constant__ Maps maps, PairParams pp) {
  using T = Geo<FMT>;
  constexpr int kAtoms = T::kAtoms, kSets = T::kSets, S = T::kStages, kStage = T::kStage;
  const Fp4MmParams& p = pp.p;
  extern __shared__ __align__(1024) uint8_t base[];  // (the tiles' swizzle counts from multiples of 1024)
  const uint32_t sb = smem_u32(base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = SPLIT ? p.split : 1;
  const uint32_t in_cluster = cluster_rank(), rank = in_cluster & 1, lead = in_cluster & ~1u;  // of the pair; its leader
  const int part = (int)(in_cluster >> 1);  // which part of K
  const uint32_t bars = sb + S * kStage + kEpi * 384;
  float* s_wf = reinterpret_cast<float*>(base + S * kStage);  // W's factors for an epilogue warp's columns: three 32s each
  auto X_of = [&](int s) { return sb + (uint32_t)(s * kStage); };
  auto W_of = [&](int s) { return X_of(s) + kXTile; };
  auto SX_of = [&](int s) { return W_of(s) + kWTile; };
  auto SW_of = [&](int s) { return SX_of(s) + T::kXScale; };
  auto full = [&](int s) { return bars + 8u * s; };         // this CTA's copies landed; leader: the other CTA's too
  auto empty = [&](int s) { return bars + 8u * (S + s); };  // the MMAs are done with it (both CTAs)
  auto acc_full = [&](int b) { return bars + 8u * (2 * S + b); };
  auto acc_free = [&](int b) { return bars + 8u * (2 * S + 2 + b); };   // leader: all of it read, by both CTAs
  auto part_free = [&](int b) { return bars + 8u * (2 * S + 4 + b); };  // leader: the shared columns read
  const uint32_t sums = bars + 8u * (2 * S + 6);  // SPLIT: the other parts' sums of this pair's columns landed
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(base + (bars - sb) + 8 * T::kBars);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);

  const int64_t first = blockIdx.x / (2u * split), step = gridDim.x / (2u * split);
  const int k0 = SPLIT ? p.stages * part / split : 0, k1 = SPLIT ? p.stages * (part + 1) / split : p.stages, tn = pp.tn;
  const uint32_t limit = p.fault_wait ? 4096u : 1u << 18;  // tries of a wait: about a second
  auto timeout = [&]() {
    atomicOr(p.flags, W4A16_DEVICE_TIMEOUT);
    *s_abort = 1;
  };
  // what a unit's stages are loaded from
  int x_row = 0, xs_tile = 0, w_row = 0, ws_tile = 0;
  auto locate = [&](int64_t u, int x_tiles) {
    int xt, nt;
    unit_tile(u, x_tiles, pp.n_tiles, xt, nt);
    int64_t expert = 0;
    x_row = xt * 256;
    if (p.tiles) {
      expert = p.tiles[xt].expert;
      x_row = p.tiles[xt].place;
    }
    x_row += 128 * (int)rank;
    xs_tile = x_row / kFp4Rows;
    w_row = (int)(expert * p.N) + nt * tn + (int)rank * (tn / 2);
    ws_tile = (int)(expert * p.row_tiles) + nt * tn / 128;  // (the tile's rows of W touch one or two 128-row tiles of scales)
  };
  auto load = [&](int s, int k) {
    const uint64_t keep = policy_evict_last();
    mbar_expect_tx(full(s), kXTile + (uint32_t)(tn / 2) * 128 + 3 * kAtoms * kFp4Atom);
    tma_load_2d(X_of(s), &maps.x, k * 128, x_row, full(s), keep);
    tma_load_2d(W_of(s), &maps.w, k * 128, w_row, full(s), keep);
    tma_load_3d(SX_of(s), &maps.xs, 0, k * kAtoms, xs_tile, full(s), keep);
    tma_load_3d(SW_of(s), &maps.ws, 0, k * kAtoms, ws_tile, full(s), keep);
  };
  uint32_t it = 0;  // stages so far

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      // (debug: an arrival that never comes)
      mbar_init(full(s), (rank == 0 ? 2 : 1) + (p.fault_wait && blockIdx.x == 0 && s == 0));
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_free(b), 2 * kEpi);
      mbar_init(part_free(b), 2 * kEpi);
    }
    if (SPLIT) mbar_init(sums, 1);
    *s_abort = 0;
    fence_barrier_init();
    fence_proxy_async();
  }
  if (warp == 1) {
    tmem_alloc2(smem_u32(s_tmem), 512);
    tmem_relinquish2();
  }
  tc_fence_before_sync();
  __syncwarp();
  cluster_arrive();
  if (threadIdx.x == 0) {
    // (The first stages are asked for before the cluster has met: they concern this CTA alone.  130 rows to 10240 x 2560:
    // 7.5 us, else 8.0; between this thread's barriers and the others' start, 8.7.)
    pdl_wait();
    const int x_tiles = p.tiles ? *p.tile_count : p.x_tiles;
    if (first < (int64_t)x_tiles * pp.n_tiles) {
      locate(first, x_tiles);
      for (; it < S && k0 + (int)it < k1; ++it) load((int)it, k0 + (int)it);
    }
  }
  __syncwarp();
  cluster_wait();
  tc_fence_after_sync();
  // (all 512 columns of tensor memory: they begin at 0, and the addresses below are constants)
  pdl_launch_dependents();
  pdl_wait();
  const int x_tiles = p.tiles ? *p.tile_count : p.x_tiles;
  const int64_t units = (int64_t)x_tiles * pp.n_tiles;

  Rows split_row{};

  if (warp == 0) {
    // ---- TMA producer ----
    if (lane == 0) {
      int k = k0 + (int)it;  // (those of the first unit that are on their way)
      for (int64_t u = first; u < units && !*s_abort; u += step, k = k0) {
        locate(u, x_tiles);
        for (; k < k1; ++k, ++it) {
          const int s = (int)(it % S);
          if (it >= (uint32_t)S && !mbar_wait_parked(empty(s), ((it / S) - 1) & 1, 1000, limit)) {
            timeout();
            break;
          }
          load(s, k);
        }
      }
      // (every arrival that the MMAs send here has come before this CTA may leave)
      for (uint32_t i = it > (uint32_t)S ? it - S : 0; i < it && !*s_abort; ++i)
        if (!mbar_wait_parked(empty((int)(i % S)), (i / S) & 1, 1000, limit)) timeout();
    }
  } else if (warp == 1 && rank == 0) {
    // ---- leader: scales and MMAs ----
    const uint32_t go = elect_one();
    const uint16_t both = (uint16_t)(3u << lead);
    const uint32_t idesc = umma_idesc_e2m1(256, tn, FMT == W4A16_FP4_MX);
    const uint64_t xd0 = umma_desc_sw128(X_of(0)), wd0 = umma_desc_sw128(W_of(0));
    const uint64_t sx0 = umma_desc(SX_of(0), 128, 128, 0), sw0 = umma_desc(SW_of(0), 128, 128, 0);
    uint32_t n = 0;                     // tiles
    int s = 0, set = 0, old = S - kSets;  // slot, scale set, and the slot of kSets stages before
    uint32_t parity = 0, old_parity = 1;
    for (int64_t u = first; u < units && !*s_abort; u += step, ++n) {
      int xt, nt;
      unit_tile(u, x_tiles, pp.n_tiles, xt, nt);
      const int b = (int)(n & 1);
      // this accumulator's last tile is read, and the columns it shares with the other's
      if ((n >= 2 && !mbar_wait_warp(acc_free(b), ((n >> 1) - 1) & 1, limit)) ||
          (n >= 1 && !mbar_wait_warp(part_free(b ^ 1), ((n - 1) >> 1) & 1, limit))) {
        if (lane == 0) timeout();
        break;
      }
      tc_fence_after_sync();
      const uint32_t acc = (uint32_t)(b * T::kAccStep);
      const uint32_t w_col = (uint32_t)(nt * tn % 128 / 32);
      bool ok = true;
      for (int k = k0; k < k1; ++k, ++it) {
        ok = mbar_wait_warp(full(s), parity, limit) &&
             (kSets >= S || it < (uint32_t)kSets || mbar_wait_warp(empty(old), old_parity, limit));
        if (!ok) {
          if (lane == 0) timeout();
          break;
        }
        tc_fence_after_sync();
        const uint64_t at = (uint64_t)(uint32_t)(s * (kStage >> 4));
        const uint64_t xd = xd0 + at, wd = wd0 + at, sx = sx0 + at, sw = sw0 + at;
        const uint32_t cx = (uint32_t)(T::kSetsAt + set * T::kSet), cw = cx + 4 * kAtoms;
        const int atoms = p.atoms - k * kAtoms, steps = (p.K - k * kFp4StageK + 63) / 64;
        auto copy = [&](int a) {
          tmem_copy_scales2(cx + 4 * a, sx + (uint64_t)(a * (kFp4Atom >> 4)));
          tmem_copy_scales2(cw + 8 * a, sw + (uint64_t)(a * (kFp4Atom >> 4)));
          tmem_copy_scales2(cw + 8 * a + 4, sw + (uint64_t)((kAtoms + a) * (kFp4Atom >> 4)));
        };
        auto mma = [&](int j) {
          if (FMT == W4A16_FP4_MX)
            umma2_mxf4(acc, xd + 2 * j, wd + 2 * j, idesc | umma_idesc_scale_byte(2 * (j & 1)), cx + 4 * (j / 2),
                       cw + 8 * (j / 2) + w_col, k > k0 || j > 0);
          else
            umma2_nvf4(acc, xd + 2 * j, wd + 2 * j, idesc, cx + 4 * j, cw + 8 * j + w_col, k > k0 || j > 0);
        };
        if (elect_one()) {
          if (steps >= 4) {
#pragma unroll
            for (int a = 0; a < kAtoms; ++a) copy(a);
#pragma unroll
            for (int j = 0; j < 4; ++j) mma(j);
          } else {  // the end of K
#pragma unroll
            for (int a = 0; a < kAtoms; ++a)
              if (a < atoms) copy(a);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j < steps) mma(j);
          }
        }
        umma_commit2_if(go, empty(s), both);
        if (++s == S) s = 0, parity ^= 1;
        if (++old == S) old = 0, old_parity ^= 1;
        if (++set == kSets) set = 0;
      }
      if (!ok) break;
      umma_commit2_if(go, acc_full(b), both);
    }
  } else if (warp == 1) {
    // ---- the other CTA: its stages landed ----
    const uint32_t to = cluster_map(bars, lead) - bars;
    for (int64_t u = first; u < units && !*s_abort; u += step) {
      bool ok = true;
      for (int k = k0; k < k1; ++k, ++it) {
        const int s = (int)(it % S);
        if (!(ok = mbar_wait_warp(full(s), (it / S) & 1, limit))) break;
        if (lane == 0) mbar_arrive_cluster(full(s) + to);
      }
      if (!ok) {
        if (lane == 0) timeout();
        break;
      }
    }
  } else {
    // ---- epilogue ----
    const int q = warp & 3, third = (warp - 2) >> 2;
    const uint32_t to = cluster_map(bars, lead) - bars;
    uint32_t n = 0;
    if (SPLIT && first < units) split_row = Rows(p, pp, first, x_tiles, 128 * (int)rank + 32 * q + lane);
    for (int64_t u = first; u < units && !*s_abort; u += step, ++n) {
      const int b = (int)(n & 1);
      if (SPLIT) {  // (the rest below)
        uint32_t lo = 0x3F800000u, hi = lo;
        for (int c = part + split * third, i = 0; c < tn / 32; c += 3 * split, ++i) {
          const float f = split_row.wf(p, split_row.n0 + 32 * c + lane);
          s_wf[96 * (warp - 2) + 32 * i + lane] = f;
          lo = min(lo, __float_as_uint(fabsf(f)));
          hi = max(hi, __float_as_uint(fabsf(f)));
        }
        split_row.span(lo, hi);
        if (!mbar_wait_warp(acc_full(0), 0, limit + (uint32_t)p.stages) && lane == 0) timeout();
        break;
      }
      Rows o(p, pp, u, x_tiles, 128 * (int)rank + 32 * q + lane);
      float* wf = s_wf + 96 * (warp - 2);
      // The i-th 32 columns to be read, those that both accumulators have first: the second's first and the first's last
      // ones.  Each of the three warps of 32 lanes takes every third.
      auto column = [&](int i) { return 32 * (b ? i : (i + T::kAccStep / 32) % 8); };
      if (o.factors) {
        uint32_t lo = 0x3F800000u, hi = lo;
        __syncwarp();
#pragma unroll
        for (int g = 0; g < 3; ++g) {
          const float f = o.wf(p, o.n0 + column(third + 3 * g) + lane);
          wf[32 * g + lane] = f;
          lo = min(lo, __float_as_uint(fabsf(f)));
          hi = max(hi, __float_as_uint(fabsf(f)));
        }
        __syncwarp();
        o.span(lo, hi);
      }
      if (!mbar_wait_warp(acc_full(b), (n >> 1) & 1, limit + (uint32_t)p.stages)) {
        if (lane == 0) timeout();
        break;
      }
      tc_fence_after_sync();
      const uint32_t acc = (uint32_t)(b * T::kAccStep) + ((uint32_t)(32 * q) << 16);
      auto exists = [&](int i) { return i < 8 && column(i) < tn && o.n0 + column(i) < p.N; };
      auto put = [&](int i, float (&v)[32]) {
        if (exists(i)) put32(p, o, wf + 32 * (i / 3), o.n0 + column(i), v);
        __syncwarp();  // (rows that are not stored are back for the next load)
      };
      // (only where a tile comes that waits for it: no arrival is on its way to a CTA that may be gone)
      auto arrive = [&](uint32_t bar, int64_t next) {
        tc_fence_before_sync();
        __syncwarp();
        if (next < units && lane == 0) mbar_arrive_cluster(bar + to);
      };
      // this warp's 32s: third, third + 3, third + 6; the first is always shared, the second may be
      float v[32], w[32];
      const bool two = third + 3 < T::kShared;
      if (exists(third)) tmem_ld32(acc + column(third), v);
      if (two && exists(third + 3)) tmem_ld32(acc + column(third + 3), w);
      tmem_wait_ld();
      arrive(part_free(b), u + step);
      put(third, v);
      if (!two && exists(third + 3)) tmem_ld32(acc + column(third + 3), w);
      if (exists(third + 6)) tmem_ld32(acc + column(third + 6), v);
      tmem_wait_ld();
      arrive(acc_free(b), u + 2 * step);
      put(third + 3, w);
      put(third + 6, v);
    }
  }

  if (SPLIT) {
    // ---- partial sums to the CTAs that add them up ----
    // By way of this CTA's stages, whose MMAs are done, into the others', once theirs are.  Copies of 4 KB (32 rows x 32
    // columns, four columns after four): as stores of 16 bytes to the other CTA, and a barrier that waits for them, 1.5 us
    // more.  A CTA that gave up sends nothing, and takes part in the rest.
    __syncthreads();
    const int q = warp & 3, third = (warp - 2) >> 2;
    const bool epilogue = first < units && warp >= 2, live = epilogue && !*s_abort;
    const uint32_t acc = (uint32_t)(32 * q) << 16;
    const int n0 = split_row.n0, chunks = min(tn, p.N - n0 + 31) / 32, most = (tn / 32 + split - 1) / split;  // 32s of columns that are there; of one pair
    auto place = [&](int g, int owner, int c) { return sb + (uint32_t)((((g - (g > owner)) * most + c / split) * 4 + q) * 4096); };
    auto staged = [&](int c) { return sb + (uint32_t)((((split - 1) * most + c - (c > part ? (c - part + split - 1) / split : 0)) * 4 + q) * 4096); };
    tc_fence_after_sync();
    if (live) {
#pragma unroll 1
      for (int c = third; c < chunks; c += 3) {
        if (c % split == part) continue;
        float v[32];
        tmem_ld32(acc + 32 * c, v);
        tmem_wait_ld();
        const uint32_t at = staged(c) + 16 * lane;
#pragma unroll
        for (int j = 0; j < 8; ++j) sts128f(at + 512 * j, v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      }
      fence_proxy_async();
    }
    __syncwarp();
    cluster_arrive_relaxed();
    cluster_wait();
    if (epilogue) {
      if (warp == 2 && lane == 0) mbar_expect_tx(sums, (uint32_t)((split - 1) * ((chunks - part + split - 1) / split) * 16384));
      if (live && lane == 0)
        for (int c = third; c < chunks; c += 3) {
          const int owner = c % split;
          const uint32_t cta = (uint32_t)(2 * owner) + rank;
          if (owner != part) bulk_copy_cluster(cluster_map(place(part, owner, c), cta), staged(c), 4096, cluster_map(sums, cta));
        }
      __syncwarp();
      if (!mbar_wait_warp(sums, 0, limit)) {
        if (lane == 0) timeout();
      } else if (live) {
#pragma unroll 1
        for (int c = part + split * third, i = 0; c < chunks; c += 3 * split, ++i) {
          float v[32], own[32];
          tmem_ld32(acc + 32 * c, own);
          tmem_wait_ld();
          for (int g = 0; g < split; ++g) {
            const uint32_t at = place(g, part, c) + 16 * lane;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 f = g == part ? make_float4(own[4 * j], own[4 * j + 1], own[4 * j + 2], own[4 * j + 3]) : lds128f(at + 512 * j);
              v[4 * j] = g ? v[4 * j] + f.x : f.x;
              v[4 * j + 1] = g ? v[4 * j + 1] + f.y : f.y;
              v[4 * j + 2] = g ? v[4 * j + 2] + f.z : f.z;
              v[4 * j + 3] = g ? v[4 * j + 3] + f.w : f.w;
            }
          }
          put32(p, split_row, s_wf + 96 * (warp - 2) + 32 * i, n0 + 32 * c, v);
          __syncwarp();
        }
      }
    }
  }

  // ---- teardown: everything in flight lands before the memories are released ----
  __syncthreads();
  if (*s_abort) {
    if (warp == 0 && lane == 0)
      for (uint32_t i = it > (uint32_t)S ? it - S : 0; i < it; ++i) mbar_wait_parked(full((int)(i % S)), (i / S) & 1, 1000, limit);
    if (warp == 1 && rank == 0 && it > 0) mbar_wait_warp(empty((int)((it - 1) % S)), ((it - 1) / S) & 1, limit);
  }
  tc_fence_before_sync();
  __syncthreads();
  // The other CTA's memories are read by this one's MMAs: neither leaves before both are done.  What one tells the other
  // of has been waited for, y's stores need not be (a release here waits 1 us for them).
  if (*s_abort) cluster_arrive();
  else cluster_arrive_relaxed();
  cluster_wait();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc2(*s_tmem, 512);
  }
}

// ---- host side ------------------------------------------------------------------------

constexpr int kPairs = 76;  // of SMs
constexpr int kMaxSplit = 4;
// Whether the partial sums that come and go have room in the stages: at most `most` 32s of columns from each other pair come,
// at most all but one of the smallest share go.
bool split_fits(int split, int tn, int stage_bytes) {
  const int chunks = tn / 32, most = (chunks + split - 1) / split;
  return ((split - 1) * most + chunks - chunks / split) * 16384 <= stage_bytes;
}
// What the exchange of a split tile's sums costs, where a stage costs tn + 64 (0.36 us at 256): 2 us.  nv, us with 1 / 2 / 4
// pairs a tile: K = 10240, N = 2560: 130 rows 14.3 / 11.1 / 11.0, 300 rows 14.7 / 12.4 / -, 512 rows 14.9 / 12.9 / -; K = 2560,
// N = 2560, 256 rows 6.5 / 7.4 / -.
constexpr int kExchange = 1800;

std::mutex g_mu;
int g_sms[64] = {};
bool g_attr[64][4] = {};

template <int FMT, bool SPLIT>
cudaError_t launch_t(const Fp4MmArgs& a, const PairParams& p, int64_t units, int pdl, cudaStream_t s) {
  auto* fn = fp4_pair_kernel<FMT, SPLIT>;
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int sms;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_sms[dev])
      if (cudaError_t e = cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev)) return e;
    bool& done = g_attr[dev][2 * SPLIT + (FMT == W4A16_FP4_MX)];
    if (!done) {
      if (cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<FMT>::kSmem)) return e;
      done = true;
    }
    sms = g_sms[dev];
  }
  Maps maps;
  if (cudaError_t e = encode_map_2d(&maps.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w.codes, a.w.K / 2, (int64_t)a.w.rows * a.w.experts,
                                    a.w.K / 2, 128, p.tn / 2, CU_TENSOR_MAP_SWIZZLE_128B))
    return e;
  if (cudaError_t e = encode_map_2d(&maps.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.xc, a.w.K / 2, a.x_rows, a.w.K / 2, 128, 128,
                                    CU_TENSOR_MAP_SWIZZLE_128B))
    return e;
  if (cudaError_t e = fp4_scale_map(&maps.ws, a.w.scales, (int64_t)p.p.row_tiles * a.w.experts, a.w.K, FMT, 2)) return e;
  if (cudaError_t e = fp4_scale_map(&maps.xs, a.xs, (a.x_rows + 127) / 128, a.w.K, FMT, 1)) return e;
  cudaLaunchConfig_t cfg = {};
  const int split = SPLIT ? p.p.split : 1;
  cfg.gridDim = dim3((unsigned)(2 * split * (SPLIT || units < sms / 2 ? units : sms / 2)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)Geo<FMT>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)(2 * split);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fn, maps, p);
}

}  // namespace

cudaError_t launch_fp4_pair(const Fp4MmArgs& a, int pdl, cudaStream_t s) {
  PairParams p;
  p.p = fp4_params(a, 256);
  p.tn = 256;
  const int x_tiles = a.tiles ? a.max_tiles : p.p.x_tiles;
  const bool mx = a.w.format == W4A16_FP4_MX;
  const int ring = mx ? Geo<W4A16_FP4_MX>::kStages * Geo<W4A16_FP4_MX>::kStage : Geo<W4A16_FP4_NV>::kStages * Geo<W4A16_FP4_NV>::kStage;
  int64_t best = INT64_MAX;
  for (int split = 1; split <= kMaxSplit; split *= 2)
    for (int tn = 256; tn >= 128; tn -= 64) {
      const int64_t tiles = (int64_t)((a.w.rows + tn - 1) / tn) * x_tiles;
      if (split > 1 && (tiles * split > kPairs || p.p.stages < 2 * split || !split_fits(split, tn, ring))) continue;
      const int64_t rounds = (tiles + kPairs - 1) / kPairs;
      const int64_t cost = rounds * ((p.p.stages + split - 1) / split) * (tn + 64) + (split > 1 ? kExchange : 0);
      if (cost < best) best = cost, p.tn = tn, p.p.split = split;
    }
  p.n_tiles = (a.w.rows + p.tn - 1) / p.tn;
  const int cols = a.act == W4A16_FP4_LINEAR ? a.w.rows : a.w.rows / 2;  // of a row of y
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.y);
  p.p.vec = cols % 16 == 0 && at % 32 == 0 ? 32 : cols % 8 == 0 && at % 16 == 0 ? 16 : 0;
  const int64_t units = (int64_t)p.n_tiles * x_tiles;
  if (p.p.split > 1) return mx ? launch_t<W4A16_FP4_MX, true>(a, p, units, pdl, s) : launch_t<W4A16_FP4_NV, true>(a, p, units, pdl, s);
  return mx ? launch_t<W4A16_FP4_MX, false>(a, p, units, pdl, s) : launch_t<W4A16_FP4_NV, false>(a, p, units, pdl, s);
}

}  // namespace w4a16
