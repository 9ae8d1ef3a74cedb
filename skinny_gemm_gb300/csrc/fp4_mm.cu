// fp4_mm.cu -- the product of microscaled 4-bit matrices, y = x W^T, on the
// fifth-generation tensor cores: the codes and scales go from HBM through TMA
// to tcgen05.mma with block scales as they lie, nothing is unpacked.
//
//   y[m][n] = fx[m] fw[n] sum_b sx[m][b] sw[n][b] sum_{k in b} x[m][k] w[n][k]
//
// in fp32, rounded to bf16 once.  128 rows of W are the MMA's M, so a few
// activation rows fill N and not M; NT activation rows are its N.  A stage is
// 256 of K: 16 KB of W codes, NT x 128 B of x codes (both 128-byte swizzled)
// and their scale atoms, four instructions of 64 of K.
//
// CTA: six warps, persistent over tiles (128 W rows x NT activation rows).
//   warp 0      TMA producer
//   warp 1      scales from shared to tensor memory, MMAs, commits
//   warps 2-5   epilogue: accumulator -> registers, factors, activation, bf16
//               stores; two accumulators, so that the next tile's MMAs run
// Two CTAs an SM: what a stage costs beside its bytes is the issue of eight
// copies of scales and four MMAs, and two warps issue side by side.
//
// K split over a cluster.  Where W has few row tiles, `split` CTAs take a
// tile's stages between them; every CTA then sends each other one its columns
// through distributed shared memory, and the sums are added in the order of K.
// The split depends on W's shape alone: up to 64 rows of x a row's result is
// the same, bit for bit, whatever the other rows of the call.
//
// A few activation rows (decode, verify) are quantised in the kernel, by the
// epilogue's warps while W's first stages come: each CTA takes its own part of K
// (and every row's peak, for nv's factor), as fp4.cu would have it, bit for bit.
// That saves the quantiser's launch.  A routed call of a few tokens (IDS) takes them
// all as the activation tile of each expert that was chosen, and stores of its
// columns those that chose it: no places, no launch before.
//
// Scales in tensor memory have a set for each slot of the ring: a stage that
// landed in a slot says that the MMAs which read the slot before are done.
// Every wait is bounded: one that gives up raises W4A16_DEVICE_TIMEOUT, all
// roles leave their loops, outstanding copies and MMAs are waited for (also
// bounded) and the tensor memory is freed before the CTA exits.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "fp4.cuh"
#include "fp4_mm.cuh"
#include "fp4_quant.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace w4a16 {
namespace {

using namespace ptx;

constexpr int kWRows = 128;
constexpr int kWTile = kWRows * 128;  // 16 KB
constexpr int kScaleTile = 2048;      // scale atoms of a stage and 128 rows (mx: half of it)
constexpr int kSetCols = 32;          // 16 columns of W's scales, 16 of x's
constexpr int kThreads = 192;
constexpr int kMaxSplit = 8;
constexpr int kCtaSmem = 113 * 1024;  // of which two fit an SM
// A ring leaves room for a CTA of the next call's quantiser beside two of its own, which else starts only when they are
// gone (5 rows x 10240 x 2560: 6.8 us, with rings of all 113 KB 7.8).
constexpr int kRing = 108 * 1024 + 512;
constexpr int kOwnAtom = 256;  // an atom's first 16 rows (the MMA's others are whatever follows)

template <int NT>
struct Geo {
  static constexpr int kX = NT * 128;
  static constexpr int kXAtom = NT == 16 ? kOwnAtom : kFp4Atom;  // bytes of an atom of x's scales that are fetched
  static constexpr int kStage = kWTile + kScaleTile + kX + 4 * kXAtom;
  static constexpr int kPast = kFp4Atom - kXAtom;  // bytes that the last atom's copy reads past the ring
  static constexpr int kStages = (kRing - kPast) / kStage;
  static constexpr int kAcc = 2;
  static constexpr uint32_t kTmemCols = 256;
  static constexpr int kBars = 2 * kStages + 2 * kAcc + 2;
  static constexpr int kSmem = kStages * kStage + kPast + kBars * 8 + 16;
  static_assert(kSmem <= kCtaSmem && kAcc * NT + kStages * kSetCols <= (int)kTmemCols, "half an SM's shared and tensor memory");
  static_assert(NT * kWRows * 4 <= kStages * kStage, "the partial sums of a split tile, which else take the stages' place");
};

struct Maps {
  CUtensorMap w;  // u8 [experts * N][K / 2], box 128 bytes x 128 rows, 128-byte swizzle
  CUtensorMap x;  // u8 [x rows][K / 2], box 128 bytes x NT rows
  CUtensorMap ws;  // scales, boxes of one row tile
  CUtensorMap xs;
};

// Activation rows that a CTA quantises: codes of its stages as the tiles that TMA would have brought, and their scales.
constexpr int kOwnRows = 16, kOwnStage = kOwnRows * 128, kOwnThreads = 128;
constexpr int kOwnUnits = 512;  // of sixteen values: most of a CTA
constexpr int kOwnIds = 32;     // most choices of a routed call that quantises its tokens: a lane each
// Room of its own for a split tile's partial sums from the other CTAs (16 columns in 2, 4 or 8 parts, all but one): a CTA
// need not wait for the others' MMAs before it sends its own (5 x 2560 x 10240: 5.9 us, else 6.2).
constexpr int kOwnParts = kOwnRows * kWRows * 4 / kMaxSplit * (kMaxSplit - 1);

struct OwnRows {
  uint32_t peak[kOwnRows], finite[kOwnRows];  // largest |x| of a row's part, and of its finite values where that is not
  uint32_t whole[kOwnRows];                   // ... of the row: the largest of the cluster's parts
  float factor[kOwnRows];
};

// A routed call of a few tokens: all of them are the activation tile of every expert that one of them chose, and a choice's
// row is stored from its expert's tile alone.
struct OwnIds {
  int expert[kOwnIds];  // the experts, `count` of them
  int id[kOwnIds];      // of the choices (-1: no expert)
  int count;
};

// All threads; what was chosen, and zeros for the rows of choices that are no expert.
__device__ __forceinline__ void own_ids(const Fp4MmParams& p, OwnIds* s) {
  const int n = p.M * p.top, cols = p.act == W4A16_FP4_LINEAR ? p.N : p.N / 2;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int id = lane < n ? p.ids[lane] : -1;
    const bool bad = id < 0 || id >= p.E;
    if (bad && lane < n && blockIdx.x == 0) atomicOr(p.flags, W4A16_DEVICE_BAD_ID);
    if (bad) id = -1;
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    const bool first = !bad && __ffs(same) - 1 == lane;
    const uint32_t all = __ballot_sync(0xffffffffu, first);
    s->id[lane] = id;
    if (first) s->expert[__popc(all & ((1u << lane) - 1))] = id;
    if (lane == 0) s->count = __popc(all);
  }
  __syncthreads();
  for (int r = blockIdx.x; r < n; r += gridDim.x)
    if (s->id[r] < 0)
      for (int i = threadIdx.x; i < cols; i += kThreads) p.y[(int64_t)r * cols + i] = 0;
}

// nv needs a row's peak before its first code.  Each CTA finds its part's, and sends it to all of the cluster
// (`told`: a barrier of M * split arrivals); a row or so (two units a thread) is read whole instead.  Us so / by the other
// way in every case: 1 x 2560 to 10240 5.9 / 6.7, 5 x 2304 gated to 9216 9.6 / 11.0, 5 x 10240 to 2560 8.9 / 17.
template <int FMT>
__device__ __forceinline__ bool quantise_own(const Fp4MmParams& p, OwnRows* own, uint32_t told, uint32_t codes, uint32_t scales, int t, int k0, int k1,
                                             uint32_t limit) {
  constexpr int kAtoms = FMT == W4A16_FP4_MX ? 2 : 4, kEach = kOwnUnits / kOwnThreads;
  const int units = p.K / 16, lane = t & 31;
  const int per = 16 * (k1 - k0), all = p.M * per;  // units of a row's part, whole stages (what lies past K is zero)
  fp4::Vec16 mine[kEach];
  int row[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int i = t + j * kOwnThreads, m = i / per, c = 16 * k0 + i - m * per;
    row[j] = min(m, p.M - 1);
    mine[j] = i < all && c < units ? fp4::load16(p.x + m * p.x_stride + 16 * c) : fp4::zero16();
  }
  constexpr int kWhole = 2;
  const bool whole = FMT == W4A16_FP4_NV && p.split > 1 && p.M * units <= kWhole * kOwnThreads;
  fp4::Vec16 rows[kWhole];
  int rows_of[kWhole];
  if (whole) {
#pragma unroll
    for (int j = 0; j < kWhole; ++j) {
      const int i = t + j * kOwnThreads, m = i / units;
      rows_of[j] = min(m, p.M - 1);
      rows[j] = m < p.M ? fp4::load16(p.x + m * p.x_stride + 16 * (i - m * units)) : fp4::zero16();
    }
  }
  bool ok = true;
  if (FMT == W4A16_FP4_NV) {
    auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kOwnThreads) : "memory"); };
    auto fold = [&](uint32_t peak, int m, uint32_t* to) {
      const int m0 = __shfl_sync(0xffffffffu, m, 0), m1 = __shfl_sync(0xffffffffu, m, 31);
      if (m1 - m0 <= 1) {  // the warp's units lie in one row or two
        const uint32_t a = __reduce_max_sync(0xffffffffu, m == m0 ? peak : 0u), b = __reduce_max_sync(0xffffffffu, m == m0 ? 0u : peak);
        if (lane == 0) atomicMax(to + m0, a);
        if (lane == 31 && m1 > m0) atomicMax(to + m1, b);
      } else {
        atomicMax(to + m, peak);
      }
    };
    auto peaks = [&](auto&& of, uint32_t* to) {
      if (whole) {
#pragma unroll
        for (int j = 0; j < kWhole; ++j) fold(of(rows[j]), rows_of[j], to);
      } else {
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          if (j * kOwnThreads >= all) break;
          fold(of(mine[j]), row[j], to);
        }
      }
    };
    peaks([](const fp4::Vec16& v) { return fp4::peak16(v); }, own->peak);
    sync();
    const uint32_t odd = __ballot_sync(0xffffffffu, lane < p.M && own->peak[lane & 15] >= 0x7F80u);
    if (odd) {  // rows with a NaN or an infinity
      peaks([](const fp4::Vec16& v) { return fp4::finite_peak16(v); }, own->finite);
      sync();
    }
    auto part = [&](int m) { return odd >> m & 1 ? own->finite[m] : own->peak[m]; };
    if (p.split > 1) cluster_wait();  // (the others are there)
    if (p.split == 1 || whole) {
      if (t < p.M) own->whole[t] = part(t);
    } else {
      if (t < p.M * p.split) {
        const int m = t % p.M, g = t / p.M;
        red_max_cluster(cluster_map(smem_u32(own->whole + m), (uint32_t)g), part(m));
        mbar_arrive_release_cluster(cluster_map(told, (uint32_t)g));
      }
      __syncwarp();
      ok = mbar_wait_acquire_cluster(told, 0, limit);
    }
    if (t < p.M) own->factor[t] = fp4::exp2n(fp4::factor_exp(own->whole[t]));
    sync();
  }
#pragma unroll
  for (int j = 0; j < kEach; ++j) {  // (whole warps)
    if (j * kOwnThreads >= all) break;
    const int i = t + j * kOwnThreads, m = row[j], u = i % per;
    uint32_t peak = fp4::peak16(mine[j]);
    if (FMT == W4A16_FP4_MX) peak = max(peak, __shfl_xor_sync(0xffffffffu, peak, 1));
    const int e = FMT == W4A16_FP4_NV ? (int)(__float_as_uint(own->factor[m]) >> 23) - 127 : 0;
    uint32_t byte;
    const uint2 code = fp4::block16<FMT>(mine[j], peak, e, byte);
    const int stage = u / 16, unit = u % 16, b = FMT == W4A16_FP4_MX ? unit / 2 : unit;
    if (i < all) {
      asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(codes + (uint32_t)(stage * kOwnStage + m * 128 + (((unit >> 1) ^ (m & 7)) << 4) + (unit & 1) * 8)),
                   "r"(code.x), "r"(code.y)
                   : "memory");
      if (FMT == W4A16_FP4_NV || !(unit & 1))
        asm volatile("st.shared.u8 [%0], %1;" ::"r"(scales + (uint32_t)((stage * kAtoms + b / 4) * kOwnAtom + m * 16 + b % 4)), "r"(byte) : "memory");
    }
  }
  fence_proxy_async();
  return ok;
}

// One sum of row `row` of W and place `at` of x, row m of y, whole warps (gate and up rows are neighbours).
__device__ __forceinline__ void store(const Fp4MmParams& p, float v, float fw, const float* xf, int at, int64_t m, int row, bool mine) {
  const float t = xf ? fp4_scaled(v, fw, xf[at]) : v * fw;
  if (p.act == W4A16_FP4_LINEAR) {
    if (mine) p.y[m * p.N + row] = f32_to_bf16_bits(t);
  } else {
    const float up = __shfl_down_sync(0xffffffffu, t, 1);
    if (mine && !(row & 1)) p.y[m * (p.N / 2) + row / 2] = f32_to_bf16_bits(fp4_activate(t, p.act) * up);
  }
}

// Four neighbouring rows of W, `row` a multiple of four, and place `at` of x.
__device__ __forceinline__ void store4(const Fp4MmParams& p, const float (&v)[4], int at, int row) {
  const int64_t m = p.row ? p.row[at] : at;
  if (p.act == W4A16_FP4_LINEAR) {
    uint16_t* y = p.y + m * p.N + row;
    if (p.vec && row + 4 <= p.N) {
      *reinterpret_cast<uint2*>(y) = make_uint2(fp4_bf16x2(v[0], v[1]), fp4_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (row + i < p.N) y[i] = f32_to_bf16_bits(v[i]);
    }
  } else {
    uint16_t* y = p.y + m * (p.N / 2) + row / 2;
    const uint32_t two = fp4_bf16x2(fp4_activate(v[0], p.act) * v[1], fp4_activate(v[2], p.act) * v[3]);
    if (row < p.N) y[0] = (uint16_t)two;
    if (row + 2 < p.N) y[1] = (uint16_t)(two >> 16);
  }
}

// Routed: the expert of activation tile `tile` (-1: there are fewer), from the ids alone, by all threads of the CTA; count:
// shared memory of E ints.  For the first unit's W, which then comes while the quantiser still places the rows.
// Rows (and experts) up to which that pays; us so / without, K = 2048, N = 1536 of 64 experts: 120 rows 15.1 / 15.9, 512 21.1 /
// 21.9, 1024 23.3 / 24.5, 2000 27.9 / 27.3, 2560 34.3 / 32.6 (the quantiser's CTAs take up the SMs longer).
constexpr int kIdsMost = 1024;
__device__ __forceinline__ int expert_of(const Fp4MmParams& p, int tile, int* count) {
  for (int e = threadIdx.x; e < p.E; e += kThreads) count[e] = 0;
  __syncthreads();
  for (int r = threadIdx.x; r < p.M; r += kThreads) {
    const int e = p.ids[r];
    if (e >= 0 && e < p.E) atomicAdd(count + e, 1);
  }
  fence_proxy_async();  // (the stages take the counts' place)
  __syncthreads();
  if (threadIdx.x >= 32) return -1;
  const int lane = threadIdx.x, per = (p.E + 31) / 32, e0 = min(lane * per, p.E), e1 = min(e0 + per, p.E);
  int tiles = 0;
  for (int e = e0; e < e1; ++e) tiles += (count[e] + p.nt - 1) / p.nt;
  int sum = tiles;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int up = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += up;
  }
  int at = sum - tiles, found = -1;
  if (tile >= at && tile < sum)
    for (int e = e0; found < 0; ++e) {
      at += (count[e] + p.nt - 1) / p.nt;
      if (tile < at) found = e;
    }
  return __reduce_max_sync(0xffffffffu, found);
}

template <int NT, int FMT, bool OWN, bool IDS>
__global__ void __launch_bounds__(kThreads, 2) fp4_mm_kernel(const __grid_constant__ Maps maps, Fp4MmParams p) {
  using G = Geo<NT>;
  constexpr int NB = G::kAcc;
  const int S = OWN ? p.slots : G::kStages;
  constexpr int kStage = OWN ? kWTile + kScaleTile : G::kStage;
  constexpr int kAtoms = FMT == W4A16_FP4_MX ? 2 : 4;  // of a stage and 128 rows
  extern __shared__ __align__(1024) uint8_t base[];  // (the tiles' swizzle counts from multiples of 1024)
  const uint32_t sb = smem_u32(base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = p.split, rank = split > 1 ? (int)cluster_rank() : 0;
  // this CTA's stages of a tile
  const int k0 = p.stages * rank / split, k1 = p.stages * (rank + 1) / split;
  const int own_stages = OWN ? (p.stages + split - 1) / split : 0;
  const uint32_t own_codes = sb + (uint32_t)(S * kStage), own_scales = own_codes + (uint32_t)(own_stages * kOwnStage);
  const uint32_t behind = OWN ? own_scales + (uint32_t)(own_stages * kAtoms * kOwnAtom + kOwnAtom) : own_codes;
  constexpr int kParts = OWN ? kOwnParts : 0;
  const uint32_t parts = kParts ? behind : sb, bars = behind + (OWN ? kParts : G::kPast);
  auto W_of = [&](int s) { return sb + (uint32_t)(s * kStage); };
  auto SW_of = [&](int s) { return W_of(s) + kWTile; };
  auto X_of = [&](int s) { return SW_of(s) + kScaleTile; };
  auto SX_of = [&](int s) { return X_of(s) + G::kX; };
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (S + s); };
  auto acc_full = [&](int b) { return bars + 8u * (2 * S + b); };
  auto acc_free = [&](int b) { return bars + 8u * (2 * S + NB + b); };
  const uint32_t own_full = bars + 8u * (2 * S + 2 * NB), told = own_full + 8;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(base + (told + 8 - sb));
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  OwnRows* own = reinterpret_cast<OwnRows*>(s_tmem + 2);
  OwnIds* ids = reinterpret_cast<OwnIds*>(own + 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1 + (p.fault_wait && blockIdx.x == 0 && s == 0));  // (debug: an arrival that never comes)
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < NB; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_free(b), 4);
    }
    mbar_init(own_full, kOwnThreads);
    if (OWN) mbar_init(told, (uint32_t)(p.M * split));
    *s_abort = 0;
    fence_barrier_init();
  }
  if (OWN && threadIdx.x >= 32 && threadIdx.x < 32 + kOwnRows) own->peak[threadIdx.x - 32] = own->finite[threadIdx.x - 32] = own->whole[threadIdx.x - 32] = 0;
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), G::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *s_tmem;
  if (kParts && split > 1) cluster_arrive();  // (this CTA is there to be written to)
  pdl_launch_dependents();
  const int64_t first = blockIdx.x / (unsigned)split, step = gridDim.x / (unsigned)split;
  const uint32_t limit = p.fault_wait ? 4096u : 1u << 18;  // tries of a wait: about a second
  // What comes before the wait for the kernel before: nothing but W (and ids), and that only where they are complete already.
  int early_expert = 0;
  if (!OWN && p.ids) early_expert = expert_of(p, (int)(first / p.row_tiles), reinterpret_cast<int*>(base));
  if (!(p.early && warp == 0)) pdl_wait();
  if (IDS) own_ids(p, ids);
  auto units_now = [&]() { return (int64_t)(IDS ? ids->count : p.tiles ? *p.tile_count : p.x_tiles) * p.row_tiles; };
  int64_t units = p.early && warp == 0 && p.tiles ? 0 : units_now();  // (the early producer: when it has waited)
  auto timeout = [&]() {
    atomicOr(p.flags, W4A16_DEVICE_TIMEOUT);
    *s_abort = 1;
  };
  uint32_t it = 0;  // stages of this CTA so far: the producer's, and the MMA warp's

  if (warp == 0) {
    // ---- TMA producer ----
    if (lane == 0) {
      const uint64_t keep = policy_evict_last(), stream = policy_evict_first();
      auto load_w = [&](int s, int k, int wrow, int ws) {
        mbar_expect_tx(full(s), kWTile + kAtoms * kFp4Atom + (OWN ? 0 : G::kX + kAtoms * G::kXAtom));
        tma_load_2d(W_of(s), &maps.w, k * 128, wrow, full(s), stream);
        tma_load_3d(SW_of(s), &maps.ws, 0, k * kAtoms, ws, full(s), stream);
      };
      int ahead = 0;  // stages whose W is requested already
      if (p.early) {
        if (p.tiles ? early_expert >= 0 : first < units) {
          const int wt = (int)(first % p.row_tiles);
          for (; ahead < S && k0 + ahead < k1; ++ahead)
            load_w(ahead, k0 + ahead, early_expert * p.N + wt * kWRows, early_expert * p.row_tiles + wt);
        }
        pdl_wait();
        units = units_now();
      }
      int s = 0;
      uint32_t parity = 1;
      for (int64_t u = first; u < units && !*s_abort; u += step) {
        const int xt = (int)(u / p.row_tiles), wt = (int)(u % p.row_tiles);
        int64_t expert = 0;
        int place = xt * NT;
        if (IDS) {
          expert = ids->expert[xt];
        } else if (p.tiles) {
          expert = p.tiles[xt].expert;
          place = p.tiles[xt].place;
        }
        const int wrow = (int)(expert * p.N + (int64_t)wt * kWRows);
        const int ws = (int)(expert * p.row_tiles) + wt, xs = place / kFp4Rows;
        for (int k = k0; k < k1; ++k, ++it) {
          if (it >= (uint32_t)S && !mbar_wait_parked(empty(s), parity, 1000, limit)) {
            timeout();
            break;
          }
          if (it >= (uint32_t)ahead) load_w(s, k, wrow, ws);
          if (!OWN) {
            tma_load_2d(X_of(s), &maps.x, k * 128, place, full(s), keep);
            tma_load_3d(SX_of(s), &maps.xs, 0, k * kAtoms, xs, full(s), keep);
          }
          if (++s == S) s = 0, parity ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    // ---- scales and MMAs ----
    const uint32_t go = elect_one();
    constexpr uint32_t kIdesc = umma_idesc_e2m1(kWRows, NT, FMT == W4A16_FP4_MX);
    const uint64_t wd0 = umma_desc_sw128(W_of(0)), xd0 = umma_desc_sw128(OWN ? own_codes : X_of(0));
    const uint64_t sw0 = umma_desc(SW_of(0), 128, 128, 0), sx0 = umma_desc(OWN ? own_scales : SX_of(0), 128, 128, 0);
    if (OWN && !mbar_wait_warp(own_full, 0, limit) && lane == 0) timeout();
    uint32_t n = 0;  // tiles
    int s = 0;
    uint32_t parity = 0;
    for (int64_t u = first; u < units && !*s_abort; u += step, ++n) {
      const int b = (int)(n % NB);
      if (n >= (uint32_t)NB && !mbar_wait_warp(acc_free(b), ((n / NB) - 1) & 1, limit)) {
        if (lane == 0) timeout();
        break;
      }
      tc_fence_after_sync();
      const uint32_t acc = tmem + (uint32_t)(b * NT);
      bool ok = true;
      for (int k = k0; k < k1; ++k, ++it) {
        if (!(ok = mbar_wait_warp(full(s), parity, limit))) {
          if (lane == 0) timeout();
          break;
        }
        tc_fence_after_sync();
        const uint64_t at = (uint64_t)(uint32_t)(s * (kStage >> 4));
        const uint64_t wd = wd0 + at, sw = sw0 + at;
        const uint64_t xd = xd0 + (OWN ? (uint64_t)(uint32_t)((k - k0) * (kOwnStage >> 4)) : at);
        const uint64_t sx = sx0 + (OWN ? (uint64_t)(uint32_t)((k - k0) * (kAtoms * kOwnAtom >> 4)) : at);
        const uint32_t cw = tmem + (uint32_t)(NB * NT + s * kSetCols), cx = cw + 16;
        const int atoms = p.atoms - k * kAtoms, steps = (p.K - k * kFp4StageK + 63) / 64;
        auto copy = [&](int a) {
          tmem_copy_scales(cw + 4 * a, sw + (uint64_t)(a * (kFp4Atom >> 4)));
          tmem_copy_scales(cx + 4 * a, sx + (uint64_t)(a * (G::kXAtom >> 4)));
        };
        auto mma = [&](int j) {
          const bool add = k > k0 || j > 0;
          if (FMT == W4A16_FP4_MX)
            umma_mxf4(acc, wd + 2 * j, xd + 2 * j, kIdesc | umma_idesc_scale_byte(2 * (j & 1)), cw + 4 * (j / 2), cx + 4 * (j / 2), add);
          else
            umma_nvf4(acc, wd + 2 * j, xd + 2 * j, kIdesc, cw + 4 * j, cx + 4 * j, add);
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
        umma_commit_if(go, empty(s));
        if (++s == S) s = 0, parity ^= 1;
      }
      if (!ok) break;
      umma_commit_if(go, acc_full(b));
    }
  } else {
    // ---- epilogue ----
    const int q = warp & 3, r = 32 * q + lane;
    if (OWN) {
      if (!quantise_own<FMT>(p, own, told, own_codes, own_scales, threadIdx.x - 64, k0, k1, limit) && lane == 0) timeout();
      mbar_arrive(own_full);
    }
    const float* xf = OWN ? (FMT == W4A16_FP4_NV ? own->factor : nullptr) : p.xf;
    uint32_t n = 0;
    for (int64_t u = first; u < units && !*s_abort; u += step, ++n) {
      const int b = (int)(n % NB);
      const int xt = (int)(u / p.row_tiles), wt = (int)(u % p.row_tiles);
      int64_t expert = 0;
      int place = xt * NT, count = min(NT, p.M - place);
      if (IDS) {
        expert = ids->expert[xt];
        place = 0;
        count = p.M;
      } else if (p.tiles) {
        expert = p.tiles[xt].expert;
        place = p.tiles[xt].place;
        count = p.tiles[xt].count;
      }
      const int row = wt * kWRows + r;
      const bool mine = row < p.N;
      const float fw = p.wf && mine ? p.wf[expert * p.N + row] : 1.0f;
      if (!mbar_wait_warp(acc_full(b), (n / NB) & 1, limit + (uint32_t)p.stages)) {  // (a tile of a long K: a try is longer than a stage)
        if (lane == 0) timeout();
        break;
      }
      if (split > 1) break;  // (one tile a cluster: the rest below)
      tc_fence_after_sync();
      const uint32_t acc = tmem + (uint32_t)(b * NT) + ((uint32_t)(32 * q) << 16);
#pragma unroll 1
      for (int c = 0; c < NT; c += 16) {
        if (c >= count) break;
        __syncwarp();  // (rows that are not stored are back)
        float v[16];
        tmem_ld16(acc + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (c + i >= count) break;
          const int at = place + c + i;
          if (IDS) {
            for (int m = at * p.top; m < (at + 1) * p.top; ++m)
              if (ids->id[m] == expert) store(p, v[i], fw, xf, at, m, row, mine);
          } else {
            store(p, v[i], fw, xf, at, p.row ? p.row[at] : at, row, mine);
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_free(b));
    }
  }

  __syncthreads();
  if (split > 1) {
    // ---- a split tile: partial sums to the CTAs that add them up ----
    // Rank g adds the columns [g per, (g + 1) per).  Where the sums take the stages' place, no MMA of the cluster may
    // read those any more; a CTA that gave up takes part in the barriers all the same.
    const int q = warp & 3, xt = (int)(first / p.row_tiles), wt = (int)(first % p.row_tiles);
    const bool live = first < units && !*s_abort;
    const int count = min(NT, p.M - xt * NT), per = (count + split - 1) / split;
    if (!kParts) cluster_arrive();
    if (!(OWN && FMT == W4A16_FP4_NV && warp >= 2)) cluster_wait();  // (those have waited)
    if (live && warp >= 2) {
      tc_fence_after_sync();
      const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16);
      int g = 0, col = 0;  // column c is the col-th of rank g's
      // a part's place at its rank; this CTA's own part lies in its stages, which are its own again
      auto part_of = [&](int to) { return to == rank || !kParts ? sb + (uint32_t)(rank * per * kWRows * 4) : parts + (uint32_t)((rank - (rank > to)) * per * kWRows * 4); };
#pragma unroll 1
      for (int c = 0; c < count; c += 16) {
        float v[16];
        tmem_ld16(acc + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (c + i >= count) break;
          st_cluster_f32(cluster_map(part_of(g) + (uint32_t)((col * kWRows + 32 * q + lane) * 4), (uint32_t)g), v[i]);
          if (++col == per) col = 0, ++g;
        }
      }
    }
    cluster_arrive();
    cluster_wait();
    if (live) {  // a warp a column, a lane four rows (and column lane's factor: there are at most half of 64)
      const int row = wt * kWRows + 4 * lane, place = xt * NT + rank * per, cols = min(per, count - rank * per);
      float fw[4], xf = 1.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) fw[i] = p.wf && row + i < p.N ? p.wf[row + i] : 1.0f;
      if (lane < cols) xf = OWN ? (FMT == W4A16_FP4_NV ? own->factor[rank * per + lane] : 1.0f) : p.xf ? p.xf[place + lane] : 1.0f;
#pragma unroll 2
      for (int c = warp; c < cols; c += kThreads / 32) {
        const float fx = __shfl_sync(0xffffffffu, xf, c);
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        for (int g = 0; g < split; ++g) {
          const uint32_t from = g == rank || !kParts ? sb + (uint32_t)(g * per * kWRows * 4) : parts + (uint32_t)((g - (g > rank)) * per * kWRows * 4);
          const float4 f = lds128f(from + (uint32_t)((c * kWRows + 4 * lane) * 4));
          v[0] += f.x;
          v[1] += f.y;
          v[2] += f.z;
          v[3] += f.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fp4_scaled(v[i], fw[i], fx);
        store4(p, v, place + c, row);
      }
    }
  }

  // ---- teardown: everything in flight lands before the memories are released ----
  if (*s_abort) {
    if (warp == 0 && lane == 0)
      for (uint32_t i = it > (uint32_t)S ? it - S : 0; i < it; ++i) mbar_wait_parked(full((int)(i % S)), (i / S) & 1, 1000, limit);
    if (warp == 1 && it > 0) mbar_wait_warp(empty((int)((it - 1) % S)), ((it - 1) / S) & 1, limit);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, G::kTmemCols);
  }
}

// ---- host side ------------------------------------------------------------------------

std::mutex g_mu;
// K is split where that leaves no CTA without a place (two an SM of 152) or a stage.  By W's shape alone.
int split_of(int row_tiles, int stages) {
  int split = 1;
  while (split < kMaxSplit && 2 * split * row_tiles <= 304 && 2 * split <= stages) split *= 2;
  return split;
}

// Where the kernel quantises: shared memory of a ring of `slots` beside a CTA's `stages` of x, and how many slots fit.
constexpr int own_smem(int slots, int stages, bool ids) {
  return slots * (kWTile + kScaleTile) + stages * (kOwnStage + 4 * kOwnAtom) + kOwnAtom + kOwnParts + (2 * slots + 6) * 8 + 8 + (int)sizeof(OwnRows) + (ids ? (int)sizeof(OwnIds) : 0);
}
int own_slots(int stages, bool ids) {
  int slots = 5;
  while (slots > 0 && own_smem(slots, stages, ids) > kCtaSmem) --slots;
  return slots;
}

struct Device {
  int sms = 0;
  bool attr[10] = {};
};
Device g_dev[64];

template <int NT, int FMT, bool OWN = false, bool IDS = false>
cudaError_t launch_t(const Fp4MmArgs& a, const Fp4MmParams& p, int pdl, cudaStream_t s) {
  using G = Geo<NT>;
  auto* fn = fp4_mm_kernel<NT, FMT, OWN, IDS>;
  constexpr int kIndex = (IDS ? 4 : OWN ? 3 : NT == 16 ? 0 : NT == 32 ? 1 : 2) * 2 + (FMT == W4A16_FP4_MX);
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int sms;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    Device& d = g_dev[dev];
    if (!d.sms)
      if (cudaError_t e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev)) return e;
    if (!d.attr[kIndex]) {
      if (cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, OWN ? kCtaSmem : G::kSmem)) return e;
      d.attr[kIndex] = true;
    }
    sms = d.sms;
  }
  Maps maps;
  if (cudaError_t e = encode_map_2d(&maps.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w.codes, a.w.K / 2, (int64_t)a.w.rows * a.w.experts,
                                    a.w.K / 2, 128, kWRows, CU_TENSOR_MAP_SWIZZLE_128B))
    return e;
  if (!OWN)
    if (cudaError_t e = encode_map_2d(&maps.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.xc, a.w.K / 2, a.x_rows, a.w.K / 2, 128, NT,
                                    CU_TENSOR_MAP_SWIZZLE_128B))
    return e;
  if (cudaError_t e = fp4_scale_map(&maps.ws, a.w.scales, (int64_t)p.row_tiles * a.w.experts, a.w.K, FMT, 1)) return e;
  if (!OWN)
    if (cudaError_t e = fp4_scale_map(&maps.xs, a.xs, (a.x_rows + 127) / 128, a.w.K, FMT, 1, G::kXAtom / 4)) return e;
  const int64_t units = (int64_t)p.row_tiles * (a.tiles ? a.max_tiles : p.x_tiles);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.split > 1 ? units * p.split : units < 2 * sms ? units : 2 * sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)(OWN ? own_smem(p.slots, (p.stages + p.split - 1) / p.split, IDS) : G::kSmem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = 0;
  if (p.split > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = (unsigned)p.split;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (pdl > 0) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, fn, maps, p);
}

}  // namespace

// The GPU's us so / with the quantiser's launch before it: nv 1 row x 2560 to 10240 5.8 / 7.1, 5 rows 7.6 to 8.5 / 7.6 to 7.9, 1 x 2560 to
// 262144 56.8 / 59.0, 5 x 2304 gated to 9216 9.6 / 9.2, 5 x 10240 to 2560 8.9 / 8.3; mx 6.0 / 7.3.  A call from the host takes
// 10.4 to 12 / 13 to 14 in all of these: five nv rows give up to 7% of the GPU's time in a captured step for that.  Past
// kOwnUnits the CTAs' part grows: 16 x 2560 (mx) 9.4 / 7.7.
bool fp4_mm_fuses(const w4a16_fp4& w, int M) {
  const int stages = (w.K + kFp4StageK - 1) / kFp4StageK, split = split_of((int)fp4_row_tiles(w.rows), stages);
  const int part = (stages + split - 1) / split;
  return M <= kOwnRows && M * 16 * part <= kOwnUnits && own_slots(part, false) >= 3;
}

// The same for routed calls; us so / with the quantiser's launch, K = 2048: 1 token x 4 of 64 experts, N = 1536
// 5.8 / 8.9, 4 x 8 10.6 / 11.5, 1 x 2 of 8 (K = 4096, N = 14336) 13.2 / 15.6, 4 x 1 of 8 (N = 6144) 7.7 / 8.4, 8 x 2 of 16
// (K = 1024, N = 2048) 7.6 / 7.1; with twice the units 8 x 1 of 8 (N = 6144) 11.2 / 9.5.  A call from the host takes 11.5 to 14 /
// 14.5 to 18.
bool fp4_mm_id_fuses(const w4a16_fp4& w, int T, int top) {
  const int64_t stages = (w.K + kFp4StageK - 1) / kFp4StageK;
  return T <= kOwnRows && (int64_t)T * top <= kOwnIds && T * 16 * stages <= kOwnUnits && own_slots((int)stages, true) >= 3;
}

// The smallest tile that takes all rows, and from 65 rows on the pair kernel's.  Us with a tile of 64 or 128 here / there:
// 64 rows to 10240 x 2560 10.2 / 9.4, to 2560 x 10240 10.5 / 15.8; 128 rows 13.2 / 9.6 and 14.7 / 16.6; 100 rows to 262144 x
// 2560 100 / 82.
int fp4_mm_tile(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 256; }

cudaError_t launch_fp4_mm(const Fp4MmArgs& a, int pdl, cudaStream_t s) {
  const int nt = a.tiles ? a.nt : fp4_mm_tile(a.M);
  if (nt == 256) return launch_fp4_pair(a, pdl, s);
  Fp4MmParams p = fp4_params(a, nt);
  p.early = a.early && pdl > 1 && (!a.tiles || (a.M <= kIdsMost && a.w.experts <= kIdsMost));
  if (a.tiles && p.early) p.ids = a.ids;
  p.vec = a.w.rows % 4 == 0 && reinterpret_cast<uintptr_t>(a.y) % 8 == 0;
  if (!a.tiles) p.split = split_of(p.row_tiles, p.stages);
  const bool mx = a.w.format == W4A16_FP4_MX;
  if (a.x) {
    p.early = 0;
    if (a.ids) {
      p.ids = a.ids;
      p.split = 1;
      p.x_tiles = (int64_t)a.M * a.top < a.w.experts ? a.M * a.top : a.w.experts;  // most
      p.slots = own_slots(p.stages, true);
      return mx ? launch_t<16, W4A16_FP4_MX, true, true>(a, p, pdl, s) : launch_t<16, W4A16_FP4_NV, true, true>(a, p, pdl, s);
    }
    p.slots = own_slots((p.stages + p.split - 1) / p.split, false);
    return mx ? launch_t<16, W4A16_FP4_MX, true>(a, p, pdl, s) : launch_t<16, W4A16_FP4_NV, true>(a, p, pdl, s);
  }
  switch (nt) {
    case 16: return mx ? launch_t<16, W4A16_FP4_MX>(a, p, pdl, s) : launch_t<16, W4A16_FP4_NV>(a, p, pdl, s);
    case 32: return mx ? launch_t<32, W4A16_FP4_MX>(a, p, pdl, s) : launch_t<32, W4A16_FP4_NV>(a, p, pdl, s);
    default: return mx ? launch_t<64, W4A16_FP4_MX>(a, p, pdl, s) : launch_t<64, W4A16_FP4_NV>(a, p, pdl, s);
  }
}

}  // namespace w4a16
