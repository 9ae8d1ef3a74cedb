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
// Scales in tensor memory have four sets: a set is written again when the MMAs
// of the stage that used it have completed.
// Every wait is bounded: one that gives up raises W4A16_DEVICE_TIMEOUT, all
// roles leave their loops, outstanding copies and MMAs are waited for (also
// bounded) and the tensor memory is freed before the CTA exits.
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

constexpr int kWRows = 128;
constexpr int kWTile = kWRows * 128;          // 16 KB
constexpr int kScaleTile = 2048;              // scale atoms of a stage and 128 rows (mx: half of it)
constexpr int kSets = 4;                      // scale sets in tensor memory
constexpr int kThreads = 192;

template <int NT>
struct Geo {
  static constexpr int kX = NT * 128;
  static constexpr int kStage = kWTile + kX + 2 * kScaleTile;
  static constexpr int kStages = (225 * 1024) / kStage > 10 ? 10 : (225 * 1024) / kStage;
  static constexpr int kAcc = 2;
  static constexpr int kSetCols = 32;  // 16 columns of W's scales, 16 of x's
  static constexpr int kCols = kAcc * NT + kSets * kSetCols;
  static constexpr uint32_t kTmemCols = kCols <= 256 ? 256 : 512;
  static constexpr int kBars = 2 * kStages + 2 * kAcc;
  static constexpr int kSmem = kStages * kStage + kBars * 8 + 16 + 1024;
  static_assert(kSmem <= 227 * 1024 && kCols <= 512, "a CTA's shared memory and the SM's tensor memory");
};

struct Maps {
  CUtensorMap w;  // u8 [experts * N][K / 2], box 128 bytes x 128 rows, 128-byte swizzle
  CUtensorMap x;  // u8 [x rows][K / 2], box 128 bytes x NT rows
};

template <int NT, int FMT>
__global__ void __launch_bounds__(kThreads, 1) fp4_mm_kernel(const __grid_constant__ Maps maps, Fp4MmParams p) {
  using G = Geo<NT>;
  constexpr int S = G::kStages, NB = G::kAcc;
  constexpr int kAtoms = FMT == W4A16_FP4_MX ? 2 : 4;  // of a stage and 128 rows
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = sb + S * G::kStage;
  auto W_of = [&](int s) { return sb + (uint32_t)(s * G::kStage); };
  auto X_of = [&](int s) { return W_of(s) + kWTile; };
  auto SW_of = [&](int s) { return X_of(s) + G::kX; };
  auto SX_of = [&](int s) { return SW_of(s) + kScaleTile; };
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (S + s); };
  auto acc_full = [&](int b) { return bars + 8u * (2 * S + b); };
  auto acc_free = [&](int b) { return bars + 8u * (2 * S + NB + b); };
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(base + (bars - sb) + 8 * G::kBars);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1 + (p.fault_wait && blockIdx.x == 0 && s == 0));  // (debug: an arrival that never comes)
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < NB; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_free(b), 4);
    }
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), G::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *s_tmem;
  pdl_launch_dependents();
  pdl_wait();
  const int x_tiles = p.tiles ? *p.tile_count : p.x_tiles;
  const int64_t units = (int64_t)x_tiles * p.row_tiles;
  const int ns = p.stages;
  const uint32_t limit = p.fault_wait ? 4096u : 1u << 18;  // tries of a wait: about a second
  auto timeout = [&]() {
    atomicOr(p.flags, W4A16_DEVICE_TIMEOUT);
    *s_abort = 1;
  };
  uint32_t it = 0;  // stages of this CTA so far: the producer's, and the MMA warp's

  if (warp == 0) {
    // ---- TMA producer ----
    if (lane == 0) {
      const uint64_t keep = policy_evict_last(), stream = policy_evict_first();
      for (int64_t u = blockIdx.x; u < units && !*s_abort; u += gridDim.x) {
        const int xt = (int)(u / p.row_tiles), wt = (int)(u % p.row_tiles);
        int64_t expert = 0;
        int place = xt * NT;
        if (p.tiles) {
          expert = p.tiles[xt].expert;
          place = p.tiles[xt].place;
        }
        const int wrow = (int)(expert * p.N + (int64_t)wt * kWRows);
        const uint8_t* ws = p.ws + (expert * p.row_tiles + wt) * p.atoms * kFp4Atom;
        const uint8_t* xs = p.xs + (int64_t)(place / kFp4Rows) * p.atoms * kFp4Atom;
        for (int k = 0; k < ns; ++k, ++it) {
          const int s = (int)(it % S);
          if (it >= (uint32_t)S && !mbar_wait_parked(empty(s), ((it / S) - 1) & 1, 1000, limit)) {
            timeout();
            break;
          }
          const uint32_t scale_bytes = (uint32_t)(min(kAtoms, p.atoms - k * kAtoms) * kFp4Atom);
          mbar_expect_tx(full(s), kWTile + G::kX + 2 * scale_bytes);
          tma_load_2d(W_of(s), &maps.w, k * 128, wrow, full(s), stream);
          bulk_load(SW_of(s), ws + k * kAtoms * kFp4Atom, scale_bytes, full(s), stream);
          tma_load_2d(X_of(s), &maps.x, k * 128, place, full(s), keep);
          bulk_load(SX_of(s), xs + k * kAtoms * kFp4Atom, scale_bytes, full(s), keep);
        }
      }
    }
  } else if (warp == 1) {
    // ---- scales and MMAs ----
    const uint32_t go = elect_one();
    constexpr uint32_t kIdesc = umma_idesc_e2m1(kWRows, NT, FMT == W4A16_FP4_MX);
    uint32_t n = 0;  // tiles
    for (int64_t u = blockIdx.x; u < units && !*s_abort; u += gridDim.x, ++n) {
      const int b = (int)(n % NB);
      if (n >= (uint32_t)NB && !mbar_wait_warp(acc_free(b), ((n / NB) - 1) & 1, limit)) {
        if (lane == 0) timeout();
        break;
      }
      tc_fence_after_sync();
      const uint32_t acc = tmem + (uint32_t)(b * NT);
      bool ok = true;
      for (int k = 0; k < ns; ++k, ++it) {
        const int s = (int)(it % S);
        const uint32_t set = tmem + (uint32_t)(NB * NT + (int)(it % kSets) * G::kSetCols);
        // the set's last MMAs: those of the stage kSets before
        const uint32_t before = it - kSets;
        ok = mbar_wait_warp(full(s), (it / S) & 1, limit) &&
             (it < (uint32_t)kSets || mbar_wait_warp(empty((int)(before % S)), (before / S) & 1, limit));
        if (!ok) {
          if (lane == 0) timeout();
          break;
        }
        tc_fence_after_sync();
        const uint64_t sw = umma_desc(SW_of(s), 128, 128, 0), sx = umma_desc(SX_of(s), 128, 128, 0);
        const uint64_t wd = umma_desc_sw128(W_of(s)), xd = umma_desc_sw128(X_of(s));
        const int atoms = min(kAtoms, p.atoms - k * kAtoms);
        const int steps = min(4, (p.K - k * kFp4StageK + 63) / 64);
#pragma unroll
        for (int a = 0; a < kAtoms; ++a)
          if (a < atoms) {
            tmem_copy_scales(go, set + 4 * a, sw + (uint64_t)(a * (kFp4Atom >> 4)));
            tmem_copy_scales(go, set + 16 + 4 * a, sx + (uint64_t)(a * (kFp4Atom >> 4)));
          }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < steps) {
            if (FMT == W4A16_FP4_MX)
              umma_mxf4(go, acc, wd + 2 * j, xd + 2 * j, kIdesc | umma_idesc_scale_byte(2 * (j & 1)), set + 4 * (j / 2),
                        set + 16 + 4 * (j / 2), k > 0 || j > 0);
            else
              umma_nvf4(go, acc, wd + 2 * j, xd + 2 * j, kIdesc, set + 4 * j, set + 16 + 4 * j, k > 0 || j > 0);
          }
        umma_commit_if(go, empty(s));
      }
      if (!ok) break;
      umma_commit_if(go, acc_full(b));
    }
  } else {
    // ---- epilogue ----
    const int q = warp & 3, r = 32 * q + lane;
    uint32_t n = 0;
    for (int64_t u = blockIdx.x; u < units && !*s_abort; u += gridDim.x, ++n) {
      const int b = (int)(n % NB);
      const int xt = (int)(u / p.row_tiles), wt = (int)(u % p.row_tiles);
      int64_t expert = 0;
      int place = xt * NT, count = min(NT, p.M - place);
      if (p.tiles) {
        expert = p.tiles[xt].expert;
        place = p.tiles[xt].place;
        count = p.tiles[xt].count;
      }
      const int row = wt * kWRows + r;
      const bool mine = row < p.N;
      const float fw = p.wf && mine ? p.wf[expert * p.N + row] : 1.0f;
      if (!mbar_wait_warp(acc_full(b), (n / NB) & 1, limit)) {
        if (lane == 0) timeout();
        break;
      }
      tc_fence_after_sync();
      const uint32_t acc = tmem + (uint32_t)(b * NT) + ((uint32_t)(32 * q) << 16);
#pragma unroll 1
      for (int c = 0; c < NT; c += 16) {
        if (c >= count) break;
        float v[16];
        tmem_ld16(acc + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (c + i >= count) break;
          const int at = place + c + i;
          const int64_t m = p.row ? p.row[at] : at;
          float t = v[i] * fw;
          if (p.xf) t *= p.xf[at];
          if (p.act == W4A16_FP4_LINEAR) {
            if (mine) p.y[m * p.N + row] = f32_to_bf16_bits(t);
          } else {
            const float up = __shfl_down_sync(0xffffffffu, t, 1);
            if (mine && !(row & 1)) p.y[m * (p.N / 2) + row / 2] = f32_to_bf16_bits(fp4_activate(t, p.act) * up);
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_free(b));
    }
  }

  // ---- teardown: everything in flight lands before the memories are released ----
  __syncthreads();
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
struct Device {
  int sms = 0;
  bool attr[8] = {};
};
Device g_dev[64];

template <int NT, int FMT>
cudaError_t launch_t(const Fp4MmArgs& a, const Fp4MmParams& p, int pdl, cudaStream_t s) {
  using G = Geo<NT>;
  auto* fn = fp4_mm_kernel<NT, FMT>;
  constexpr int kIndex = (NT == 16 ? 0 : NT == 32 ? 1 : NT == 64 ? 2 : 3) * 2 + (FMT == W4A16_FP4_MX);
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
      if (cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem)) return e;
      d.attr[kIndex] = true;
    }
    sms = d.sms;
  }
  Maps maps;
  if (cudaError_t e = encode_map_2d(&maps.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w.codes, a.w.K / 2, (int64_t)a.w.rows * a.w.experts,
                                    a.w.K / 2, 128, kWRows, CU_TENSOR_MAP_SWIZZLE_128B))
    return e;
  if (cudaError_t e = encode_map_2d(&maps.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.xc, a.w.K / 2, a.x_rows, a.w.K / 2, 128, NT,
                                    CU_TENSOR_MAP_SWIZZLE_128B))
    return e;
  const int64_t units = (int64_t)p.row_tiles * (a.tiles ? a.max_tiles : p.x_tiles);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units < sms ? units : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)G::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fn, maps, p);
}

}  // namespace

int fp4_mm_tile(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256; }

cudaError_t launch_fp4_mm(const Fp4MmArgs& a, int pdl, cudaStream_t s) {
  const int nt = a.tiles ? a.nt : fp4_mm_tile(a.M);
  if (nt == 256) return launch_fp4_pair(a, pdl, s);
  const Fp4MmParams p = fp4_params(a, nt);
  const bool mx = a.w.format == W4A16_FP4_MX;
  switch (nt) {
    case 16: return mx ? launch_t<16, W4A16_FP4_MX>(a, p, pdl, s) : launch_t<16, W4A16_FP4_NV>(a, p, pdl, s);
    case 32: return mx ? launch_t<32, W4A16_FP4_MX>(a, p, pdl, s) : launch_t<32, W4A16_FP4_NV>(a, p, pdl, s);
    case 64: return mx ? launch_t<64, W4A16_FP4_MX>(a, p, pdl, s) : launch_t<64, W4A16_FP4_NV>(a, p, pdl, s);
    default: return mx ? launch_t<128, W4A16_FP4_MX>(a, p, pdl, s) : launch_t<128, W4A16_FP4_NV>(a, p, pdl, s);
  }
}

}  // namespace w4a16
