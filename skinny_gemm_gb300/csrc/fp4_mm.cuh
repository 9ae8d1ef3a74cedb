// fp4_mm.cuh -- what the two product kernels of microscaled 4-bit matrices
// (fp4_mm.cu, fp4_pair.cu) share.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp4.cuh"
#include "launch.h"

namespace w4a16 {

constexpr int kFp4StageK = 256;  // codes of K per stage: 128 bytes a row

struct Fp4MmParams {
  const uint16_t* x;  // bf16 rows that the kernel quantises itself, or nullptr
  int64_t x_stride;
  const float* wf;  // row factors of W and of x (nullptr: 1)
  const float* xf;
  uint16_t* y;
  const Fp4Tile* tiles;  // routed, or nullptr
  const int32_t* tile_count;
  const int32_t* row;
  const int32_t* ids;  // routed, to find the first unit's expert before the tiles are there (fp4_mm.cu), or nullptr
  int* flags;
  int N, K, M, act;
  int row_tiles, x_tiles;  // 128-row tiles of an expert's W; activation tiles (not routed)
  int atoms, stages;       // scale atoms along K; stages along K
  int vec;                 // y's rows take 8-byte stores (fp4_pair.cu: of how many bytes, 32, 16 or 0)
  int split, early;        // CTAs that share a tile's K; W may be fetched before the wait for the kernel before
  int E, nt;               // ids: experts, rows of a tile
  int top;                 // choices of a token, where the kernel quantises these
  int slots;               // of the ring, where the kernel quantises
  int fault_wait;
};

// Both activations are g / (1 + exp(-t)): t = g, and for the tanh form of gelu, as (1 + tanh u) / 2 = 1 / (1 + exp(-2u)),
// t = 2 sqrt(2 / pi) (g + 0.044715 g^3).  As g 2^-24 / (2^-24 + 2^(-t log2(e) - 24)): without the 2^-24 the divisor overflows
// where act(g) is still a normal number, some 2^-120; with it, where it is below 2^-142.  The hardware's 2^x (2 ulp) and
// reciprocal (1 ulp), 2^-20 for the rounding of 2^x's argument and |t| 2^-23 for t's: the output keeps 2^-8.  (Gated mx 1500 x
// 2560: 34.6 us; as the formula stands, with CUDA's division, 35.7; below zero as g exp(t) / (1 + exp(t)), 37.3.)
__device__ __forceinline__ float fp4_activate(float g, int act) {
  const float t = act == W4A16_FP4_SILU ? g : 1.5957691216057308f * __fmaf_rn(0.044715f * g * g, g, g);
  constexpr float kDown = 1.0f / (1 << 24);
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmaf_rn(t, -1.4426950408889634f, -24.0f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(kDown + e));
  return g * (r * kDown);
}

// v times the row factors of W and x, each anywhere in fp32's range.  Where their product is a normal number, as for one
// above 1 and one below, it comes first.  Else both are above 1 or both below, and v is multiplied by one after the other: what
// is in between lies between v and the result.  (Either order alone gives 0 or infinity for some results that are neither.)
__device__ __forceinline__ bool fp4_normal(float f) { return ((__float_as_uint(f) + 0x00800000u) & 0x7FFFFFFFu) >= 0x01000000u; }
__device__ __forceinline__ float fp4_scaled(float v, float fw, float fx) {
  const float f = fw * fx;
  return fp4_normal(f) ? v * f : v * fw * fx;
}

__device__ __forceinline__ uint32_t fp4_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

inline Fp4MmParams fp4_params(const Fp4MmArgs& a, int x_tile) {
  Fp4MmParams p;
  p.x = a.x;
  p.x_stride = a.x_stride;
  p.wf = a.w.row_scale;
  p.xf = a.xf;
  p.y = a.y;
  p.tiles = a.tiles;
  p.tile_count = a.tile_count;
  p.row = a.row;
  p.ids = nullptr;
  p.flags = a.flags;
  p.N = a.w.rows;
  p.K = a.w.K;
  p.M = a.M;
  p.act = a.act;
  p.row_tiles = (int)fp4_row_tiles(a.w.rows);
  p.x_tiles = a.tiles ? 0 : (a.M + x_tile - 1) / x_tile;
  p.atoms = fp4_atoms(a.w.K, a.w.format);
  p.stages = (a.w.K + kFp4StageK - 1) / kFp4StageK;
  p.vec = 0;
  p.split = 1;
  p.early = 0;
  p.E = a.w.experts;
  p.nt = x_tile;
  p.top = a.top;
  p.slots = 0;
  p.fault_wait = a.fault_wait;
  return p;
}

// The scales' map: [row tiles][atoms along K][128 words], boxes of `tiles` x a stage's atoms (what lies past the end
// is read as zeros).  Tiled copies: as untiled ones of 2 KB, three a stage, they took 330 cycles of the copy engine.
// words: of an atom's 128, 64 for its first 16 rows.
inline cudaError_t fp4_scale_map(CUtensorMap* map, const void* scales, int64_t row_tiles, int K, int format, int tiles, int words = 128) {
  const int atoms = fp4_atoms(K, format);
  const int64_t dims[3] = {kFp4Atom / 4, atoms, row_tiles}, strides[2] = {kFp4Atom, (int64_t)atoms * kFp4Atom};
  const int box[3] = {words, format == W4A16_FP4_MX ? 2 : 4, tiles};
  return encode_map_3d(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, scales, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

cudaError_t launch_fp4_pair(const Fp4MmArgs& a, int pdl, cudaStream_t s);

}  // namespace w4a16
