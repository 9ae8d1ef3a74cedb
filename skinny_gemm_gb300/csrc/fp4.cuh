// fp4.cuh -- internal interface between the C-ABI (api.cu) and the kernels of
// the microscaled 4-bit matrices (fp4.cu, fp4_mm.cu), and their layout.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "w4a16.h"

namespace w4a16 {

// Scales are kept in atoms of 512 bytes, 128 rows x 4 blocks of K, as the
// tensor cores take them: byte 16 (row % 32) + 4 (row / 32) + block.  A matrix
// is [row tiles][atoms along K] of them.
constexpr int kFp4Rows = 128, kFp4Atom = 512;

__host__ __device__ constexpr int fp4_block(int format) { return format == W4A16_FP4_MX ? 32 : 16; }
__host__ __device__ constexpr int fp4_atoms(int K, int format) {  // along K
  return (K + 4 * fp4_block(format) - 1) / (4 * fp4_block(format));
}
__host__ __device__ constexpr int64_t fp4_row_tiles(int rows) { return ((int64_t)rows + kFp4Rows - 1) / kFp4Rows; }
inline int64_t fp4_scale_bytes(int rows, int K, int format) {  // of one expert
  return fp4_row_tiles(rows) * fp4_atoms(K, format) * kFp4Atom;
}

struct Fp4QuantArgs {
  const uint16_t* x;  // bf16 rows, x_stride elements apart
  int64_t x_stride;
  uint8_t* codes;
  uint8_t* scales;
  float* row_scale;
  int rows, K;     // rows of x
  int group;       // rows of one expert: their scale tiles start anew
  int format;
};
cudaError_t launch_fp4_quant(const Fp4QuantArgs& a, int pdl, cudaStream_t s);
cudaError_t launch_fp4_dequant(const w4a16_fp4& w, uint16_t* y, int pdl, cudaStream_t s);

// A tile of at most `nt` rows of one expert: `count` of them from place `place` on.
struct Fp4Tile {
  int expert, place, count, unused;
};
struct Fp4RouteArgs {
  const int32_t* ids;  // [rows]: the `top` choices of token after token
  int rows, top, E, nt;  // nt: most rows of a tile
  int span;            // places of a tile: nt up to a multiple of 128
  int32_t* place;      // [rows]: where the row's codes go, -1 for a bad id
  int32_t* row;        // [places]: the row of a place
  Fp4Tile* tiles;
  int32_t* count;      // [1]: tiles
  uint16_t* y;         // rows of bad ids are zeroed: y_row values each
  int64_t y_row;
  int* flags;
};
// The rows' places, and the tokens x (q.rows of them) quantised into those.
cudaError_t launch_fp4_route_quant(const Fp4RouteArgs& a, const Fp4QuantArgs& q, int pdl, cudaStream_t s);

struct Fp4MmArgs {
  const uint16_t* x;  // bf16 rows that the product quantises itself (fp4_mm_fuses), or nullptr and:
  int64_t x_stride;
  const uint8_t* xc;  // codes of the activations
  const uint8_t* xs;
  const float* xf;    // row factors or nullptr
  int64_t x_rows;     // rows of xc
  w4a16_fp4 w;
  uint16_t* y;
  int M, act;
  // routed (tiles != nullptr)
  const Fp4Tile* tiles;
  const int32_t* tile_count;
  const int32_t* row;
  int max_tiles, nt;
  const int32_t* ids; // routed: the experts of the rows; with x (fp4_mm_id_fuses), [M][top]
  int top;
  bool early;         // the weights (and ids) are complete before the kernel before this one lets it start
  int* flags;
  int fault_wait;     // debug (W4A16_FAULT=wait): the first CTA's first stage waits for bytes that never come
};
cudaError_t launch_fp4_mm(const Fp4MmArgs& a, int pdl, cudaStream_t s);
bool fp4_mm_fuses(const w4a16_fp4& w, int M);  // whether a product of M rows quantises them itself
bool fp4_mm_id_fuses(const w4a16_fp4& w, int T, int top);  // ... a routed one its tokens
int fp4_mm_tile(int M);  // rows of the activation tile that a call of M rows takes

}  // namespace w4a16
