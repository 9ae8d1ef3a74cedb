// fp4.cu -- microscaled 4-bit matrices: rows of bf16 into e2m1 codes and
// block scales and back, and the order of routed rows.
//
// e2m1 holds 0, 0.5, 1, 1.5, 2, 3, 4 and 6 with a sign.  Two formats:
//   mx  blocks of 32, scale 2^e, e = floor(log2(max |x|)) - 2 (at least -127)
//   nv  blocks of 16, scale s (e4m3) times a factor f of the whole row, the
//       smallest power of two (at least 2^-126) with max |x| of the row
//       <= 6 * 448 f;  s = e4m3(max |x| of the block / f / 6)
// and code = e2m1(x / scale), to nearest, ties to the even code, at most 6.
#include <cuda_runtime.h>

#include "common.cuh"
#include "fp4.cuh"
#include "ptx.cuh"

namespace w4a16 {
namespace {

using namespace ptx;

cudaError_t launch(const void* fn, dim3 grid, int threads, void** args, int pdl, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl > 0 ? 1 : 0;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

// Eight values to eight codes, value i in bits 4 i.
__device__ __forceinline__ uint32_t codes8(const float (&y)[8]) {
  uint32_t d;
  asm("{ .reg .b8 a, b, c, e;\n"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 e, %8, %7;\n"
      "mov.b32 %0, {a, b, c, e}; }"
      : "=r"(d)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return d;
}

// The largest |x| of eight bf16 values as bits (bf16 magnitudes order like integers).
__device__ __forceinline__ uint32_t peak8(const uint4& v) {
  const uint32_t a = __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), b = __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu);
  const uint32_t m = __vmaxu2(a, b);
  return max(m & 0xFFFFu, m >> 16);
}

// ... of its finite values.
__device__ __forceinline__ uint32_t finite_peak8(const uint4& v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = word_of(v, i) & 0x7FFF7FFFu, lo = w & 0xFFFFu, hi = w >> 16;
    m = max(m, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
  }
  return m;
}

// 2^e for e in -149 .. 127.
__device__ __forceinline__ float exp2i(int e) {
  return e >= -126 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(1u << (e + 149));
}

// The nv factor's exponent from the row's largest finite |x| (bf16 bits): 2688 = 1.3125 * 2^11, and 1.3125 has
// significand bits 0x28 of 7.  Subnormal peaks are below every bound that counts.
__device__ __forceinline__ int factor_exp(uint32_t peak) {
  const int e = (int)(peak >> 7) - 127 - 11 + ((peak & 0x7Fu) > 0x28u ? 1 : 0);
  return max(e, -126);
}

constexpr int kQuantThreads = 256;

// One CTA a row.  A thread takes eight values (16 bytes) at a time; two (nv) or four (mx) neighbours hold a block.
template <int FMT>
__global__ void __launch_bounds__(kQuantThreads) fp4_quant_kernel(Fp4QuantArgs p) {
  constexpr int kLanes = FMT == W4A16_FP4_MX ? 4 : 2;
  const int tid = threadIdx.x, chunks = p.K / 8;
  const int r = blockIdx.x;
  __shared__ uint32_t s_peak[kQuantThreads / 32];
  pdl_wait();
  pdl_launch_dependents();  // (not before: what the next kernel reads early is then complete)
  const uint16_t* x = p.x + (int64_t)r * p.x_stride;
  int e = 0;
  if (FMT == W4A16_FP4_NV) {
    uint32_t peak = 0;
    for (int c = tid; c < chunks; c += kQuantThreads) peak = max(peak, finite_peak8(*reinterpret_cast<const uint4*>(x + 8 * c)));
    peak = __reduce_max_sync(0xffffffffu, peak);
    if ((tid & 31) == 0) s_peak[tid >> 5] = peak;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQuantThreads / 32; ++i) peak = max(peak, s_peak[i]);
    e = factor_exp(peak);
  }
  const float inv = exp2i(-e);
  const int atoms = fp4_atoms(p.K, FMT);
  for (int j = 0; j < (p.place ? p.top : 1); ++j) {
    int64_t at = r;
    int64_t tile = (int64_t)(r / p.group) * fp4_row_tiles(p.group) + r % p.group / kFp4Rows;
    int lane_row = r % p.group % kFp4Rows;
    if (p.place) {
      at = p.place[(int64_t)r * p.top + j];
      if (at < 0) {  // no such expert: a row of zeros
        uint16_t* y = p.y + ((int64_t)r * p.top + j) * p.y_row;
        for (int64_t i = tid; i < p.y_row; i += kQuantThreads) y[i] = 0;
        continue;
      }
      tile = at / kFp4Rows;
      lane_row = (int)(at % kFp4Rows);
    }
    uint32_t* codes = reinterpret_cast<uint32_t*>(p.codes + at * (p.K / 2));
    uint8_t* scales = p.scales + tile * atoms * kFp4Atom + 16 * (lane_row & 31) + 4 * (lane_row >> 5);
    if (FMT == W4A16_FP4_NV && tid == 0) p.row_scale[at] = exp2i(e);
    // whole warps: blocks past K, up to the last atom's end, get scale 0
    for (int c0 = 0; c0 < atoms * 4 * kLanes; c0 += kQuantThreads) {
      const int c = c0 + tid;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (c < chunks) v = *reinterpret_cast<const uint4*>(x + 8 * c);
      uint32_t peak = peak8(v);
#pragma unroll
      for (int d = 1; d < kLanes; d *= 2) peak = max(peak, __shfl_xor_sync(0xffffffffu, peak, d));
      float y[8];
      widen8(v, y);
      uint32_t byte, code;
      if (FMT == W4A16_FP4_MX) {
        // floor(log2 peak) - 2 + 127 is the exponent field less 2; a subnormal peak gives 0
        byte = max((int)(peak >> 7) - 2, 0);
        const float s = exp2i(127 - (int)byte);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(y[i], s);
        code = codes8(y);
        if (peak >= 0x7F80u) byte = 0xFFu, code = 0;
      } else {
        const float want = __fdiv_rn(__fmul_rn(bf16_bits_to_f32((uint16_t)peak), inv), 6.0f);
        uint16_t pair;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(pair) : "f"(0.0f), "f"(want));
        byte = pair & 0xFFu;
        // s back in fp32: e4m3's bits at half the place of fp32's, times 2^120
        const float s = __fmul_rn(__uint_as_float(byte << 20), exp2i(120));
        if (byte == 0) {
          code = 0;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(__fmul_rn(y[i], inv), s);
          code = codes8(y);
        }
        if (peak >= 0x7F80u) byte = 0x7Fu, code = 0;
      }
      if (c < chunks) codes[c] = code;
      if (c < atoms * 4 * kLanes && c % kLanes == 0) {
        const int b = c / kLanes;
        scales[(int64_t)(b / 4) * kFp4Atom + b % 4] = (uint8_t)byte;
      }
    }
  }
}

// One CTA a row, eight values a thread: value = bf16(code * scale * factor), exact unless it leaves bf16's range.
__global__ void __launch_bounds__(kQuantThreads) fp4_dequant_kernel(w4a16_fp4 w, uint16_t* y) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t r = blockIdx.x;
  const int atoms = fp4_atoms(w.K, w.format), lanes = fp4_block(w.format) / 8;
  const int64_t n = r % w.rows, tile = r / w.rows * fp4_row_tiles(w.rows) + n / kFp4Rows;
  const uint8_t* scales = w.scales + tile * atoms * kFp4Atom + 16 * (n & 31) + 4 * (n % kFp4Rows >> 5);
  const float f = w.row_scale ? w.row_scale[r] : 1.0f;
  for (int c = threadIdx.x; c < w.K / 8; c += kQuantThreads) {
    const uint32_t code = *reinterpret_cast<const uint32_t*>(w.codes + r * (w.K / 2) + 4 * c);
    const int b = c / lanes;
    const uint32_t byte = scales[(int64_t)(b / 4) * kFp4Atom + b % 4];
    float s;
    if (w.format == W4A16_FP4_MX) s = byte == 255 ? __uint_as_float(0x7FC00000u) : exp2i((int)byte - 127);
    else s = (byte & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FC00000u) : __fmul_rn(__uint_as_float((byte & 0x7Fu) << 20 | (byte & 0x80u) << 24), exp2i(120));
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t pair;
      asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, a; }" : "=r"(pair) : "r"(code >> (8 * i)));
      const __half2 h = *reinterpret_cast<const __half2*>(&pair);
      const float lo = __fmul_rn(__fmul_rn(__low2float(h), s), f), hi = __fmul_rn(__fmul_rn(__high2float(h), s), f);
      out[i] = (uint32_t)f32_to_bf16_bits(lo) | ((uint32_t)f32_to_bf16_bits(hi) << 16);
    }
    *reinterpret_cast<uint4*>(y + r * w.K + 8 * c) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

// ---- routed rows ------------------------------------------------------------------------

constexpr int kRouteThreads = 1024;

// One CTA: rows counted by expert, the experts' tiles numbered, every row given a place in its expert's tiles.  A tile
// starts at a place that is a multiple of 128, as its scales do.  Which of an expert's rows takes which place is left
// to the order of the atomics: no output depends on it.
__global__ void __launch_bounds__(kRouteThreads) fp4_route_kernel(Fp4RouteArgs p) {
  extern __shared__ int s_count[];  // [E] rows, then the expert's first tile
  int* s_next = s_count + p.E;      // [E] rows placed
  __shared__ int s_warp[kRouteThreads / 32], s_base;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  for (int e = tid; e < p.E; e += kRouteThreads) s_count[e] = s_next[e] = 0;
  if (tid == 0) s_base = 0;
  __syncthreads();
  bool bad = false;
  for (int r = tid; r < p.rows; r += kRouteThreads) {
    const int e = p.ids[r];
    if (e >= 0 && e < p.E) atomicAdd(&s_count[e], 1);
    else bad = true;
  }
  if (bad) atomicOr(p.flags, W4A16_DEVICE_BAD_ID);
  __syncthreads();
  for (int e0 = 0; e0 < p.E; e0 += kRouteThreads) {
    const int e = e0 + tid, n = e < p.E ? s_count[e] : 0;
    const int tiles = (n + p.nt - 1) / p.nt;
    int sum = tiles;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int up = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += up;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    int first = s_base + sum - tiles;
    for (int w = 0; w < warp; ++w) first += s_warp[w];
    for (int t = 0; t < tiles; ++t)
      p.tiles[first + t] = Fp4Tile{e, (first + t) * kFp4Rows, min(p.nt, n - t * p.nt), 0};
    if (e < p.E) s_count[e] = first;
    __syncthreads();
    if (tid == kRouteThreads - 1) s_base = first + tiles;
    __syncthreads();
  }
  if (tid == 0) *p.count = s_base;
  for (int r = tid; r < p.rows; r += kRouteThreads) {
    const int e = p.ids[r];
    int place = -1;
    if (e >= 0 && e < p.E) {
      const int i = atomicAdd(&s_next[e], 1);
      place = (s_count[e] + i / p.nt) * kFp4Rows + i % p.nt;
      p.row[place] = r;
    }
    p.place[r] = place;
  }
}

}  // namespace

cudaError_t launch_fp4_quant(const Fp4QuantArgs& a, int pdl, cudaStream_t s) {
  void* args[] = {const_cast<Fp4QuantArgs*>(&a)};
  const void* fn = a.format == W4A16_FP4_MX ? (const void*)fp4_quant_kernel<W4A16_FP4_MX> : (const void*)fp4_quant_kernel<W4A16_FP4_NV>;
  return launch(fn, dim3((unsigned)a.rows), kQuantThreads, args, pdl, s);
}

cudaError_t launch_fp4_dequant(const w4a16_fp4& w, uint16_t* y, int pdl, cudaStream_t s) {
  void* args[] = {const_cast<w4a16_fp4*>(&w), &y};
  return launch((const void*)fp4_dequant_kernel, dim3((unsigned)(w.rows * w.experts)), kQuantThreads, args, pdl, s);
}

cudaError_t launch_fp4_route(const Fp4RouteArgs& a, int pdl, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kRouteThreads);
  cfg.dynamicSmemBytes = (size_t)a.E * 8;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fp4_route_kernel, a);
}

}  // namespace w4a16
