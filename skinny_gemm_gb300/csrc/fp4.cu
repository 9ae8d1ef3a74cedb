// fp4.cu -- microscaled 4-bit matrices: rows of bf16 into e2m1 codes and
// block scales and back, and the order of routed rows.
//
// e2m1 holds 0, 0.5, 1, 1.5, 2, 3, 4 and 6 with a sign.  Two formats:
//   mx  blocks of 32, scale 2^e, e = floor(log2(max |x|)) - 2 (at least -127)
//   nv  blocks of 16, scale s (e4m3) times a factor f of the whole row, the
//       smallest power of two (at least 2^-126) with max |x| of the row
//       <= 6 * 448 f;  s = e4m3(max |x| of the block / f / 6)
// and code = e2m1(x / scale), to nearest, ties to the even code, at most 6.
#include <cuda_fp16.h>
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
__device__ __forceinline__ uint32_t codes8(const float* y) {
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

// Sixteen bf16 values, 32 bytes.
struct Vec16 {
  uint4 a, b;
};
__device__ __forceinline__ Vec16 load16(const uint16_t* p) { return Vec16{ld_nc_v4(p), ld_nc_v4(p + 8)}; }
__device__ __forceinline__ Vec16 zero16() { return Vec16{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}; }

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

// 2^e for e in -126 .. 127.
__device__ __forceinline__ float exp2n(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The nv factor's exponent from the row's largest finite |x| (bf16 bits): 2688 = 1.3125 * 2^11, and 1.3125 has
// significand bits 0x28 of 7.  Subnormal peaks are below every bound that counts.
__device__ __forceinline__ int factor_exp(uint32_t peak) {
  const int e = (int)(peak >> 7) - 127 - 11 + ((peak & 0x7Fu) > 0x28u ? 1 : 0);
  return max(e, -126);
}

__device__ __forceinline__ uint32_t peak16(const Vec16& v) { return max(peak8(v.a), peak8(v.b)); }
__device__ __forceinline__ uint32_t finite_peak16(const Vec16& v) { return max(finite_peak8(v.a), finite_peak8(v.b)); }

__device__ __forceinline__ float rcp(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// Two sums a b + c at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{ .reg .b64 a, b, c; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 a, a, b, c; mov.b64 {%0, %1}, a; }"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{ .reg .b64 a, b; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 a, a, b; mov.b64 {%0, %1}, a; }"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

constexpr int kQuantThreads = 256;  // of the way back
constexpr int kQuantMost = 768;     // threads of a row: 80 registers each

// Sixteen values to codes and their block's scale byte; peak is the block's largest |x| (bf16 bits).
//
// nv.  The codes depend on which side of a border (a multiple of 1/4 up to 5) the quotient y = x / (s f) lies, ties
// included.  x has 8 significant bits and s 4, so that a y that is not on a border is at least 2^-10 from it.  x times an
// approximate reciprocal is off by 2^-20 at most; rounded to a multiple of 2^-12 (by adding and taking off 1.5 * 2^11) it is
// on a border where y is, and on y's side of it elsewhere.  The same for the scale: p / f / 6 against the borders of
// e4m3, 5 significant bits: at least 2^-9 of it away, or on it; kept to 2^-16 of it.
template <int FMT>
__device__ __forceinline__ uint2 block16(const Vec16& v, uint32_t peak, int e, uint32_t& byte) {
  float y[16];
  widen8(v.a, y);
  widen8(v.b, y + 8);
  if (FMT == W4A16_FP4_MX) {
    // floor(log2 peak) - 2 + 127 is the exponent field less 2; a subnormal peak gives 0
    byte = max((int)(peak >> 7) - 2, 0);
    const float s = exp2n(127 - (int)byte);
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(y[i], s);
    if (peak >= 0x7F80u) byte = 0xFFu;
  } else {
    const float p = __fmul_rn(bf16_bits_to_f32((uint16_t)peak), exp2n(-e));
    const float want = __uint_as_float((__float_as_uint(__fmul_rn(p, 1.0f / 6.0f)) + 64u) & ~127u);
    uint16_t pair;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(pair) : "f"(0.0f), "f"(want));
    byte = pair & 0xFFu;
    // the scale in fp32: e4m3's bits at half the place of fp32's, times 2^120
    float s = __fmul_rn(__uint_as_float(byte << 20), exp2n(120));
    if (e < -90) {  // s f might leave fp32's normal range
      const float inv = exp2n(-e);
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(y[i], inv);
    } else {
      s = __fmul_rn(s, exp2n(e));
    }
    const float r = byte ? rcp(s) : 0.0f;
    const float2 rr = make_float2(r, r), up = make_float2(3072.0f, 3072.0f), down = make_float2(-3072.0f, -3072.0f);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 q = add2(fma2(make_float2(y[i], y[i + 1]), rr, up), down);
      y[i] = q.x;
      y[i + 1] = q.y;
    }
    if (peak >= 0x7F80u) byte = 0x7Fu;
  }
  if (peak >= 0x7F80u) return make_uint2(0, 0);
  return make_uint2(codes8(y), codes8(y + 8));
}

// One CTA a row; a thread holds up to C units of sixteen values (32 bytes) in registers between the row's peak and its
// codes, longer rows are read again.  A thread has a whole nv block, two neighbours an mx one.  What bounds it is HBM (2
// bytes a value in, 0.56 out) for many rows, and a load, the row's reduction and the launch for few.
template <int FMT, int C, bool ROUTED>
__global__ void __launch_bounds__(kQuantMost, 1) fp4_quant_kernel(Fp4QuantArgs p) {
  constexpr int kWord = FMT == W4A16_FP4_MX ? 8 : 4;  // units of an atom's word of four scales
  const int tid = threadIdx.x, threads = blockDim.x, units = p.K / 16;
  const int n = blockIdx.x;  // row of expert blockIdx.y
  const int64_t r = (int64_t)blockIdx.y * p.group + n;
  __shared__ uint32_t s_peak[32];
  pdl_wait();
  pdl_launch_dependents();  // (not before: what the next kernel reads early is then complete)
  const uint16_t* x = p.x + r * p.x_stride;
  Vec16 v[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = i * threads + tid;
    v[i] = c < units ? load16(x + 16 * c) : zero16();
  }
  int e = 0;
  if (FMT == W4A16_FP4_NV) {
    auto over_row = [&](uint32_t peak) {
      peak = __reduce_max_sync(0xffffffffu, peak);
      if (threads > 32) {
        if ((tid & 31) == 0) s_peak[tid >> 5] = peak;
        __syncthreads();
        peak = __reduce_max_sync(0xffffffffu, (tid & 31) < threads / 32 ? s_peak[tid & 31] : 0u);
        __syncthreads();
      }
      return peak;
    };
    uint32_t peak = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) peak = max(peak, peak16(v[i]));
    for (int c = C * threads + tid; c < units; c += threads) peak = max(peak, peak16(load16(x + 16 * c)));
    peak = over_row(peak);
    if (peak >= 0x7F80u) {  // a NaN or an infinity in the row
      peak = 0;
#pragma unroll
      for (int i = 0; i < C; ++i) peak = max(peak, finite_peak16(v[i]));
      for (int c = C * threads + tid; c < units; c += threads) peak = max(peak, finite_peak16(load16(x + 16 * c)));
      peak = over_row(peak);
    }
    e = factor_exp(peak);
  }
  const int atoms = fp4_atoms(p.K, FMT), all = atoms * kWord;  // units with those past K that fill the last atom
#pragma unroll 1
  for (int j = 0; j < (ROUTED ? p.top : 1); ++j) {
    int64_t at = r, tile;
    int lane_row;
    if (ROUTED) {
      at = p.place[r * p.top + j];
      if (at < 0) {  // no such expert: a row of zeros
        uint16_t* y = p.y + (r * p.top + j) * p.y_row;
        for (int64_t i = tid; i < p.y_row; i += threads) y[i] = 0;
        continue;
      }
      tile = at / kFp4Rows;
      lane_row = (int)(at % kFp4Rows);
    } else {
      tile = (int64_t)blockIdx.y * fp4_row_tiles(p.group) + n / kFp4Rows;
      lane_row = n % kFp4Rows;
    }
    uint2* codes = reinterpret_cast<uint2*>(p.codes + at * (p.K / 2)) + tid;
    if (FMT == W4A16_FP4_NV && tid == 0) p.row_scale[at] = exp2n(e);
    // a word of an atom is four blocks' bytes, kWord threads' units; the CTA's threads are a multiple of that
    uint8_t* words = p.scales + tile * atoms * kFp4Atom + 16 * (lane_row & 31) + 4 * (lane_row >> 5) + tid / kWord * kFp4Atom;
    const int place = 8 * (tid / (kWord / 4) % 4);
    const bool first = tid % kWord == 0;
    auto write = [&](int c0, const Vec16& w) {  // units c0 + tid (whole warps)
      uint32_t peak = peak16(w);
      if (FMT == W4A16_FP4_MX) peak = max(peak, __shfl_xor_sync(0xffffffffu, peak, 1));
      uint32_t byte;
      const uint2 code = block16<FMT>(w, peak, e, byte);
      if (tid < units - c0) codes[c0] = code;
      uint32_t word = byte << place;
      word |= __shfl_xor_sync(0xffffffffu, word, kWord / 4);
      word |= __shfl_xor_sync(0xffffffffu, word, kWord / 2);
      if (first && tid < all - c0) *reinterpret_cast<uint32_t*>(words + c0 / kWord * kFp4Atom) = word;
    };
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i * threads < all) write(i * threads, v[i]);
#pragma unroll 1
    for (int c0 = C * threads; c0 < all; c0 += threads) write(c0, c0 + tid < units ? load16(x + 16 * (c0 + tid)) : zero16());
  }
}

// Units of sixteen values: value = bf16(code * scale * factor), exact unless it leaves bf16's range.  code * scale is
// exact in fp16 for nv (6 significant bits, 2^-10 to 2688).
constexpr int kBack = 1;  // units a thread

__global__ void __launch_bounds__(kQuantThreads) fp4_dequant_kernel(w4a16_fp4 w, uint16_t* y) {
  pdl_wait();
  pdl_launch_dependents();
  const int n = blockIdx.x, part = blockIdx.z;  // row of expert blockIdx.y
  const int64_t r = (int64_t)blockIdx.y * w.rows + n;
  const bool mx = w.format == W4A16_FP4_MX;
  const int atoms = fp4_atoms(w.K, w.format), units = w.K / 16;
  const int64_t tile = (int64_t)blockIdx.y * fp4_row_tiles(w.rows) + n / kFp4Rows;
  const uint8_t* scales = w.scales + tile * atoms * kFp4Atom + 16 * (n & 31) + 4 * (n % kFp4Rows >> 5);
  const float factor = w.row_scale ? w.row_scale[r] : 1.0f;
  uint2 code[kBack];
  uint32_t byte[kBack];
#pragma unroll
  for (int i = 0; i < kBack; ++i) {
    const int c = (part * kBack + i) * kQuantThreads + threadIdx.x, b = mx ? c / 2 : c;
    code[i] = make_uint2(0, 0);
    byte[i] = 0;
    if (c < units) {
      code[i] = *reinterpret_cast<const uint2*>(w.codes + r * (w.K / 2) + 8 * (int64_t)c);
      byte[i] = scales[(int64_t)(b / 4) * kFp4Atom + b % 4];
    }
  }
#pragma unroll
  for (int i = 0; i < kBack; ++i) {
    const int c = (part * kBack + i) * kQuantThreads + threadIdx.x;
    if (c >= units) break;
    float s = 1.0f, f = factor;
    if (mx) f = __fmul_rn(byte[i] == 255 ? __uint_as_float(0x7FC00000u) : exp2i((int)byte[i] - 127), factor);
    else s = (byte[i] & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FC00000u) : __fmul_rn(__uint_as_float((byte[i] & 0x7Fu) << 20 | (byte[i] & 0x80u) << 24), exp2n(120));
    const __half2 sh = __float2half2_rn(s);
    uint32_t out[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t pair;
      asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, a; }" : "=r"(pair) : "r"((k < 4 ? code[i].x : code[i].y) >> (8 * (k % 4))));
      const float2 h = __half22float2(__hmul2(*reinterpret_cast<const __half2*>(&pair), sh));
      const __nv_bfloat162 o = __floats2bfloat162_rn(__fmul_rn(h.x, f), __fmul_rn(h.y, f));
      out[k] = *reinterpret_cast<const uint32_t*>(&o);
    }
    uint4* to = reinterpret_cast<uint4*>(y + r * w.K + 16 * (int64_t)c);
    to[0] = make_uint4(out[0], out[1], out[2], out[3]);
    to[1] = make_uint4(out[4], out[5], out[6], out[7]);
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

namespace {

template <int FMT>
cudaError_t quant_f(const Fp4QuantArgs& a, int pdl, cudaStream_t s) {
  void* args[] = {const_cast<Fp4QuantArgs*>(&a)};
  // Few rows: a thread a unit, for the latency (1 x 2560 1.4 us; 333 x 2304 1.6 us so and with four units a thread).
  // Many: four, whose loads are in flight together; us with one / two / four, nv: 4096 x 2560 6.9 / 6.2 / 6.2, 4001 x
  // 10240 47 / 22.5 / 20.1, 8192 x 16384 119 / 71 / 55 (HBM's 51).
  const int all = fp4_atoms(a.K, FMT) * 4 * fp4_block(FMT) / 16;
  const bool one = !a.place && a.rows <= 152 && all <= kQuantMost;
  int threads = ((one ? all : (all + 3) / 4) + 31) / 32 * 32;
  threads = threads > kQuantMost ? kQuantMost : threads;
  const void* fn = a.place ? (const void*)fp4_quant_kernel<FMT, 4, true>
                   : one   ? (const void*)fp4_quant_kernel<FMT, 1, false>
                           : (const void*)fp4_quant_kernel<FMT, 4, false>;
  return launch(fn, dim3((unsigned)a.group, (unsigned)(a.rows / a.group)), threads, args, pdl, s);
}

}  // namespace

cudaError_t launch_fp4_quant(const Fp4QuantArgs& a, int pdl, cudaStream_t s) {
  return a.format == W4A16_FP4_MX ? quant_f<W4A16_FP4_MX>(a, pdl, s) : quant_f<W4A16_FP4_NV>(a, pdl, s);
}

cudaError_t launch_fp4_dequant(const w4a16_fp4& w, uint16_t* y, int pdl, cudaStream_t s) {
  const int64_t parts = (w.K / 16 + kBack * kQuantThreads - 1) / (kBack * kQuantThreads);
  void* args[] = {const_cast<w4a16_fp4*>(&w), &y};
  if (parts > 65535) return cudaErrorInvalidConfiguration;
  return launch((const void*)fp4_dequant_kernel, dim3((unsigned)w.rows, (unsigned)w.experts, (unsigned)parts), kQuantThreads, args, pdl, s);
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
