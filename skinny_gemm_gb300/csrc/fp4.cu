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
#include "fp4_quant.cuh"
#include "ptx.cuh"

namespace w4a16 {
namespace {

using namespace ptx;
using namespace fp4;

cudaError_t launch(const void* fn, dim3 grid, int threads, size_t smem, void** args, int pdl, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl > 0 ? 1 : 0;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

constexpr int kBackThreads = 256;   // most threads of the way back
constexpr int kGridZ = 65535;       // most CTAs of a grid's third axis
constexpr int kQuantMost = 768;     // threads of a row: 80 registers each
constexpr int kFoundMost = 1 << 20; // tokens x routed rows, up to which every token's CTA finds its places itself

// ---- routed rows ------------------------------------------------------------------------
//
// Rows are counted by expert, the experts' tiles numbered, every row given a place in its expert's tiles.  A tile starts
// at a place that is a multiple of 128, as its scales do.

// The tiles of the experts, from their counts of rows; count[e] becomes the expert's first tile.  All threads of a CTA
// (whole warps); WRITE: the tiles are written down.
template <bool WRITE>
__device__ __forceinline__ void number_tiles(const Fp4RouteArgs& p, int* count) {
  __shared__ int s_warp[32], s_base;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  if (tid == 0) s_base = 0;
  __syncthreads();
  for (int e0 = 0; e0 < p.E; e0 += threads) {
    const int e = e0 + tid, n = e < p.E ? count[e] : 0;
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
    if (WRITE)
      for (int t = 0; t < tiles; ++t)
        p.tiles[first + t] = Fp4Tile{e, (first + t) * p.span, min(p.nt, n - t * p.nt), 0};
    if (e < p.E) count[e] = first;
    __syncthreads();
    if (tid == threads - 1) s_base = first + tiles;
    __syncthreads();
  }
  if (WRITE && tid == 0) *p.count = s_base;
}

// The places of token t's choices into to[top], found by every CTA for itself: it counts all ids, and those of the
// tokens before its own.  counts: [2 E].  (500 tokens x 4 of 64 experts: 5.7 us, the counting in a launch of its own and
// the places read back 12.)
__device__ __forceinline__ void place_rows(const Fp4RouteArgs& p, int t, int* to, int* counts) {
  const int tid = threadIdx.x, threads = blockDim.x;
  int *count = counts, *before = counts + p.E;
  for (int e = tid; e < 2 * p.E; e += threads) counts[e] = 0;
  __syncthreads();
  bool bad = false;
  for (int r = tid; r < p.rows; r += threads) {
    const int e = p.ids[r];
    if (e >= 0 && e < p.E) {
      atomicAdd(count + e, 1);
      if (r < t * p.top) atomicAdd(before + e, 1);
    } else {
      bad = true;
    }
  }
  if (bad && t == 0) atomicOr(p.flags, W4A16_DEVICE_BAD_ID);
  __syncthreads();
  if (t == 0) number_tiles<true>(p, count);
  else number_tiles<false>(p, count);
  __syncthreads();
  for (int j = tid; j < p.top; j += threads) {
    const int r = t * p.top + j, e = p.ids[r];
    int place = -1;
    if (e >= 0 && e < p.E) {
      int i = before[e];
      for (int k = 0; k < j; ++k) i += p.ids[t * p.top + k] == e;  // (an expert may be chosen twice)
      place = (count[e] + i / p.nt) * p.span + i % p.nt;
      p.row[place] = r;
    }
    to[j] = place;
  }
  __syncthreads();
}

// The same in one CTA for many rows.  Which of an expert's rows takes which place is left to the order of the atomics: no
// output depends on it.
constexpr int kRouteThreads = 1024;

__global__ void __launch_bounds__(kRouteThreads) fp4_route_kernel(Fp4RouteArgs p) {
  extern __shared__ int s_count[];  // [E] rows, then the expert's first tile
  int* s_next = s_count + p.E;      // [E] rows placed
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  for (int e = tid; e < p.E; e += kRouteThreads) s_count[e] = s_next[e] = 0;
  __syncthreads();
  bool bad = false;
  for (int r = tid; r < p.rows; r += kRouteThreads) {
    const int e = p.ids[r];
    if (e >= 0 && e < p.E) atomicAdd(&s_count[e], 1);
    else bad = true;
  }
  if (bad) atomicOr(p.flags, W4A16_DEVICE_BAD_ID);
  __syncthreads();
  number_tiles<true>(p, s_count);
  __syncthreads();
  for (int r = tid; r < p.rows; r += kRouteThreads) {
    const int e = p.ids[r];
    int place = -1;
    if (e >= 0 && e < p.E) {
      const int i = atomicAdd(&s_next[e], 1);
      place = (s_count[e] + i / p.nt) * p.span + i % p.nt;
      p.row[place] = r;
    }
    p.place[r] = place;
  }
}

// One CTA a row; a thread holds up to C units of sixteen values (32 bytes) in registers between the row's peak and its
// codes, longer rows are read again.  A thread has a whole nv block, two neighbours an mx one.  What bounds it is HBM (2
// bytes a value in, 0.56 out) for many rows, and a load, the row's reduction and the launch for few.
//
// ROUTE: the row is a token, whose codes go to the places of its choices; the places are read (kGiven) or found here
// (kFound: every CTA counts all ids, see place_rows).
enum Route { kNone, kGiven, kFound };

template <int FMT, int C, int ROUTE>
__global__ void __launch_bounds__(kQuantMost, 1) fp4_quant_kernel(Fp4QuantArgs p, Fp4RouteArgs route) {
  constexpr int kWord = FMT == W4A16_FP4_MX ? 8 : 4;  // units of an atom's word of four scales
  const int tid = threadIdx.x, threads = blockDim.x, units = p.K / 16;
  const int n = blockIdx.x;  // row of expert blockIdx.y
  const int64_t r = (int64_t)blockIdx.y * p.group + n;
  extern __shared__ int s_route[];  // ROUTE: [top] places, then what place_rows counts
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
  if (ROUTE == kGiven) {
    for (int j = tid; j < route.top; j += threads) s_route[j] = route.place[r * route.top + j];
    __syncthreads();
  }
  if (ROUTE == kFound) place_rows(route, n, s_route, s_route + route.top);
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
  // a word of an atom is four blocks' bytes, kWord threads' units; the CTA's threads are a multiple of that
  const int shift = 8 * (tid / (kWord / 4) % 4);
  const bool first = tid % kWord == 0;
  auto write = [&](int c0, const Vec16& w) {  // units c0 + tid (whole warps)
    uint32_t peak = peak16(w);
    if (FMT == W4A16_FP4_MX) peak = max(peak, __shfl_xor_sync(0xffffffffu, peak, 1));
    uint32_t byte;
    const uint2 code = block16<FMT>(w, peak, e, byte);
    uint32_t word = byte << shift;
    word |= __shfl_xor_sync(0xffffffffu, word, kWord / 4);
    word |= __shfl_xor_sync(0xffffffffu, word, kWord / 2);
    auto put = [&](int64_t at, int64_t tile, int lane_row) {
      if (tid < units - c0) reinterpret_cast<uint2*>(p.codes + at * (p.K / 2))[c0 + tid] = code;
      if (first && tid < all - c0)
        *reinterpret_cast<uint32_t*>(p.scales + (tile * atoms + (c0 + tid) / kWord) * kFp4Atom + 16 * (lane_row & 31) + 4 * (lane_row >> 5)) = word;
    };
    if (ROUTE == kNone) {
      put(r, (int64_t)blockIdx.y * fp4_row_tiles(p.group) + n / kFp4Rows, n % kFp4Rows);
    } else {
      for (int j = 0; j < route.top; ++j)
        if (const int at = s_route[j]; at >= 0) put(at, at / kFp4Rows, at % kFp4Rows);
    }
  };
#pragma unroll
  for (int i = 0; i < C; ++i)
    if (i * threads < all) write(i * threads, v[i]);
#pragma unroll 1
  for (int c0 = C * threads; c0 < all; c0 += threads) write(c0, c0 + tid < units ? load16(x + 16 * (c0 + tid)) : zero16());
  if constexpr (ROUTE == kNone) {
    if (tid == 0 && (FMT == W4A16_FP4_NV || p.row_scale)) p.row_scale[r] = FMT == W4A16_FP4_NV ? exp2n(e) : 1.0f;
  } else {
    for (int j = 0; j < route.top; ++j) {
      const int at = s_route[j];
      if (at >= 0) {
        if (FMT == W4A16_FP4_NV && tid == 0) p.row_scale[at] = exp2n(e);
      } else {  // no such expert: a row of zeros
        uint16_t* y = route.y + (r * route.top + j) * route.y_row;
        for (int64_t i = tid; i < route.y_row; i += threads) y[i] = 0;
      }
    }
  }
}

// Units of sixteen values: value = bf16(code * scale * factor), exact unless it leaves bf16's range.  code * scale is
// exact in fp16 for nv (6 significant bits, 2^-10 to 2688).  A thread has one unit (of rows past 2^28 values, more).
__global__ void __launch_bounds__(kBackThreads) fp4_dequant_kernel(w4a16_fp4 w, uint16_t* y) {
  pdl_wait();
  pdl_launch_dependents();
  const int n = blockIdx.x, part = blockIdx.z;  // row of expert blockIdx.y
  const int64_t r = (int64_t)blockIdx.y * w.rows + n;
  const bool mx = w.format == W4A16_FP4_MX;
  const int atoms = fp4_atoms(w.K, w.format), units = w.K / 16;
  const int64_t tile = (int64_t)blockIdx.y * fp4_row_tiles(w.rows) + n / kFp4Rows;
  const uint8_t* scales = w.scales + tile * atoms * kFp4Atom + 16 * (n & 31) + 4 * (n % kFp4Rows >> 5);
  const float factor = w.row_scale ? w.row_scale[r] : 1.0f;
  for (int c = part * blockDim.x + threadIdx.x; c < units; c += gridDim.z * blockDim.x) {
    const int b = mx ? c / 2 : c;
    const uint2 code = *reinterpret_cast<const uint2*>(w.codes + r * (w.K / 2) + 8 * (int64_t)c);
    const uint32_t byte = scales[(int64_t)(b / 4) * kFp4Atom + b % 4];
    float s = 1.0f, f = factor;
    if (mx) {
      const float e = byte == 255 ? __uint_as_float(0x7FC00000u) : exp2i((int)byte - 127);
      f = __fmul_rn(e, factor);
      // past fp32's range, 2^8 of it go to the codes (exact in fp16), and what is still past it makes all of them infinite but 0
      if (isinf(f)) s = 256.0f, f = fmaxf(fminf(__fmul_rn(__fmul_rn(e, 1.0f / 256), factor), 3.4028235e38f), -3.4028235e38f);
    } else s = (byte & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FC00000u) : __fmul_rn(__uint_as_float((byte & 0x7Fu) << 20 | (byte & 0x80u) << 24), exp2n(120));
    const __half2 sh = __float2half2_rn(s);
    uint32_t out[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t pair;
      asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, a; }" : "=r"(pair) : "r"((k < 4 ? code.x : code.y) >> (8 * (k % 4))));
      const float2 h = __half22float2(__hmul2(*reinterpret_cast<const __half2*>(&pair), sh));
      const __nv_bfloat162 o = __floats2bfloat162_rn(__fmul_rn(h.x, f), __fmul_rn(h.y, f));
      out[k] = *reinterpret_cast<const uint32_t*>(&o);
    }
    uint4* to = reinterpret_cast<uint4*>(y + r * w.K + 16 * (int64_t)c);
    to[0] = make_uint4(out[0], out[1], out[2], out[3]);
    to[1] = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

}  // namespace

namespace {

template <int FMT>
cudaError_t quant_f(const Fp4QuantArgs& a, int pdl, cudaStream_t s) {
  Fp4RouteArgs none = {};
  void* args[] = {const_cast<Fp4QuantArgs*>(&a), &none};
  // Up to some 1600 units an SM: a thread a unit, for the latency.  A product's call in us so / with four or five units a
  // thread: 256 rows x 2560 9.7 / 10.2, 512 x 2560 14.4 / 16.4, 800 x 2304 15.3 / 16.9, 1500 x 2560 (gated, mx) 35.4 / 37.0,
  // 300 x 10240 16.4 / 17.0; but 512 x 10240 19.8 / 17.6, 777 x 10240 26.7 / 22.1.
  // More: four or five, whose loads are in flight together, whichever leaves fewer threads without; us with one / two /
  // four / five, nv: 4096 x 2560 6.9 / 6.2 / 6.4 / 5.5, 4001 x 10240 47 / 22.5 / 21.0 / 19.0 (HBM's 15.6), 8192 x 16384
  // 119 / 71 / 56.3 / 59.3 (HBM's 51).
  const int all = fp4_atoms(a.K, FMT) * 4 * fp4_block(FMT) / 16;
  const bool one = (int64_t)a.rows * all <= 152 * 1600 && all <= kQuantMost;
  auto threads_of = [&](int units) { return ((all + units - 1) / units + 31) / 32 * 32; };
  const int each = one ? 1 : 5 * threads_of(5) <= 4 * threads_of(4) ? 5 : 4;
  const int threads = threads_of(each) > kQuantMost ? kQuantMost : threads_of(each);
  const void* fn = each == 1   ? (const void*)fp4_quant_kernel<FMT, 1, kNone>
                   : each == 4 ? (const void*)fp4_quant_kernel<FMT, 4, kNone>
                               : (const void*)fp4_quant_kernel<FMT, 5, kNone>;
  return launch(fn, dim3((unsigned)a.group, (unsigned)(a.rows / a.group)), threads, 0, args, pdl, s);
}

template <int FMT>
cudaError_t route_quant_f(const Fp4RouteArgs& r, const Fp4QuantArgs& q, bool found, int pdl, cudaStream_t s) {
  void* args[] = {const_cast<Fp4QuantArgs*>(&q), const_cast<Fp4RouteArgs*>(&r)};
  const int all = fp4_atoms(q.K, FMT) * 4 * fp4_block(FMT) / 16;
  // two units a thread, and at least 256 to count the ids
  int threads = ((all + 1) / 2 + 31) / 32 * 32;
  if (found && threads < 256) threads = 256;
  threads = threads > kQuantMost ? kQuantMost : threads;
  const size_t smem = 4 * ((size_t)r.top + (found ? 2 * (size_t)r.E : 0));
  const void* fn = found ? (const void*)fp4_quant_kernel<FMT, 2, kFound> : (const void*)fp4_quant_kernel<FMT, 2, kGiven>;
  return launch(fn, dim3((unsigned)q.rows), threads, smem, args, pdl, s);
}

}  // namespace

cudaError_t launch_fp4_quant(const Fp4QuantArgs& a, int pdl, cudaStream_t s) {
  return a.format == W4A16_FP4_MX ? quant_f<W4A16_FP4_MX>(a, pdl, s) : quant_f<W4A16_FP4_NV>(a, pdl, s);
}

cudaError_t launch_fp4_route_quant(const Fp4RouteArgs& r, const Fp4QuantArgs& q, int pdl, cudaStream_t s) {
  // Every token's CTA reads all ids, which grows with their number times the tokens'.  The call in us so / with a launch
  // for the places: 8 tokens x 1 9.5 / 11.0, 64 x 8 21.3 / 23.3, 500 x 4 31.9 / 32.9, 2000 x 2 50 / 40, 4000 x 1 63 / 43.
  const bool found = (int64_t)q.rows * r.rows <= kFoundMost;
  if (!found) {
    void* args[] = {const_cast<Fp4RouteArgs*>(&r)};
    if (cudaError_t e = launch((const void*)fp4_route_kernel, dim3(1), kRouteThreads, (size_t)r.E * 8, args, pdl, s)) return e;
  }
  return q.format == W4A16_FP4_MX ? route_quant_f<W4A16_FP4_MX>(r, q, found, pdl, s) : route_quant_f<W4A16_FP4_NV>(r, q, found, pdl, s);
}

cudaError_t launch_fp4_dequant(const w4a16_fp4& w, uint16_t* y, int pdl, cudaStream_t s) {
  // equal parts of a row, of whole warps
  const int units = w.K / 16, all = (units + kBackThreads - 1) / kBackThreads, parts = all < kGridZ ? all : kGridZ;
  const int threads = parts < kGridZ ? ((units + parts - 1) / parts + 31) / 32 * 32 : kBackThreads;
  void* args[] = {const_cast<w4a16_fp4*>(&w), &y};
  return launch((const void*)fp4_dequant_kernel, dim3((unsigned)w.rows, (unsigned)w.experts, (unsigned)parts), threads, 0, args, pdl, s);
}

}  // namespace w4a16
