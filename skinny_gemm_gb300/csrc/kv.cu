// kv.cu -- the paged key/value cache in 8 bits: block tables and slots from
// request lengths (w4a16_kv_plan) and the quantising write (w4a16_kv_append).
// The formulas are those of include/w4a16.h "Paged key/value cache".
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv.cuh"
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

// ---- plan ----------------------------------------------------------------------------------
//
// Two exclusive prefix sums over the requests (new tokens, blocks to take),
// then every token and every taken block finds its request by bisection in
// the sums.  A call is a few kilobytes: the floor is the launch and three
// dependent loads (lengths, table or free list, store).  Every CTA computes
// the sums itself (requests in chunks of kPlanThreads, the running totals
// carried in registers), so nothing is handed between CTAs and one launch
// does it all.  On the GPU 8 requests take 2.2 us, 200 requests of five tokens
// 3.7 us, 333 prompt chunks (0.57 MB in and out) 5.2 us.

constexpr int kPlanThreads = 1024;
constexpr int kPlanTokens = 2048;  // tokens per CTA

struct PlanParams {
  KvPlanArgs a;
  int shift;    // log2(block)
  int advance;  // lens is cached, and several CTAs read it: kv_advance_kernel writes it
};

// What is taken for request b's cached tokens, whatever its entry says.
__device__ __forceinline__ int cached_of(const KvPlanArgs& a, int cached) { return min(max(cached, 0), INT32_MAX - a.T); }

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(PlanParams p) {
  __shared__ int s_cu[kPlanThreads + 1], s_first[kPlanThreads + 1], s_cached[kPlanThreads];
  __shared__ int s_warp[2][32];
  const KvPlanArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_thr = blockDim.x;
  const int t0 = blockIdx.x * kPlanTokens, t1 = min(t0 + kPlanTokens, a.T);
  pdl_launch_dependents();
  pdl_wait();
  const int start = a.head ? *a.head : 0, head = max(start, 0);
  int tok = 0;  // tokens and blocks of the requests before this chunk; both stay within T
  int taken = 0;
  bool bad = start < 0;
  for (int b0 = 0; b0 < a.B; b0 += n_thr) {
    const int b = b0 + tid, n = min(n_thr, a.B - b0);
    int cached = 0, fresh = 0;
    if (b < a.B) {
      cached = a.cached[b];
      fresh = a.fresh[b];
      if (cached < 0 || fresh < 0 || fresh > a.T || cached > INT32_MAX - a.T) {
        bad = true;
        cached = cached_of(a, cached);
        fresh = min(max(fresh, 0), a.T);
      }
    }
    // inclusive sum over the chunk, saturated at T after every step (T < 2^30: no overflow)
    int c = fresh;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, c, d);
      if (lane >= d) c = min(c + o, a.T);
    }
    if (lane == 31) s_warp[0][warp] = c;
    __syncthreads();
    if (warp == 0) {
      int w = lane < (n_thr >> 5) ? s_warp[0][lane] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w = min(w + o, a.T);
      }
      s_warp[0][lane] = w;
    }
    __syncthreads();
    const int incl = min((warp ? min(c + s_warp[0][warp - 1], a.T) : c) + tok, a.T);
    if (tid == 0) s_cu[0] = tok;
    s_cu[tid + 1] = incl;
    __syncthreads();
    const int mine = incl - s_cu[tid];  // tokens this request gets (fewer only past T)
    bad |= mine < fresh;
    const int len = cached + mine;
    const int have = min((int)(((int64_t)cached + a.block - 1) >> p.shift), a.max_blocks);
    const int want = (int)(((int64_t)len + a.block - 1) >> p.shift), need = min(want, a.max_blocks);
    bad |= need < want;
    const int take = b < a.B ? need - have : 0;  // at most the request's new tokens
    int f = take;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, f, d);
      if (lane >= d) f += o;
    }
    if (lane == 31) s_warp[1][warp] = f;
    __syncthreads();
    if (warp == 0) {
      int w = lane < (n_thr >> 5) ? s_warp[1][lane] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += o;
      }
      s_warp[1][lane] = w;
    }
    __syncthreads();
    const int fincl = f + (warp ? s_warp[1][warp - 1] : 0) + taken;
    if (tid == 0) s_first[0] = taken;
    s_first[tid + 1] = fincl;
    s_cached[tid] = cached;
    if (blockIdx.x == 0 && b < a.B) {
      a.cu[b] = s_cu[tid];
      if (!p.advance) a.lens[b] = len;
    }
    __syncthreads();
    // request of item x: the last i with sums[i] <= x (x is below the chunk's total)
    auto find = [&](const int* sums, int x) {
      int lo = 0, hi = n;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x) lo = mid;
        else hi = mid;
      }
      return lo;
    };
    auto free_block = [&](int i) {  // entry `head + i` of the free list, -1 past its end
      const int64_t at = (int64_t)head + i;
      if (at >= a.n_free) {
        bad = true;
        return -1;
      }
      return a.free_blocks[at];
    };
    for (int t = max(t0, tok) + tid; t < min(t1, s_cu[n]); t += n_thr) {
      const int i = find(s_cu, t);
      const int pos = s_cached[i] + t - s_cu[i], j = pos >> p.shift;
      int entry = -1;
      if (j < a.max_blocks) {
        const int held = (int)(((uint32_t)s_cached[i] + (uint32_t)a.block - 1) >> p.shift);
        entry = j < held ? a.table[(int64_t)(b0 + i) * a.max_blocks + j] : free_block(s_first[i] + j - held);
      }
      const int64_t slot = ((int64_t)entry << p.shift) + (pos & (a.block - 1));
      const bool ok = entry >= 0 && slot <= INT32_MAX;
      bad |= !ok;
      a.slots[t] = ok ? (int)slot : -1;
      a.positions[t] = pos;
    }
    for (int e = taken + blockIdx.x * n_thr + tid; e < s_first[n]; e += gridDim.x * n_thr) {
      const int i = find(s_first, e);
      const int held = (int)(((uint32_t)s_cached[i] + (uint32_t)a.block - 1) >> p.shift);
      a.table[(int64_t)(b0 + i) * a.max_blocks + held + e - s_first[i]] = free_block(e);
    }
    tok = s_cu[n];
    taken = s_first[n];
    __syncthreads();
  }
  for (int t = max(t0, tok) + tid; t < t1; t += n_thr) {  // past the last token (a padded batch)
    a.slots[t] = -1;
    a.positions[t] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.cu[a.B] = tok;
    *a.head_out = (int)min((int64_t)head + taken, (int64_t)max(head, a.n_free));
  }
  if (bad) atomicOr(a.flags, W4A16_DEVICE_KV_RANGE);
}

// Lengths advanced in place, after every CTA of the plan has read them.
__global__ void __launch_bounds__(256) kv_advance_kernel(KvPlanArgs a) {
  for (int b = blockIdx.x * 256 + threadIdx.x; b < a.B; b += gridDim.x * 256)
    a.lens[b] = cached_of(a, a.cached[b]) + a.cu[b + 1] - a.cu[b];
}

// ---- append --------------------------------------------------------------------------------
//
// A run is a maximal stretch of consecutive tokens of the call with
// consecutive slots of one block; one (run, head, K or V) sets the scale of
// one (block, head), so it belongs to one warp (up to kWarpChunks 16-byte
// chunks a lane) or, if it is longer or the block's earlier rows have to be
// re-coded, to the whole CTA.  A CTA looks at `per` consecutive tokens and
// `hg` heads of K or V, a warp taking every eighth (run, head): neighbouring
// heads of a token side by side (its row is read in one stretch), as many
// tokens as give each warp about one run; single heads of 112 tokens where runs
// are long enough for the whole CTA.
// Bytes: 2 in and 1 out per element; a run's rows stay in registers between
// the maximum and the codes.  10k tokens of 8 heads x 128 in blocks of 16 (64 MB):
// 14.7 us, 4.4 TB/s (one head a CTA 17.6); 48 tokens 2.2 us.  No unit is full
// (issue slots 54%, ALU 49%, DRAM 29%): a warp requests one run's rows, waits,
// reduces and stores before the next run's, and 1304 CTAs are 2.1 rounds of the
// 608 that fit.

constexpr int kAppendThreads = 256, kAppendWarps = 8;
constexpr int kMaxPer = 112, kMaxHeads = 8;  // tokens and heads of a CTA
constexpr int kWarpChunks = 8;  // 16-byte chunks a lane holds
constexpr int kCtaChunks = 8;   // a thread holds of a run that the CTA takes; the rest of a longer one (more than
                                // 64 rows of 256) is read again, from L2
constexpr int kMinExp = -64;

__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126..127
__device__ __forceinline__ int exp_of(float s) { return (int)((__float_as_uint(s) >> 23) & 255) - 127; }

// The smallest e >= kMinExp with a <= 448 * 2^e, for a finite bf16 magnitude
// given by its bits: 448 = 1.75 * 2^8, so e is the exponent less 8, one more
// when the significand is above 1.75 (subnormals are below 2^(kMinExp)).
__device__ __forceinline__ int scale_exp(uint32_t bits) {
  const int e = (int)(bits >> 7) - 127 - 8 + ((bits & 127) > 96 ? 1 : 0);
  return max(e, kMinExp);
}

// The larger magnitudes (bf16 bits) of eight values and of those before, a pair a word.
__device__ __forceinline__ uint32_t peak8(const uint4& v, uint32_t m) {
  m = __vmaxu2(m, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu));
  return __vmaxu2(m, __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
}
// (rare) the same without NaN and infinities.
__device__ __forceinline__ uint32_t finite_peak8(const uint4& v, uint32_t m) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = word_of(v, i) & 0x7FFF7FFFu;
    m = __vmaxu2(m, ((w & 0xFFFFu) >= 0x7F80u ? 0u : w & 0xFFFFu) | (w >= 0x7F800000u ? 0u : w & 0xFFFF0000u));
  }
  return m;
}
__device__ __forceinline__ uint32_t larger(uint32_t pair) { return max(pair & 0xFFFFu, pair >> 16); }

// Eight bf16 values times `inv` as e4m3 codes, round to nearest even (one
// rounding: the product with a power of two is exact).  odd: some are not
// finite; NaN and infinities become the NaN code (the conversion alone would
// clamp infinities to 448).
__device__ __forceinline__ uint2 codes8(const uint4& v, float inv, bool odd) {
  float f[8];
  widen8(v, f);
  if (odd) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (isinf(f[i])) f[i] = __uint_as_float(0x7FC00000u);
  }
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(f[2 * i], inv), __fmul_rn(f[2 * i + 1], inv)), __NV_SATFINITE,
                                    __NV_E4M3);
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// Four e4m3 codes at a larger scale: times `ratio` (a power of two below 1).
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    out |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(f.x, ratio), __fmul_rn(f.y, ratio)), __NV_SATFINITE,
                                              __NV_E4M3)
           << (16 * i);
  }
  return out;
}

struct AppendParams {
  KvAppendArgs a;
  int shift;   // log2(block)
  int lpr;     // log2(16-byte chunks of a row): dim = 8 << lpr
  int slots;   // blocks * block
  int per, hg;  // tokens and heads per CTA
};

__global__ void __launch_bounds__(kAppendThreads, 4) kv_append_kernel(AppendParams p) {
  __shared__ int s_slot[1 + kMaxPer + 128];  // from the token before this CTA's on, as far as a run can reach
  __shared__ int2 s_job[kMaxPer * kMaxHeads];  // (token << 16 | head, length) of the runs left to the CTA
  __shared__ int s_jobs;
  __shared__ uint32_t s_peak[kAppendWarps];
  const KvAppendArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h0 = blockIdx.y * p.hg, val = blockIdx.z, t0 = blockIdx.x * p.per;
  const int heads = a.cache.heads, dim = a.cache.dim, block = a.cache.block, lpr = p.lpr;
  const uint16_t* src = val ? a.v : a.k;
  const int hg = min(p.hg, heads - h0);
  const int64_t stride = val ? a.v_stride : a.k_stride;
  uint8_t* codes = val ? a.cache.v : a.cache.k;
  float* scales = val ? a.cache.v_scale : a.cache.k_scale;
  pdl_launch_dependents();
  pdl_wait();

  if (tid == 0) s_jobs = 0;
  for (int i = tid; i < 1 + p.per + block; i += kAppendThreads) {
    const int t = t0 - 1 + i;
    int s = t >= 0 && t < a.T ? a.slots[t] : -1;
    if (s < -1 || s >= p.slots) {
      if (h0 == 0 && val == 0 && i > 0 && i <= p.per) atomicOr(a.flags, W4A16_DEVICE_KV_RANGE);
      s = -1;
    }
    s_slot[i] = s;
  }
  __syncthreads();
  const int* slot_of = s_slot + 1;
  // the tokens that begin a run, 32 at a time; warp w takes every eighth
  int nth = 0;
  for (int i0 = 0; i0 < p.per; i0 += 32) {
    const int i = i0 + lane, s = i < p.per ? slot_of[i] : -1, before = i < p.per ? slot_of[i - 1] : -1;
    const bool joins = before >= 0 && before + 1 == s && (before >> p.shift) == (s >> p.shift);
    const unsigned leaders = __ballot_sync(0xffffffffu, s >= 0 && !joins);
    const int count = __popc(leaders) * hg;
    // (run, head) number nth + q of the CTA, this warp's q
    for (int q = (warp - nth) & (kAppendWarps - 1); q < count; q += kAppendWarps) {
      const int which = q / hg, h = h0 + q - which * hg;
      const int ti = i0 + __fns(leaders, 0, which + 1), slot = slot_of[ti];
      const int blk = slot >> p.shift, off = slot & (block - 1), room = block - off;
      int n = 0;  // tokens of the run
      for (;;) {
        const unsigned go = __ballot_sync(0xffffffffu, n + lane < room && slot_of[ti + n + lane] == slot + n + lane);
        n += go == 0xffffffffu ? 32 : __ffs(~go) - 1;
        if (go != 0xffffffffu) break;
      }
      const int chunks = n << lpr;
      bool job = chunks > 32 * kWarpChunks;
      if (!job) {
        // chunk 32 k + lane: the lane's column stays, its row advances
        const int64_t step = (32 >> lpr) * stride;
        const uint16_t* from = src + (t0 + ti + (lane >> lpr)) * stride + h * dim + 8 * (lane & ((1 << lpr) - 1));
        const int64_t at = (int64_t)blk * heads + h;
        uint4 v[kWarpChunks];
        const float old = off ? scales[at] : 0.f;
#pragma unroll
        for (int k = 0; k < kWarpChunks; ++k) {
          if (32 * k >= chunks) break;
          v[k] = make_uint4(0, 0, 0, 0);
          if (32 * k + lane < chunks) v[k] = ld_nc_v4(from);
          from += step;
        }
        uint32_t pair = 0;
#pragma unroll
        for (int k = 0; k < kWarpChunks; ++k) {
          if (32 * k >= chunks) break;
          pair = peak8(v[k], pair);
        }
        uint32_t peak = __reduce_max_sync(0xffffffffu, larger(pair));
        const bool odd = peak >= 0x7F80u;
        if (odd) {
          pair = 0;
#pragma unroll
          for (int k = 0; k < kWarpChunks; ++k) {
            if (32 * k >= chunks) break;
            pair = finite_peak8(v[k], pair);
          }
          peak = __reduce_max_sync(0xffffffffu, larger(pair));
        }
        int e = scale_exp(peak);
        if (off) {
          const int eo = exp_of(old);
          job = e > eo;  // earlier codes move to a larger scale
          e = max(e, eo);
        }
        if (!job) {
          const float inv = exp2i(-e);
          uint8_t* to = codes + ((at << p.shift) + off) * dim + 8 * lane;
#pragma unroll
          for (int k = 0; k < kWarpChunks; ++k) {
            if (32 * k >= chunks) break;
            if (32 * k + lane < chunks) *reinterpret_cast<uint2*>(to + 256 * k) = codes8(v[k], inv, odd);
          }
          if (off == 0 && lane == 0) scales[at] = exp2i(e);
        }
      }
      if (job && lane == 0) s_job[atomicAdd(&s_jobs, 1)] = make_int2(ti << 16 | h, n);
    }
    nth += count;
  }
  __syncthreads();

  // the CTA's runs, one after another (in no fixed order: they touch different blocks)
  const int jobs = s_jobs;
  for (int w = 0; w < jobs; ++w) {
    const int ti = s_job[w].x >> 16, h = s_job[w].x & 0xFFFF, n = s_job[w].y, slot = slot_of[ti], off = slot & (block - 1);
    const int64_t at = (int64_t)(slot >> p.shift) * heads + h;
    const int64_t step = (kAppendThreads >> lpr) * stride;
    const uint16_t* from = src + (t0 + ti + (tid >> lpr)) * stride + h * dim + 8 * (tid & ((1 << lpr) - 1));
    uint4 v[kCtaChunks];
    uint32_t pair = 0;
    const int chunks = n << lpr;
#pragma unroll
    for (int k = 0; k < kCtaChunks; ++k) {
      if (k * kAppendThreads >= chunks) break;
      v[k] = make_uint4(0, 0, 0, 0);
      if (k * kAppendThreads + tid < chunks) v[k] = ld_nc_v4(from + k * step);
    }
    const float old = off ? scales[at] : 0.f;
#pragma unroll
    for (int k = 0; k < kCtaChunks; ++k) {
      if (k * kAppendThreads >= chunks) break;
      pair = peak8(v[k], pair);
    }
    auto rest = [&](int x) { return ld_nc_v4(from + (x / kAppendThreads) * step); };
    for (int x = kCtaChunks * kAppendThreads + tid; x < chunks; x += kAppendThreads) pair = peak8(rest(x), pair);
    auto over_cta = [&]() {
      const uint32_t m = __reduce_max_sync(0xffffffffu, larger(pair));
      if (lane == 0) s_peak[warp] = m;
      __syncthreads();
      uint32_t all = 0;
#pragma unroll
      for (int i = 0; i < kAppendWarps; ++i) all = max(all, s_peak[i]);
      __syncthreads();
      return all;
    };
    uint32_t peak = over_cta();
    const bool odd = peak >= 0x7F80u;
    if (odd) {
      pair = 0;
#pragma unroll
      for (int k = 0; k < kCtaChunks; ++k) {
        if (k * kAppendThreads >= chunks) break;
        pair = finite_peak8(v[k], pair);
      }
      for (int x = kCtaChunks * kAppendThreads + tid; x < chunks; x += kAppendThreads) pair = finite_peak8(rest(x), pair);
      peak = over_cta();
    }
    int e = scale_exp(peak);
    uint8_t* base = codes + (at << p.shift) * dim;
    if (off) {
      const int eo = exp_of(old);
      if (e > eo) {
        const float ratio = exp2i(max(eo - e, -126));
        uint4* q = reinterpret_cast<uint4*>(base);
        for (int x = tid; x < off << (lpr - 1); x += kAppendThreads) {
          uint4 w4 = q[x];
          w4.x = recode4(w4.x, ratio);
          w4.y = recode4(w4.y, ratio);
          w4.z = recode4(w4.z, ratio);
          w4.w = recode4(w4.w, ratio);
          q[x] = w4;
        }
      }
      e = max(e, eo);
    }
    const float inv = exp2i(-e);
#pragma unroll
    for (int k = 0; k < kCtaChunks; ++k) {
      if (k * kAppendThreads >= chunks) break;
      const int x = k * kAppendThreads + tid;
      if (x < chunks) *reinterpret_cast<uint2*>(base + off * dim + 8 * x) = codes8(v[k], inv, odd);
    }
    for (int x = kCtaChunks * kAppendThreads + tid; x < chunks; x += kAppendThreads)
      *reinterpret_cast<uint2*>(base + off * dim + 8 * x) = codes8(rest(x), inv, odd);
    __syncthreads();  // every thread has read the old scale (and s_peak)
    if (tid == 0) scales[at] = exp2i(e);
  }
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs& a, int pdl, cudaStream_t s) {
  PlanParams p{a, __builtin_ctz((unsigned)a.block), 0};
  // a thread per request and per token up to the CTA's size, at least four warps
  int threads = a.B > a.T ? a.B : a.T;
  threads = threads < 128 ? 128 : threads > kPlanThreads ? kPlanThreads : (threads + 31) / 32 * 32;
  const int grid = a.T > 0 ? (a.T + kPlanTokens - 1) / kPlanTokens : 1;
  // One CTA reads its requests' lengths before it writes them; where several read them all, a second launch advances
  // them when they are done (333 prompt chunks 1.1 us more than with lens apart).
  p.advance = grid > 1 && a.lens == a.cached;
  void* args[] = {&p};
  cudaError_t e = launch((const void*)kv_plan_kernel, dim3((unsigned)grid), threads, args, pdl, s);
  if (e != cudaSuccess || !p.advance) return e;
  void* advance[] = {&p.a};
  const int ctas = a.B / 256 + 1;
  return launch((const void*)kv_advance_kernel, dim3((unsigned)(ctas < 608 ? ctas : 608)), 256, advance, 0, s);
}

cudaError_t launch_kv_append(const KvAppendArgs& a, int pdl, cudaStream_t s) {
  AppendParams p{a, __builtin_ctz((unsigned)a.cache.block), __builtin_ctz((unsigned)a.cache.dim) - 3,
                 a.cache.blocks * a.cache.block, 0, 0};
  const int heads = a.cache.heads;
  p.hg = heads < kMaxHeads ? heads : kMaxHeads;
  // Which tokens make runs is known on the device only, so the rule goes by their number: few are taken for runs of one
  // or a few (decode, verify), many for runs of a block, which a warp holds up to 2048 values of.  Measured as (first /
  // second / third form), us, 8 heads of 128.  Few: 48 single tokens 2.4 / 17 / 7.6; 200 x 5 5.8 / 7.2 / 7.0; but one
  // prompt of 1024, which the rule takes for short runs, 5.9 / 3.9 / 4.8 in blocks of 16, 13 / 9.6 / 5.4 of 64, 17 / 13 /
  // 4.9 of 128 (2 heads of 256 in blocks of 64: 5.5 / 7.8 / 5.2).  Many: a prompt of 10k in blocks of 16 34 / 9.9 / 11.8; of
  // 64 44 / 19 / 15; of 128 47 / 28 / 13; 2 heads of 256, blocks of 64, 14 / 14 / 9.0.  4000 single tokens 28 / 25 / 23.
  if (a.T < 2048) {
    p.per = kAppendWarps / p.hg;
  } else if (a.cache.block * a.cache.dim <= 32 * kWarpChunks * 8) {
    p.per = a.cache.block * (kAppendWarps / p.hg);
    if (p.per > kMaxPer) p.per = kMaxPer;
  } else {
    p.per = kMaxPer;
    p.hg = 1;
  }
  void* args[] = {&p};
  return launch((const void*)kv_append_kernel,
                dim3((unsigned)((a.T + p.per - 1) / p.per), (unsigned)((heads + p.hg - 1) / p.hg), 2), kAppendThreads, args, pdl, s);
}

}  // namespace w4a16
