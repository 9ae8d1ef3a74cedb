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
// e4m3's range whatever the blocks' scales; the row sum takes the weight
// without vs, over all of 2^-64 to 2^120 (an exponential of z - max, from which
// the product's weight follows by a power of two; taken the other way round, it
// was lost where vs was 2^134 below another's).
//
// Split.  A tile is 128 tokens at a fixed position; a group eight tiles.  A
// tile gives (maximum m, sum l, O) per row; a group folds its tiles in order, a
// row joins its groups pairwise as a binary tree.  All tiles of the call form
// one line (request, row tile, key head, tile) cut into equal ranges, one per
// CTA: a group that lies in one range is folded in registers, one that a cut
// divides is written tile by tile, and the CTA that completes it (a counter)
// folds the tiles with the same operations at its end.  So the cut follows the
// load and the bits do not.  Rows of one group are finished there; several
// groups are joined by kv_combine_kernel.
//
// Bound: HBM for a few rows a key head.  64 requests of 1 x 4 rows to 16k tokens
// of 2 heads x 256: 87 us, 5.67 TB/s; one of 131k tokens 35 us, 3.9 TB/s, where
// set-up (2 us), the first copies (2 us), the groups that a cut divides (2 to 5
// us) and the join (4 us) weigh more.  A CTA has two to five tiles (64 KB each with
// heads of 256) in flight.  From 16 rows on the softmax warps' instructions and
// the chain of waits and issues in the MMA warp, each about 2000 clocks a tile of
// 32 rows (3 prompt chunks of 300 over 6k tokens, 28/4 heads of 128: 198 us, 229
// TFLOP/s; a prompt of 8192 from an empty cache, 32/8 of 128, 2.0 ms, 271; S and O
// issued by two warps: 208 instead of 194 of the chunks).
//
// CTA: 4 NG + 4 NG + 3 warps (NG groups of R query rows).
//   softmax warps  a thread per token: scores from TMEM, mask, maximum,
//                  weights into shared memory, row sums
//   fold warps     a thread per output column (TMEM lane): O from TMEM into the
//                  running accumulators, partial results out
//   one warp       work list: descriptors with block ids and scales, up to eight
//                  tiles ahead
//   one warp       copies: TMA of K and V blocks as slots become free, queries
//   one warp       tensor memory, MMA issue
// A tile passes load -> S -> softmax -> O -> fold; softmax of one tile, fold of
// the one before and the copies of the next run side by side.
// Every wait is bounded: one that gives up raises W4A16_DEVICE_TIMEOUT, the
// roles leave their loops, copies and MMAs in flight are waited for (bounded)
// and the tensor memory is freed.
#include <cuda.h>
#include <cuda_fp8.h>
#include <cudaTypedefs.h>

#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "kv.cuh"
#include "kv_line.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace w4a16 {
namespace {

using namespace ptx;

constexpr int kGroupTiles = 8;  // tiles per group
constexpr int kGroupTokens = kTile * kGroupTiles;
constexpr int kDescs = 8;       // tile descriptors in flight
constexpr int kRing = 4;        // row sums and weights' barriers: softmax may be two tiles ahead of the fold
constexpr int kSms = 152;
constexpr uint32_t kTries = 1u << 18;  // of a wait: about a second (a limit in the parameters: prompt chunks 200 -> 213 us)
constexpr float kLog2e = 1.4426950408889634f;

// flags of a tile descriptor
constexpr int kNewSeg = 1;     // another (request, row tile, head) than the tile before
constexpr int kEnd = 2;        // no tile: the CTA's range is empty
constexpr int kFix = 4;        // some token of the tile is not seen by some row, or its block is not in the cache
constexpr int kGroupBegin = 8; // first tile of a group folded here
constexpr int kGroupEnd = 16;  // its last tile
constexpr int kPart = 32;      // the result goes to a slot for parts of divided groups
constexpr int kDirect = 64;    // the segment is this one group, and whole
constexpr int kLastPart = 128; // the range's last part of a divided group
constexpr int kTail = 256;     // ... which goes on in the next range (else it began in an earlier one)
constexpr int kNextSeg = 512;  // the range's next tile begins another segment
constexpr int kFinal = 1024;   // the range's last tile

struct Desc {
  int flags, h, j0, tile;      // key head, first token of the row tile in its request
  int base, fresh, c0, at;     // tokens before the step, new tokens, first row, group slot (kPart: slot for parts)
  int id[8];                   // block ids; -1: not needed or not in the cache
  float ks[8], vs[8];          // scales of the tile's blocks (0: no such block)
};
static_assert(sizeof(Desc) % 16 == 0, "16-byte rows");

// A group that a cut divides, as a CTA's end needs it.
struct CutGroup {
  int owner, count, mine;         // CTA of its first tile, its tiles, those in this range
  int c0, j0, h, toks;            // rows: first of the request, first token of the row tile, key head, tokens
  int gi, single;                 // group slot; the segment's only group
  int parts, slot[kGroupTiles];   // its parts in order: the first range's fold, then tiles
};

// RP rows of a row tile (query tokens x heads of a group), R to a softmax warp
// group: more rows a thread spread its fixed work per tile (waits, exchange of
// maxima) over more of them, as far as registers go (32 rows in groups of 8:
// 240 instead of 231 us).  Row tiles of 4, 8, 12, 16, 24 and 32: without 12 and
// 24, 40 x 12 rows take 25.5 instead of 24.2 and 16 x 20 rows 68.6 instead of
// 62.1; without 4, 32 x 4 rows 53.5 instead of 52.9.
// CTAs per SM and K/V slots (128 tokens each): as many bytes in flight as the
// shared memory holds, in two CTAs where registers leave room and both have
// work side by side.  One CTA instead: 4 rows of 128 61.0 (two: 52.9), 12 rows of
// 128 61.1 (56.3), 16 rows of 64 59.0 (48.5); but 16 rows of 128 27.1 (28.1).
template <int D, int RP>
struct Geo {
  static constexpr int R = RP == 24 ? 12 : RP < 16 ? RP : 16;
  static constexpr int kGroups = RP / R;
  static constexpr int kThreads = 256 * kGroups + 96;
  static constexpr int kCols = (2 * RP + 15) / 16 * 16;        // columns of S and O: first and second terms
  static constexpr int kPanels = D <= 128 ? 1 : D / 128;       // 128-byte column panels of K and V
  static constexpr int kRowB = D <= 128 ? D : 128;             // bytes of a panel's row
  static constexpr int kPanelBytes = kTile * kRowB;
  static constexpr int kSlot = kTile * D;
  static constexpr int kQ = kPanels * kCols * 128;
  // a segment's query rows as they come, ahead of its turn, where the slots leave room (32 rows of 128: 196.5 us, read
  // by the softmax warps themselves 198.6)
  static constexpr int kStage = D == 256 && RP == 24 ? 0 : RP * D * 2;
  static constexpr int kP = kTile * kCols;
  static constexpr int kCtas = RP <= 8 || (D == 128 && RP == 12) || (D == 64 && RP <= 16) ? 2 : 1;
  static constexpr int kSlots = D == 256 ? (RP <= 8 ? 3 : RP <= 24 ? 6 : 5)
                                : D == 128 ? (RP <= 8 ? 6 : RP == 12 ? 5 : 10) : RP <= 16 ? 10 : 12;
  static constexpr int kBars = 2 * kSlots + 3 * kDescs + 2 + kRing + 4 + 5 + kGroups;
  // rows (bits) of a tile that see a NaN in a thread's columns
  using Marks = std::conditional_t<(kPanels * R > 16), uint32_t, uint16_t>;
  // warps' maxima (two tiles), sums (kRing tiles x four warps), maxima (kRing), fold factors per warp, row factors and
  // limits; NaN marks (kRing tiles)
  static constexpr int kRowData = RP * 4 * (2 * 4 + kRing * 4 + kRing + 2 * 4 + 2 * 3) + kRing * 128 * kGroups * (int)sizeof(Marks);
  static constexpr int kSmem = kSlots * kSlot + kQ + 2 * kP + kStage + kDescs * (int)sizeof(Desc) + kRowData + 8 * kBars + 48 + 2 * (int)sizeof(CutGroup);
  static constexpr int kTmemCols = 2 * kCols * (1 + kPanels);  // S twice, O twice
  static constexpr uint32_t kTmem = kTmemCols <= 64 ? 64 : kTmemCols <= 128 ? 128 : kTmemCols <= 256 ? 256 : 512;
  static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
  static_assert(kCtas * kTmem <= 512, "tensor memory of an SM");
};

struct Params : Line {
  const uint16_t* q;
  int64_t q_stride;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  uint16_t* out;
  int q_heads, heads, G;  // G query heads per key head
  int blocks, shift, max_blocks;
  float qk_scale;  // scale * log2(e)
  int gmax;        // group slots per row
  int grid;
  int seg_cost;    // positions before a segment's first tile
  int t_slots;     // slots for parts per CTA
  // workspace
  float* g_acc;  // [gmax][T][q_heads][D]
  float2* g_ml;  // [gmax][T][q_heads]
  float* t_acc;  // [grid][t_slots][RP][D]
  float2* t_ml;  // [grid][t_slots][RP]
  int* refused;   // [1] the step's offsets step back (written by every call)
  int arrivals;  // that complete the first CTA's first slot: 1 (see KvAttentionArgs::fault_wait)
  int* counters;  // [grid] tiles done of divided groups, by the CTA of the first; zero between calls
  int* flags;
};

struct Maps {
  CUtensorMap k, v;
};

// ---- shared pieces -----------------------------------------------------------------------------

__device__ __forceinline__ float ex2(float x) {  // 2^x; results below 2^-126 are 0
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two fp32 operations an instruction, each rounded as by itself.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{ .reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7}; fma.rn.f32x2 d, a, b, c; "
      "mov.b64 {%0, %1}, d; }"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{ .reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d; }"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{ .reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mul.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d; }"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// a, b as hi + lo / 16 (each two e4m3 codes, a in the low byte), in fp32: exact for bf16 values in range
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const float2 h = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi, __NV_E4M3)));
  lo = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(__fsub_rn(a, h.x), 16.f), __fmul_rn(__fsub_rn(b, h.y), 16.f)),
                                __NV_SATFINITE, __NV_E4M3);
}

// The same for weights, two at a time in fp16: rounding to 11 bits first
// (2^-11) on top of the two terms' 2^-9 stays below bf16's 2^-8.
__device__ __forceinline__ void split2h(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 x = __floats2half2_rn(a, b);
  hi = __nv_cvt_halfraw2_to_fp8x2((__half2_raw)x, __NV_SATFINITE, __NV_E4M3);
  const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi, __NV_E4M3));
  lo = __nv_cvt_halfraw2_to_fp8x2((__half2_raw)__hmul2(__hsub2(x, h), __float2half2_rn(16.f)), __NV_SATFINITE, __NV_E4M3);
}

// One step of a fold: the running (m, l) takes in (mt, lt); al and be are
// what the running and the new accumulators are multiplied by.  An empty
// side (m = -inf) leaves the other as it is, bit for bit.  Each factor is a
// square, and the sum takes its root twice: below 2^-126 the accumulators it
// stands for vanish beside the others, but the sum, which does not hold the V
// scales that m holds, may be as large as 2^80 then.
__device__ __forceinline__ void fold_ml(float& m, float& l, float mt, float lt, float& al, float& be) {
  const float top = fmaxf(m, mt), ref = top == -INFINITY ? 0.f : top;
  const float a = ex2(__fmul_rn(m - ref, 0.5f)), b = ex2(__fmul_rn(mt - ref, 0.5f));
  al = __fmul_rn(a, a);
  be = __fmul_rn(b, b);
  l = __fmaf_rn(__fmul_rn(l, a), a, __fmul_rn(__fmul_rn(lt, b), b));
  m = top;
}

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[N]) {
  if constexpr (N == 8) {
    tmem_ld8(addr, v);
  } else {
#pragma unroll
    for (int i = 0; i + 16 <= N; i += 16) {
      float t[16];
      tmem_ld16(addr + i, t);
#pragma unroll
      for (int k = 0; k < 16; ++k) v[i + k] = t[k];
    }
    if constexpr (N % 16 == 8) {
      float t[8];
      tmem_ld8(addr + N - 8, t);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[N - 8 + k] = t[k];
    }
  }
}

// ---- joining a row's groups --------------------------------------------------------------------

struct State {
  float m, l;
  float4 a;
};

__device__ __forceinline__ State empty_state() { return State{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)}; }

__device__ __forceinline__ void fold_state(State& s, const State& o) {
  float al, be;
  fold_ml(s.m, s.l, o.m, o.l, al, be);
  s.a.x = __fmaf_rn(s.a.x, al, __fmul_rn(o.a.x, be));
  s.a.y = __fmaf_rn(s.a.y, al, __fmul_rn(o.a.y, be));
  s.a.z = __fmaf_rn(s.a.z, al, __fmul_rn(o.a.z, be));
  s.a.w = __fmaf_rn(s.a.w, al, __fmul_rn(o.a.w, be));
}

__device__ __forceinline__ void write_out(const Params& p, int64_t at, const State& s) {  // four columns
  const float f = s.l != 0.f ? __frcp_rn(s.l) : 0.f;  // (NaN: stays)
  uint2 w;
  w.x = (uint32_t)f32_to_bf16_bits(__fmul_rn(s.a.x, f)) | (uint32_t)f32_to_bf16_bits(__fmul_rn(s.a.y, f)) << 16;
  w.y = (uint32_t)f32_to_bf16_bits(__fmul_rn(s.a.z, f)) | (uint32_t)f32_to_bf16_bits(__fmul_rn(s.a.w, f)) << 16;
  *reinterpret_cast<uint2*>(p.out + at) = w;
}

// The groups of a row that the call computed: n of them, the first one's
// result at at0 (rows of D floats), `stride` rows from one to the next.
template <int D>
struct RowGroups {
  int64_t at0, stride;
  int n;
  __device__ __forceinline__ RowGroups(const Params& p, const Req& r, int j, int hq) {
    const int pos = r.base + j;
    const int ga = p.window > 0 ? max(0, pos - p.window + 1) / kGroupTokens : 0;
    n = pos / kGroupTokens - ga + 1;
    at0 = ((int64_t)(ga - first_tile(p, r, 0) / kGroupTiles) * p.T + r.c0 + j) * p.q_heads + hq;
    stride = (int64_t)p.T * p.q_heads;
  }
  __device__ __forceinline__ State group(const Params& p, int i, int col) const {
    if (i >= n) return empty_state();
    const int64_t at = at0 + i * stride;
    const float2 ml = p.g_ml[at];
    return State{ml.x, ml.y, *reinterpret_cast<const float4*>(p.g_acc + at * D + col)};
  }
  // The join of groups i .. i + m - 1 (m a power of two; those from n on are
  // empty), four requested together: a binary counter of joined pairs.
  __device__ __forceinline__ State tree(const Params& p, int i, int m, int col) const {
    if (m < 4) {
      State s = group(p, i, col);
      if (m == 2) fold_state(s, group(p, i + 1, col));
      return s;
    }
    State level[20];  // (local memory: only rows of more than four groups a set come here)
    const int fours = (min(i + m, n) - i + 3) / 4;
    if (fours == 1) return four(p, i, col);
#pragma unroll 1
    for (int f = 0; f < fours; ++f) {
      State s = four(p, i + 4 * f, col);
      int k = 0;
      for (; (f >> k) & 1; ++k) {
        State left = level[k];
        fold_state(left, s);
        s = left;
      }
      level[k] = s;
    }
    State s = level[__ffs(fours) - 1];  // what is left, from the right
#pragma unroll 1
    for (int k = __ffs(fours); fours >> k; ++k)
      if ((fours >> k) & 1) {
        State left = level[k];
        fold_state(left, s);
        s = left;
      }
    return s;
  }
  __device__ __forceinline__ State four(const Params& p, int i, int col) const {
    State st[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) st[k] = group(p, i + k, col);
    fold_state(st[0], st[1]);
    fold_state(st[2], st[3]);
    fold_state(st[0], st[2]);
    return st[0];
  }
};

// The last b with cu[b] <= t.
__device__ __forceinline__ int find_request(const int32_t* cu, int B, int t) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---- the kernel -----------------------------------------------------------------------------------

template <int D, int RP>
__global__ void __launch_bounds__(Geo<D, RP>::kThreads, Geo<D, RP>::kCtas)
    kv_attention_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  using X = Geo<D, RP>;
  constexpr int NS = X::kSlots, NP = X::kPanels, NG = X::kGroups, R = X::R, C = X::kCols, ND = kDescs;
  constexpr int W_FOLD = 4 * NG, W_LIST = 8 * NG, W_LOAD = 8 * NG + 1, W_MMA = 8 * NG + 2;
  extern __shared__ __align__(1024) uint8_t base[];
  uint8_t* q_mem = base + NS * X::kSlot;
  uint8_t* p_mem = q_mem + X::kQ;
  uint8_t* stage = p_mem + 2 * X::kP;
  Desc* descs = reinterpret_cast<Desc*>(stage + X::kStage);
  float* s_max = reinterpret_cast<float*>(descs + ND);               // [2][4 warps][RP]
  float* s_sum = s_max + 2 * 4 * RP;                                 // [kRing][4 warps][RP]
  float* s_top = s_sum + kRing * 4 * RP;                             // [kRing][RP]
  float2* s_ab = reinterpret_cast<float2*>(s_top + kRing * RP);      // [4 warps][RP]
  float* s_qf2 = reinterpret_cast<float*>(s_ab + 4 * RP);            // [2][RP] score factor of a row, by segment
  int2* s_lim2 = reinterpret_cast<int2*>(s_qf2 + 2 * RP);            // [2][RP] first and last token a row sees
  auto* s_taint = reinterpret_cast<typename X::Marks*>(s_lim2 + 2 * RP);  // [kRing][128 NG]
  uint64_t* bar_mem = reinterpret_cast<uint64_t*>(s_taint + kRing * 128 * NG);
  const uint32_t slots = smem_u32(base), q_s = smem_u32(q_mem), p_s = smem_u32(p_mem), bars = smem_u32(bar_mem);
  auto full = [&](int i) { return bars + 8u * i; };                  // slot: copies landed
  auto empty = [&](int i) { return bars + 8u * (NS + i); };          // slot: MMAs done with it
  auto d_full = [&](int i) { return bars + 8u * (2 * NS + i); };     // descriptor written
  auto d_free = [&](int i) { return bars + 8u * (2 * NS + ND + i); };
  auto d_scales = [&](int i) { return bars + 8u * (2 * NS + 2 * ND + i); };  // its scales landed
  const uint32_t bars2 = bars + 8u * (2 * NS + 3 * ND);
  auto s_full = [&](int i) { return bars2 + 8u * i; };
  auto o_full = [&](int i) { return bars2 + 8u * (2 + i); };
  auto o_free = [&](int i) { return bars2 + 8u * (4 + i); };
  auto p_full = [&](int i) { return bars2 + 8u * (6 + i); };         // [kRing] weights, sums and maxima written
  const uint32_t q_full = bars2 + 8u * (6 + kRing), drained = q_full + 8, all_sync = q_full + 16;
  const uint32_t st_full = q_full + 24, st_free = q_full + 32;       // staged query rows
  auto grp_sync = [&](int g) { return q_full + 40 + 8u * g; };       // the four softmax warps of a group
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bar_mem + X::kBars);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  volatile int* s_nan = reinterpret_cast<volatile int*>(s_tmem + 2);  // [kRing] 1 + a tile whose marks are in s_taint
  volatile int* s_last = reinterpret_cast<volatile int*>(s_tmem + 6);  // [2] this CTA completed the divided group
  volatile int* s_rest = reinterpret_cast<volatile int*>(s_tmem + 8);  // rows of no (valid) request, all tiles
  CutGroup* s_cut = reinterpret_cast<CutGroup*>(s_tmem + 12);          // [2] at the range's beginning, at its end
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  auto wait = [](uint32_t bar, uint32_t parity) { return mbar_wait_warp(bar, parity, kTries); };
  auto give_up = [&]() {
    atomicOr(p.flags, W4A16_DEVICE_TIMEOUT);
    *s_abort = 1;
  };

  // ---- set-up; meanwhile the listing warp finds the CTA's range of the line ----
  const int nb = kTile >> p.shift, block = 1 << p.shift;  // blocks per tile
  bool bad = false;
  int total = 0, beg = 0, end = 0, b0 = 0;
  Req mine{0, 0, 0}, r{0, 0, 0};  // the listing warp: this lane's request of 32, and the current one
  int b = 0, rt = 0, h = 0, tile = 0, t_first = 0, t_last = -1;
  int seg0 = 0;  // position of the segment's first tile
  int id = -2;
  int loads = 0;  // slots requested
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
  // block id of this lane for a tile: -2 not needed, -1 (or any bad id) not in the cache
  auto load_id = [&]() {
    const int lo = p.window > 0 ? max(0, r.base + rt * p.TQ - p.window + 1) : 0;
    const int hi = r.base + min((rt + 1) * p.TQ, r.fresh) - 1;
    const int j = tile * nb + lane;
    if (lane >= nb || j * block + (block - 1) < lo || j * block > hi) return -2;  // (below 2^31 in every tile)
    return j < p.max_blocks ? p.table[(int64_t)b * p.max_blocks + j] : -1;
  };
  if (warp == W_LOAD) {
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.k) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.v) : "memory");
    }
  } else if (warp == W_LIST) {
    pdl_wait();
    int mine_end = 0;         // inclusive prefix of this lane's request
    int rows = 0;             // of valid requests
    bool back = false;
    auto scan = [&](const RawReq& w) {  // 32 requests; their inclusive prefix of tiles after `total`
      mine = check_req(p, w, &bad);
      const int rts = row_tiles(p, mine);
      int n = rts > 0 ? (tiles_before(p, mine, rts) + p.seg_cost * rts) * p.heads : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, n, d);
        if (lane >= d) n += o;
      }
      mine_end = total + n;
    };
    int ends = 0;  // lane i: tiles up to the end of the i-th 32 requests (the first 1024)
    RawReq ahead(p, lane);
    for (; b0 < p.B; b0 += 32) {
      const RawReq w = ahead;
      if (b0 + 32 < p.B) ahead = RawReq(p, b0 + 32 + lane);
      back |= steps_back(w);
      scan(w);
      total = __shfl_sync(0xffffffffu, mine_end, 31);
      rows += mine.fresh;
      if (b0 == 32 * lane) ends = total;
    }
    rows = __reduce_add_sync(0xffffffffu, rows);
    const bool refused = __any_sync(0xffffffffu, back);
    if (refused) rows = total = 0;
    if (lane == 0) {
      s_rest[0] = p.T - rows;
      s_rest[1] = total;
      if (blockIdx.x == 0) *p.refused = refused;
    }
    if (bad && blockIdx.x == 0) atomicOr(p.flags, W4A16_DEVICE_KV_RANGE);
    const Cut cut(total, p.grid);
    beg = cut.begin(blockIdx.x);
    end = cut.begin(blockIdx.x + 1);
    // the request of `beg`
    total = 0;
    b0 = 0;
    if (p.B > 32) {
      const unsigned after = __ballot_sync(0xffffffffu, 32 * lane < p.B && ends > beg);
      const int skip = after ? __ffs(after) - 1 : 32;
      if (skip > 0) total = __shfl_sync(0xffffffffu, ends, skip - 1);
      for (b0 = 32 * skip; b0 < p.B; b0 += 32) {
        scan(RawReq(p, b0 + lane));
        const int e = __shfl_sync(0xffffffffu, mine_end, 31);
        if (e > beg) break;
        total = e;
      }
    }
    if (beg < end) {
      const unsigned past = __ballot_sync(0xffffffffu, mine_end > beg);
      const int bl = __ffs(past) - 1;
      const int before = __shfl_sync(0xffffffffu, mine_end, max(bl - 1, 0));
      take(bl);
      int off = beg - (bl > 0 ? before : total);
      // its row tile: a lane looks at every step-th
      int skipped = 0;  // tiles before it
      for (int hi = row_tiles(p, r); hi - rt > 1;) {
        const int step = (hi - rt + 31) / 32, mid = rt + lane * step;
        const int first = mid < hi ? (tiles_before(p, r, mid) + p.seg_cost * mid) * p.heads : 0;
        const int le = __popc(__ballot_sync(0xffffffffu, mid < hi && first <= off)) - 1;
        skipped = __shfl_sync(0xffffffffu, first, le);
        rt += le * step;
        hi = min(hi, rt + step);
      }
      off -= skipped;
      enter();
      const int n = p.seg_cost + t_last - t_first + 1;
      h = off / n;
      off -= h * n + p.seg_cost;  // (below 0: in the segment's positions before its first tile)
      tile = t_first + max(off, 0);
      seg0 = beg - off;
      id = load_id();
    }
  } else if (warp == W_MMA) {
    tmem_alloc(smem_u32(s_tmem), X::kTmem);
    tmem_relinquish();
  } else if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full(i), i == 0 && blockIdx.x == 0 ? p.arrivals : 1);
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < ND; ++i) {
      mbar_init(d_full(i), 1);
      mbar_init(d_scales(i), 32);
      mbar_init(d_free(i), 8 * NG + 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(o_full(i), 1);
      mbar_init(o_free(i), 4 * NG);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(p_full(i), 4 * NG);
      s_nan[i] = 0;
    }
    mbar_init(q_full, 4 * NG);
    mbar_init(drained, 1);
    mbar_init(all_sync, 4 * NG);
    mbar_init(st_full, 1);
    mbar_init(st_free, 4 * NG);
    for (int i = 0; i < NG; ++i) mbar_init(grp_sync(i), 4);
    *s_abort = 0;
    s_last[0] = s_last[1] = 0;
    fence_barrier_init();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *s_tmem;
  const uint32_t s_col = tmem, o_col = tmem + 2 * C;  // S: two tiles of C columns; O: two tiles of NP panels of C

  if (warp == W_LIST) {
    // (after the wait, so that what the next kernel reads of this call's inputs is there when it starts; and after the
    // set-up: a next kernel's CTA must not hold tensor memory that a CTA it waits for has yet to get)
    pdl_launch_dependents();
    // ---- work list ----
    bool fresh_seg = true, ok = true;
    const Cut cut(s_rest[1], p.grid);
    int x = beg < end ? seg0 + tile - t_first : end, t = 0, next;
    for (; x < end; x = next, ++t) {
      const int ds = t % ND;
      const bool same = tile < t_last;
      next = same ? x + 1 : x + 1 + p.seg_cost;
      const int g_lo = max(seg0, x - tile % kGroupTiles), g_hi = min(seg0 + t_last - t_first, x - tile % kGroupTiles + kGroupTiles - 1);
      const int j0 = rt * p.TQ, toks = min(p.TQ, r.fresh - j0), pos0 = r.base + j0, pos1 = pos0 + toks - 1;
      // the group's first tile begins a fold, its last ends it; a cut ends it, too, and after one every tile is by itself
      const bool late = g_lo < beg, part = late || g_hi >= end;
      int fl = (fresh_seg ? kNewSeg : 0) | (part ? kPart : 0) | (x == g_lo || late ? kGroupBegin : 0) |
               (x == g_hi || x + 1 == end || late ? kGroupEnd : 0) |
               (part && (x == g_hi || x + 1 == end) ? kLastPart : 0) | (late ? 0 : kTail) |
               (next >= end ? kFinal : same ? 0 : kNextSeg);
      const int at = !part ? tile / kGroupTiles - first_tile(p, r, 0) / kGroupTiles
                           : (int)blockIdx.x * p.t_slots + (late ? x - beg : p.t_slots - 1);
      const bool single = t_first / kGroupTiles == t_last / kGroupTiles;
      if (!(fl & kPart) && single) fl |= kDirect;
      if (fl & kLastPart) {  // for the CTA's end
        CutGroup& c = s_cut[!late];
        const int owner = late ? cut.owner(g_lo) : (int)blockIdx.x;
        const int rest = cut.begin(owner + 1);  // the first tile after the first range
        if (lane == 0) {
          c.owner = owner, c.count = g_hi - g_lo + 1, c.mine = min(end, g_hi + 1) - max(beg, g_lo);
          c.c0 = r.c0, c.j0 = j0, c.h = h, c.toks = toks;
          c.gi = tile / kGroupTiles - first_tile(p, r, 0) / kGroupTiles, c.single = single;
          c.parts = g_hi - rest + 2;
        }
        if (lane < kGroupTiles && rest + lane - 1 <= g_hi) {
          const int y = rest + lane - 1, own = lane ? cut.owner(y) : owner;
          c.slot[lane] = own * p.t_slots + (lane ? y - cut.begin(own) : p.t_slots - 1);
        }
        __syncwarp();
      }
      const bool valid = id >= 0 && id < p.blocks;
      const unsigned need = __ballot_sync(0xffffffffu, id != -2), have = __ballot_sync(0xffffffffu, valid);
      if (need != have || tile * kTile + kTile - 1 > pos0 || (p.window > 0 && tile * kTile < pos1 - p.window + 1)) fl |= kFix;
      if (t >= ND && !(ok = wait(d_free(ds), ((t / ND) - 1) & 1))) break;
      Desc& de = descs[ds];
      if (lane == 0) {
        *reinterpret_cast<int4*>(&de.flags) = make_int4(fl, h, j0, tile);
        *reinterpret_cast<int4*>(&de.base) = make_int4(r.base, r.fresh, r.c0, at);
        if (need != have) atomicOr(p.flags, W4A16_DEVICE_KV_RANGE);
      }
      if (lane < 8) de.id[lane] = valid ? id : -1;
      if (lane < nb) {
        if (valid) {
          cp_async4(smem_u32(&de.ks[lane]), p.k_scale + (int64_t)id * p.heads + h);
          cp_async4(smem_u32(&de.vs[lane]), p.v_scale + (int64_t)id * p.heads + h);
        } else {
          de.ks[lane] = 0.f;
          de.vs[lane] = 0.f;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(d_full(ds));
      cp_async_arrive(d_scales(ds));
      // the next tile
      if (next < end) {
        if (same) {
          ++tile;
        } else {
          seg0 = next;
          if (++h == p.heads) {
            h = 0;
            if (++rt == row_tiles(p, r)) {
              rt = 0;
              int bl = b - b0;
              for (;;) {  // the next request with new tokens (there is one: the line goes on)
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
        id = load_id();
      }
      fresh_seg = !same;
    }
    if (t == 0 && lane == 0) {  // no tile
      descs[0].flags = kEnd;
      mbar_arrive(d_full(0));
    }
    if (!ok && lane == 0) give_up();
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == W_LOAD) {
    // ---- copies ----
    bool ok = true;
    int fl = 0, staged = 0;  // segments whose query rows were requested
    for (int t = 0; ok && !(fl & kFinal); ++t) {
      const int ds = t % ND;
      if (!(ok = wait(d_full(ds), (t / ND) & 1))) break;
      const Desc& de = descs[ds];
      const int4 dd = *reinterpret_cast<const int4*>(&de.flags), dx = *reinterpret_cast<const int4*>(&de.base);
      fl = dd.x;
      if (fl & kEnd) break;
      // lane (block, panel): one copy each of K, then of V
      const int blk = lane / NP, panel = lane % NP;
      const int my_id = blk < nb ? de.id[blk & 7] : -1;
      const int row = (my_id * p.heads + dd.y) << p.shift;
      const int copies = __popc(__ballot_sync(0xffffffffu, my_id >= 0));  // of kRowB bytes x block rows
      if (lane == 0) mbar_arrive(d_free(ds));
      const int toks = min(p.TQ, dx.y - dd.z);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int slot = loads % NS;
        if (loads >= NS && !(ok = wait(empty(slot), ((loads / NS) - 1) & 1))) break;
        if (lane == 0) mbar_expect_tx(full(slot), (uint32_t)(copies * block * X::kRowB));
        __syncwarp();
        if (my_id >= 0)
          tma_load_2d(slots + slot * X::kSlot + panel * X::kPanelBytes + blk * block * X::kRowB, kv ? &maps.v : &maps.k,
                      panel * 128, row, full(slot));
        ++loads;
        if (X::kStage > 0 && kv == 0 && (fl & kNewSeg)) {  // the segment's query rows, a copy per token
          if (staged > 0 && !(ok = wait(st_free, (staged - 1) & 1))) break;
          const uint32_t bytes = (uint32_t)(p.G * D * 2);
          if (lane == 0) mbar_expect_tx(st_full, toks * bytes);
          __syncwarp();
          if (lane < toks)
            bulk_load(smem_u32(stage) + lane * bytes, p.q + (int64_t)(dx.z + dd.z + lane) * p.q_stride + (int64_t)dd.y * p.G * D,
                      bytes, st_full, policy_evict_first());
          ++staged;
        }
      }
    }
    if (!ok && lane == 0) give_up();
    if (staged > 0) wait(st_full, (staged - 1) & 1);  // (nobody else may be left to wait for them)
  } else if (warp == W_MMA) {
    // ---- MMA issue: S of tile t, then O of tile t - 1 (the warp together, one thread issues) ----
    constexpr uint32_t id_s = umma_idesc_e4m3(128, C, false, false);
    constexpr uint32_t id_o = umma_idesc_e4m3(128, C, true, true);
    const uint32_t go = elect_one();
    bool ok = true, more = true;
    int seg = 0, fl = 0;
    for (int t = 0; more; ++t) {
      const int ds = t % ND;
      more = !(fl & kFinal);
      if (more) {
        const int slot = (2 * t) % NS;
        if (!(ok = wait(d_full(ds), (t / ND) & 1))) break;
        fl = descs[ds].flags;
        if (fl & kEnd) break;
        if (fl & kNewSeg) ok = wait(q_full, seg++ & 1);
        // (the scores of tile t - 2 were read before its weights were complete)
        ok = ok && wait(d_scales(ds), (t / ND) & 1) && wait(full(slot), ((2 * t) / NS) & 1);
        if (!ok) break;
        if (go) mbar_arrive(d_free(ds));
        tc_fence_after_sync();
        const uint32_t ka = slots + slot * X::kSlot, d = s_col + (t & 1) * C;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const uint32_t kk = ka + (k / 4) * X::kPanelBytes + (k % 4) * 32;
          const uint64_t ad = D < 128 ? umma_desc(kk, 16, 512, 4) : umma_desc(kk, 16, 1024, 2);
          umma_f8(go, d, ad, umma_desc(q_s + (k / 4) * C * 128 + (k % 4) * 32, 16, 1024, 2), id_s, k > 0);
        }
        umma_commit_if(go, s_full(t & 1));
        umma_commit_if(go, empty(slot));
      }
      if (t > 0) {  // O = V^T P^T of tile t - 1
        const int u = t - 1, slot = (2 * u + 1) % NS;
        ok = wait(full(slot), ((2 * u + 1) / NS) & 1) && (u < 2 || wait(o_free(u & 1), ((u >> 1) - 1) & 1)) &&
             wait(p_full(u % kRing), (u / kRing) & 1);
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t va = slots + slot * X::kSlot, pa = p_s + (u & 1) * X::kP, d = o_col + (u & 1) * NP * C;
#pragma unroll
        for (int c = 0; c < NP; ++c)
#pragma unroll
          for (int k = 0; k < kTile / 32; ++k) {
            const uint32_t vk = va + c * X::kPanelBytes + k * 32 * X::kRowB;
            // heads of 64: the MMA's rows 64 .. 127 repeat whatever lies 512 bytes on, and nobody reads them
            const uint64_t ad = D < 128 ? umma_desc(vk, 512, 512, 4) : umma_desc(vk, 1024, 1024, 2);
            umma_f8(go, d + c * C, ad, umma_desc(pa + k * 512, 128, 2048, 0), id_o, k > 0);
          }
        umma_commit_if(go, empty(slot));  // (first: whoever sees O done knows that no arrival is on its way)
        umma_commit_if(go, o_full(u & 1));
      }
    }
    if (!ok && lane == 0) give_up();
  } else if (warp < W_FOLD) {
    // ---- softmax: thread = token of the tile; rows R grp .. R grp + R - 1 ----
    const int grp = warp >> 2, w4 = warp & 3, tt = tid & 127;
    const uint32_t lane_col = ((uint32_t)(32 * w4) << 16) + 2 * R * grp;  // this group's columns: R first terms, R second
    uint32_t n_grp = 0, n_all = 0;  // barrier phases
    int seg = 0;
    bool ok = true;
    auto sync_group = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(grp_sync(grp));
      ok &= wait(grp_sync(grp), n_grp++ & 1);
    };
    auto sync_all = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(all_sync);
      ok &= wait(all_sync, n_all++ & 1);
    };

    // one wait a tile: its scores are there once its descriptor, its scales and O of tile t - 2 (and with it the weights'
    // buffer) are, too, as the MMA warp waits for the first two and the MMAs run in order
    int fl = kNextSeg;
    float* s_qf = s_qf2;  // this segment's (no warp is two segments ahead of another: scores wait for all)
    int2* s_lim = s_lim2;
    for (int t = 0; !(fl & kFinal); ++t) {
      const int ds = t % ND, par = t & 1, ring = t % kRing;
      const Desc& de = descs[ds];
      if (fl & kNextSeg) {
        if (!(ok = wait(d_full(ds), (t / ND) & 1))) break;
        if (de.flags & kEnd) break;
        const int j0 = de.j0, toks = min(p.TQ, de.fresh - j0);
        if (X::kStage > 0 && !(ok = wait(st_full, seg & 1))) break;
        s_qf = s_qf2 + (seg & 1) * RP;
        s_lim = s_lim2 + (seg & 1) * RP;
        ++seg;
        // query rows as e4m3 terms: TPR threads a row
        constexpr int TPR = RP <= 8 ? 128 / RP : 8, CPT = (D / 8 + TPR - 1) / TPR;
        const int row = tid / TPR, c = tid % TPR;
        const int j = row / p.G;
        const bool live = row < RP && j < toks;
        uint4 v[CPT];
        uint32_t peak = 0;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          v[i] = make_uint4(0, 0, 0, 0);
          const int ch = c + i * TPR;
          if (live && ch < D / 8)
            v[i] = X::kStage > 0 ? *reinterpret_cast<const uint4*>(stage + row * (2 * D) + ch * 16)
                                 : ld_nc_v4(p.q + (int64_t)(de.c0 + j0 + j) * p.q_stride +
                                            (int64_t)(de.h * p.G + row - j * p.G) * D + 8 * ch);
        }
#pragma unroll
        for (int i = 0; i < CPT; ++i)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t u = word_of(v[i], w) & 0x7FFF7FFFu;
            peak = max(peak, max(u & 0xFFFF, u >> 16));
          }
#pragma unroll
        for (int d = TPR / 2; d; d >>= 1) peak = max(peak, __shfl_xor_sync(0xffffffffu, peak, d));
        // largest element into (224, 448]: 448 = 1.75 * 2^8
        const int e = min(max((int)(peak >> 7) - 127 - 8 + ((peak & 127) > 96 ? 1 : 0), -120), 120);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
          const int ch = c + i * TPR;
          if (row < RP && ch < D / 8) {
            float f[8];
            widen8(v[i], f);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) split2(__fmul_rn(f[2 * w], inv), __fmul_rn(f[2 * w + 1], inv), hi[w], lo[w]);
            // K-major, 128-byte swizzle: row n = 2 R (row / R) + row % R (second terms R further) of panel ch / 16
            const int n = (row / R) * 2 * R + row % R;
            auto at = [&](int m) {
              return reinterpret_cast<uint2*>(q_mem + (ch / 16) * C * 128 + m * 128 + ((((ch % 16) >> 1) ^ (m & 7)) << 4) +
                                              (ch & 1) * 8);
            };
            *at(n) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
            *at(n + R) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
          }
        }
        if (c == 0 && row < RP) {
          const float unit = __uint_as_float((uint32_t)(127 + e) << 23);
          // a row with a NaN or an infinity is NaN as a whole
          s_qf[row] = peak >= 0x7F80 ? __uint_as_float(0x7FC00000u) : __fmul_rn(unit, p.qk_scale);
          const int pos = de.base + j0 + j;
          s_lim[row] = live ? make_int2(p.window > 0 ? pos - p.window + 1 : 0, pos) : make_int2(0, -1);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(q_full);
          if (X::kStage > 0) mbar_arrive(st_free);
        }
      }
      if (!(ok = wait(s_full(par), (t >> 1) & 1))) break;
      tc_fence_after_sync();
      // the V scale is a power of two: its exponent, and its reciprocal
      fl = de.flags;
      const int blk = tt >> p.shift;
      const float ks = de.ks[blk];
      int ve = (int)(__float_as_uint(de.vs[blk]) >> 23) - 127;
      float s[R];
      {
        float raw[2 * R];
        tmem_ld<2 * R>(s_col + par * C + lane_col, raw);
        tmem_wait_ld();
        tc_fence_before_sync();
#pragma unroll
        for (int i = 0; i < R; i += 4) {
          const float4 f = *reinterpret_cast<const float4*>(s_qf + R * grp + i);
          const float2 ff[2] = {make_float2(f.x, f.y), make_float2(f.z, f.w)};
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const float2 z = mul2(fma2(make_float2(raw[R + i + k], raw[R + i + k + 1]), make_float2(0.0625f, 0.0625f),
                                       make_float2(raw[i + k], raw[i + k + 1])), ff[k / 2]);
            s[i + k] = z.x;
            s[i + k + 1] = z.y;
          }
        }
      }
      if (fl & kFix) {
        // scores that a row does not see; V rows that no row sees (stale shared
        // memory, unset blocks) become zeros; NaN codes that only some rows see
        // are taken out of V and put into those rows' results
        const int tile = de.tile, tok = tile * kTile + tt;
        const int j0 = de.j0, toks = min(p.TQ, de.fresh - j0), pos0 = de.base + j0, pos1 = pos0 + toks - 1;
        const bool dead = ks == 0.f || tok > pos1 || (p.window > 0 && tok < pos0 - p.window + 1);
        if (dead) ve = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int2 lim = s_lim[R * grp + i];
          s[i] = dead || tok < lim.x || tok > lim.y ? -INFINITY : __fmul_rn(s[i], ks);
        }
        uint8_t* v_row = base + ((2 * t + 1) % NS) * X::kSlot;
        constexpr int kRowB = X::kRowB, kCh = kRowB / 16;
        ok = wait(full((2 * t + 1) % NS), ((2 * t + 1) / NS) & 1);
        if (!ok) break;
        bool nan_code = false;
        const bool partly = toks > 1 && !dead && (tok > pos0 || (p.window > 0 && tok < pos1 - p.window + 1));
        if (grp == 0 && (dead || partly)) {
#pragma unroll 1
          for (int c = 0; c < NP; ++c)
#pragma unroll 2
            for (int i = 0; i < kCh; ++i) {
              uint4* w = reinterpret_cast<uint4*>(v_row + c * X::kPanelBytes + tt * kRowB + ((i + tt) % kCh) * 16);
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
        if (toks > 1) {
          if (nan_code) s_nan[ring] = t + 1;
          sync_all();
          if (!ok) break;
          if (s_nan[ring] == t + 1) {
            // (rare) which tokens hold NaN in this thread's columns, which rows see one
            uint32_t taint = 0;
#pragma unroll 1
            for (int c = 0; c < NP; ++c) {
              uint32_t hit[4] = {0, 0, 0, 0};
              if (tt < kRowB)
                for (int k = 0; k < kTile; ++k) {
                  const int sw = D < 128 ? (k >> 1) & 3 : k & 7;
                  const uint8_t code = v_row[c * X::kPanelBytes + k * kRowB + (((tt >> 4) ^ sw) << 4) + (tt & 15)];
                  if ((code & 0x7F) == 0x7F) hit[k >> 5] |= 1u << (k & 31);
                }
              for (int i = 0; i < R; ++i) {
                const int2 lim = s_lim[R * grp + i];
                bool sees = false;
                for (int k = max(0, lim.x - tile * kTile); k < kTile && k <= lim.y - tile * kTile; ++k)
                  sees |= (hit[k >> 5] >> (k & 31)) & 1;
                if (sees) taint |= 1u << (c * R + i);
              }
            }
            s_taint[ring * 128 * NG + tid] = (typename X::Marks)taint;
            sync_all();
            if (!ok) break;
            if (nan_code) {
#pragma unroll 1
              for (int c = 0; c < NP; ++c)
                for (int i = 0; i < kRowB; ++i) {
                  uint8_t& code = v_row[c * X::kPanelBytes + tt * kRowB + i];
                  if ((code & 0x7F) == 0x7F) code = 0;
                }
            }
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < R; i += 2) {
          const float2 z = mul2(make_float2(s[i], s[i + 1]), make_float2(ks, ks));
          s[i] = z.x;
          s[i + 1] = z.y;
        }
      }
      // maxima over the tile: the warp, then the group's four
      float* sm = s_max + par * 4 * RP + R * grp;
      {
        const float lv = (float)ve;
        float m[R];
#pragma unroll
        for (int i = 0; i < R; i += 2) {
          const float2 z = add2(make_float2(s[i], s[i + 1]), make_float2(lv, lv));
          m[i] = warp_max(z.x);
          m[i + 1] = warp_max(z.y);
        }
        if (lane == 0) {
#pragma unroll
          for (int i = 0; i < R; i += 4)
            *reinterpret_cast<float4*>(sm + w4 * RP + i) = make_float4(m[i], m[i + 1], m[i + 2], m[i + 3]);
        }
      }
      sync_group();
      if (!ok) break;
      float top;
      {
        const float* a = sm + lane % R;
        top = fmaxf(fmaxf(a[0], a[RP]), fmaxf(a[2 * RP], a[3 * RP]));
        if (w4 == 0 && lane < R) s_top[ring * RP + R * grp + lane] = top;
        top = top == -INFINITY ? 0.f : __fsub_rn(top, 28.f);
      }
      // exp(z) in the sum's unit; times vs, it is the weight in the product's: 256 for the tile's largest (sums and O
      // carry that factor, their quotient does not).  The sum's is 2^20 of it more, so that neither is flushed where
      // it counts for vs from 2^-64 to 2^120: the largest terms of a sum are 2^(28 - log2 vs) = 2^-92 to 2^92.
#pragma unroll
      for (int i = 0; i < R; ++i) s[i] = ex2(__fsub_rn(s[i], __shfl_sync(0xffffffffu, top, i)));
      {
        const float w_unit = __uint_as_float((uint32_t)max(ve + 127 - 20, 0) << 23);
        uint32_t hi[R / 2], lo[R / 2], w[R / 2];
#pragma unroll
        for (int i = 0; i < R; i += 2) {
          const float2 pw = mul2(make_float2(s[i], s[i + 1]), make_float2(w_unit, w_unit));
          split2h(pw.x, pw.y, hi[i / 2], lo[i / 2]);
        }
#pragma unroll
        for (int i = 0; i < R / 4; ++i) {
          w[i] = hi[2 * i] | hi[2 * i + 1] << 16;
          w[R / 4 + i] = lo[2 * i] | lo[2 * i + 1] << 16;
        }
        // column 2 R grp + (R first terms, R second) of the weights: 16 columns a 16-byte row of a token, 2048 bytes on
        // the next 16
        uint8_t* dst = p_mem + par * X::kP + (2 * R * grp / 16) * 2048 + tt * 16;
        if constexpr (R == 4) {
          *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], 0, 0);
        } else if constexpr (R == 12) {  // 24 bytes: the second group's begin in the middle of a 16-byte row
          if (grp == 0) {
            *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint2*>(dst + 2048) = make_uint2(w[4], w[5]);
          } else {
            *reinterpret_cast<uint2*>(dst + 8) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint4*>(dst + 2048) = make_uint4(w[2], w[3], w[4], w[5]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < R / 8; ++i)
            *reinterpret_cast<uint4*>(dst + i * 2048) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
      }
      fence_proxy_async();
      // row sums over the warp: halves exchanged until a lane has one row, then added (one tree for every R)
      {
        constexpr int N = R == 12 ? 16 : R;  // (a power of two)
        float v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i < R ? s[i < R ? i : 0] : 0.f;
        int off = 16;
#pragma unroll
        for (int n = N / 2; n; n >>= 1, off >>= 1) {
          const bool up = lane & off;
#pragma unroll
          for (int i = 0; i < n; ++i) {
            const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, off));
          }
        }
#pragma unroll
        for (; off; off >>= 1) v[0] = __fadd_rn(v[0], __shfl_xor_sync(0xffffffffu, v[0], off));
        constexpr int kRep = 32 / N;  // lanes with the same row
        if (lane % kRep == 0 && lane / kRep < R) s_sum[(ring * 4 + w4) * RP + R * grp + lane / kRep] = v[0];
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(p_full(ring));
        mbar_arrive(d_free(ds));
      }
    }
    if (!ok && lane == 0) give_up();
  } else {
    // ---- fold: thread = output column; O of tile t into the accumulators, or out to the workspace ----
    const int fw = warp - W_FOLD, grp = fw >> 2, w4 = fw & 3, tt = 32 * w4 + lane;
    const uint32_t lane_col = ((uint32_t)(32 * w4) << 16) + 2 * R * grp;
    const bool live = D >= 128 || tt < D;
    float acc[NP][R];
    float m_run = -INFINITY, l_run = 0.f;  // lane i (< R) of every warp: row i of the group
    bool ok = true;
    ok = wait(d_full(0), 0);
    int fl = ok ? descs[0].flags & kEnd : kEnd;
    for (int t = 0; !(fl & (kFinal | kEnd)); ++t) {
      const int ds = t % ND, par = t & 1, ring = t % kRing;
      if (!(ok = wait(p_full(ring), (t / kRing) & 1))) break;
      const Desc& de = descs[ds];
      fl = de.flags;
      float mt = -INFINITY, lt = 0.f;
      if (lane < R) {
        const float* a = s_sum + ring * 4 * RP + R * grp + lane;
        mt = s_top[ring * RP + R * grp + lane];
        lt = __fmul_rn(__fadd_rn(__fadd_rn(a[0], a[RP]), __fadd_rn(a[2 * RP], a[3 * RP])), 0x1p-20f);  // in O's unit
      }
      if (fl & kGroupBegin) {
        m_run = -INFINITY;
        l_run = 0.f;
#pragma unroll
        for (int c = 0; c < NP; ++c)
#pragma unroll
          for (int i = 0; i < R; ++i) acc[c][i] = 0.f;
      }
      {
        float al, be;
        fold_ml(m_run, l_run, mt, lt, al, be);
        if (lane < R) {  // (al, al', be, be') of two rows
          float* ab = reinterpret_cast<float*>(s_ab + w4 * RP + R * grp) + (lane & ~1) * 2 + (lane & 1);
          ab[0] = al;
          ab[2] = be;
        }
        __syncwarp();
      }
      if (!(ok = wait(o_full(par), (t >> 1) & 1))) break;
      tc_fence_after_sync();
      const uint32_t poison = s_nan[ring] == t + 1 ? s_taint[ring * 128 * NG + 128 * grp + tt] : 0;
#pragma unroll
      for (int c = 0; c < NP; ++c) {
        float raw[2 * R];
        tmem_ld<2 * R>(o_col + (par * NP + c) * C + lane_col, raw);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < R; i += 2) {
          const float2 z = fma2(make_float2(raw[R + i], raw[R + i + 1]), make_float2(0.0625f, 0.0625f), make_float2(raw[i], raw[i + 1]));
          raw[i] = z.x;
          raw[i + 1] = z.y;
        }
        if (poison) {
#pragma unroll
          for (int i = 0; i < R; ++i)
            if ((poison >> (c * R + i)) & 1) raw[i] = __uint_as_float(0x7FC00000u);
        }
#pragma unroll
        for (int i = 0; i < R; i += 2) {
          const float4 ab = *reinterpret_cast<const float4*>(s_ab + w4 * RP + R * grp + i);
          const float2 z = fma2(make_float2(acc[c][i], acc[c][i + 1]), make_float2(ab.x, ab.y),
                                mul2(make_float2(raw[i], raw[i + 1]), make_float2(ab.z, ab.w)));
          acc[c][i] = z.x;
          acc[c][i + 1] = z.y;
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free(par));
      if (fl & kGroupEnd) {
        // the result: out (the segment's only group), its group slot, or its tile slot
        const int rows = min(p.TQ, de.fresh - de.j0) * p.G - R * grp;
        const bool direct = fl & kDirect, part = fl & kPart;
        const int j = R * grp / p.G, g0 = R * grp - j * p.G;
        const int64_t row0 = part ? (int64_t)de.at * RP + R * grp
                                  : ((int64_t)(direct ? 0 : de.at) * p.T + de.c0 + de.j0 + j) * p.q_heads + de.h * p.G + g0;
        const int jump = part ? 0 : (p.q_heads - p.G) * D;  // from a token's last head to the next token's first
        int64_t at = row0 * D + tt;
        int g = g0;
        float* dst = part ? p.t_acc : p.g_acc;
        const float rl = l_run != 0.f ? __frcp_rn(l_run) : 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float f = __shfl_sync(0xffffffffu, rl, i);
          if (i < rows && live) {
#pragma unroll
            for (int c = 0; c < NP; ++c) {
              if (direct) p.out[at + c * 128] = f32_to_bf16_bits(__fmul_rn(acc[c][i], f));
              else dst[at + c * 128] = acc[c][i];
            }
          }
          at += D;
          if (++g == p.G) {
            g = 0;
            at += jump;
          }
        }
        if (!direct && w4 == 0 && lane < R && lane < rows) {
          const int jl = (g0 + lane) / p.G;
          const int64_t row = row0 + lane + (part ? 0 : (int64_t)jl * (p.q_heads - p.G));
          (part ? p.t_ml : p.g_ml)[row] = make_float2(m_run, l_run);
        }
        if (fl & kLastPart) {
          // this range's parts are written: counted warp by warp; whoever counts the last will go on with the fold
          const int k = fl & kTail ? 1 : 0;
          __threadfence();
          __syncwarp();
          if (lane == 0) {
            int* n = p.counters + s_cut[k].owner;
            const int mine = s_cut[k].mine;
            if (atomicAdd(n, mine) + mine == 4 * NG * s_cut[k].count) {
              *n = 0;
              s_last[k] = 1;
              __threadfence();
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(d_free(ds));
    }
    if (!ok && lane == 0) give_up();
  }

  // ---- teardown: copies and MMAs in flight land before memory is released ----
  __syncthreads();
  if (*s_abort) {
    if (warp == W_LOAD && lane == 0)
      for (int i = max(0, loads - NS); i < loads; ++i) mbar_wait_parked(full(i % NS), (i / NS) & 1, 1000, kTries);
    if (warp == W_MMA && elect_one()) {  // one more commit covers every MMA that this thread issued
      umma_commit(drained);
      mbar_wait_parked(drained, 0, 1000, kTries);
    }
  }
  if (warp == W_MMA) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, X::kTmem);
  }
  if (*s_abort) return;

  // ---- the CTA's end: divided groups, rows that nobody computes ----
  //
  // A divided group's fold, acc = acc al_k + O_k be_k over its parts k (the
  // first range's fold, then tiles), takes its factors from the parts' (m, l)
  // alone: a thread per row works them out while the O_k are on their way to a
  // thread per four columns, all its loads in flight at once (parts by bulk copy
  // to shared memory: 16 x 20 rows over 16k tokens 62.1 instead of 61.3 us, 16 x
  // 16 rows over 4k 30.5 instead of 28.5).
  constexpr int NT = X::kThreads, V = 4;  // columns a thread takes
  if (s_last[0] | s_last[1]) {
    float2* w_ab = reinterpret_cast<float2*>(base);   // [2][RP][kGroupTiles]
    float2* w_ml = w_ab + 2 * RP * kGroupTiles;       // [2][RP]
    auto weights = [&](int k, int rr) {  // of group k's parts, row rr
      const CutGroup& c = s_cut[k];
      if (rr < 0 || rr >= c.toks * p.G) return;
      float2 ml[kGroupTiles];
#pragma unroll
      for (int z = 0; z < kGroupTiles; ++z)
        ml[z] = z < c.parts ? __ldcg(p.t_ml + c.slot[z] * RP + rr) : make_float2(-INFINITY, 0.f);
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int z = 0; z < kGroupTiles; ++z) {
        float al, be;
        fold_ml(m, l, ml[z].x, ml[z].y, al, be);
        w_ab[(k * RP + rr) * kGroupTiles + z] = make_float2(al, be);
      }
      w_ml[k * RP + rr] = make_float2(m, l);
    };
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      if (!s_last[k]) continue;
      const CutGroup& c = s_cut[k];
      const int count = c.parts, rows = c.toks * p.G;
      auto put = [&](int rr, int col, const float (&a)[V]) {
        const int jj = rr / p.G;
        const float2 ml = w_ml[k * RP + rr];
        const int64_t row = (int64_t)(c.c0 + c.j0 + jj) * p.q_heads + c.h * p.G + rr - jj * p.G;
        if (c.single) {
          const float f = ml.y != 0.f ? __frcp_rn(ml.y) : 0.f;
          uint2 w;
          w.x = (uint32_t)f32_to_bf16_bits(__fmul_rn(a[0], f)) | (uint32_t)f32_to_bf16_bits(__fmul_rn(a[1], f)) << 16;
          w.y = (uint32_t)f32_to_bf16_bits(__fmul_rn(a[2], f)) | (uint32_t)f32_to_bf16_bits(__fmul_rn(a[3], f)) << 16;
          *reinterpret_cast<uint2*>(p.out + row * D + col) = w;
        } else {
          const int64_t at = row + (int64_t)c.gi * p.T * p.q_heads;
          *reinterpret_cast<float4*>(p.g_acc + at * D + col) = make_float4(a[0], a[1], a[2], a[3]);
          if (col == 0) p.g_ml[at] = ml;
        }
      };
      bool first = true;
      for (int i = tid; i < (rows * (D / V) + NT - 1) / NT * NT; i += NT) {
        const int rr = i / (D / V), col = V * (i - rr * (D / V));
        float v[kGroupTiles][V];
#pragma unroll
        for (int z = 0; z < kGroupTiles; ++z) {
          const bool is = z < count && rr < rows;
          const float* from = p.t_acc + ((int64_t)(is ? c.slot[z] : 0) * RP + (is ? rr : 0)) * D + col;
          const float4 u = is ? __ldcg(reinterpret_cast<const float4*>(from)) : make_float4(0.f, 0.f, 0.f, 0.f);
          v[z][0] = u.x, v[z][1] = u.y, v[z][2] = u.z, v[z][3] = u.w;
        }
        if (first) {
          first = false;
          weights(k, tid);
          __syncthreads();
        }
        if (rr >= rows) continue;
        float a[V];
#pragma unroll
        for (int q = 0; q < V; ++q) a[q] = 0.f;
#pragma unroll
        for (int z = 0; z < kGroupTiles; ++z) {
          const float2 ab = w_ab[(k * RP + rr) * kGroupTiles + z];
#pragma unroll
          for (int q = 0; q < V; ++q) a[q] = __fmaf_rn(a[q], ab.x, __fmul_rn(v[z][q], ab.y));
        }
        put(rr, col, a);
      }
    }
  }
  if (s_rest[0] > 0) {
    // (rare) padding rows and rows of requests that were left out: zeros
    for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
      bool bad_req = false;
      const Req rq = load_req(p, find_request(p.cu, p.B, p.t0 + t), &bad_req);
      if (s_rest[1] > 0 && t >= rq.c0 && t < rq.c0 + rq.fresh) continue;  // (no tiles: a refused step)
      for (int i = tid; i < p.q_heads * (D / 8); i += NT)
        *reinterpret_cast<uint4*>(p.out + (int64_t)t * p.q_heads * D + 8 * i) = make_uint4(0, 0, 0, 0);
    }
  }
}

// ---- combine -----------------------------------------------------------------------------------
//
// The join of rows of several groups.  A thread has four columns; SETS thread
// sets share a row's groups, neighbouring ones each, and join as a tree in
// shared memory: 4; 1 for many rows of at most eight groups, all requested at
// once; or 128 for few rows of very many, 32 columns a CTA.  Reads what the
// attention kernel wrote a moment ago (L2), so it is a chain of latencies:
// request (guessed, then checked), its lengths, results; about 4 us of a call.
// Whole calls with 1 and 4 sets: 1024 rows of 8 groups 52.9 and 52.0 us, 17.5k
// rows of 6 groups 192.8 and 210.6; with 4 and 128: 8 rows of 128 groups 43.8
// and 34.7.

template <int D, int SETS>
__global__ void __launch_bounds__(SETS == 128 ? 1024 : 256) kv_combine_kernel(const __grid_constant__ Params p) {
  constexpr int LANES = SETS == 128 ? 8 : D / 4, kPer = SETS == 128 ? 1 : 256 / LANES / SETS;  // rows of a CTA
  __shared__ State s_set[SETS == 1 ? 1 : kPer * SETS][LANES];
  const int set = threadIdx.x / LANES % SETS, sub = threadIdx.x / (LANES * SETS), c = threadIdx.x % LANES;
  const int col = (SETS == 128 ? (int)blockIdx.y * 32 : 0) + 4 * c, rows = p.T * p.q_heads;
  // (no early launch of what follows: a next attention call's CTAs would fill the SMs unevenly around this kernel's:
  // 32 ragged requests to 8k back to back 73 instead of 54 us)
  // The first row's request is looked up before the wait.  What is read there may be older than this step's (only a
  // wait makes another grid's writes visible), so one thread a row looks again beside the results' loads (the lookup
  // after the wait: 53.1 instead of 52.1 us of 32 requests, window 24.6 instead of 23.4).
  bool waited = false;
  for (int row0 = (int)blockIdx.x * kPer; row0 < rows; row0 += kPer * (int)gridDim.x) {
    const int row = min(row0 + sub, rows - 1), t = row / p.q_heads, hq = row - t * p.q_heads;
    State out;
    bool mine;
    for (bool again = true; again;) {
      int b = min((p.t0 + t) / p.max_new, p.B - 1);  // right where every request has max_new new tokens
      RawReq raw(p, b);
      if (raw.c0 > p.t0 + t || raw.c1 <= p.t0 + t) {
        b = find_request(p.cu, p.B, p.t0 + t);
        raw = RawReq(p, b);
      }
      bool bad = false;
      const Req r = check_req(p, raw, &bad);
      const int j = t - r.c0;
      const int rt = r.fresh <= p.TQ ? 0 : j / p.TQ;
      // (other rows are written already)
      mine = row0 + sub < rows && j >= 0 && j < r.fresh &&
             first_tile(p, r, rt) / kGroupTiles != last_tile(p, r, rt) / kGroupTiles;
      out = empty_state();
      const RowGroups<D> g(p, r, j, hq);
      RawReq now = raw;
      int odd = 0;
      if (!waited) {
        pdl_wait();
        if (set == 0 && c == 0) now = RawReq(p, b), odd = __ldcg(p.refused);
      }
      if (mine) {
        if constexpr (SETS == 1) {
          State st[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) st[k] = g.group(p, k, col);
#pragma unroll
          for (int n = 1; n < 8; n <<= 1)
#pragma unroll
            for (int k = 0; k + n < 8; k += 2 * n) fold_state(st[k], st[k + n]);
          out = st[0];
        } else {
          int per = 1;
          while (per * SETS < g.n) per *= 2;
          if (per * set < g.n) out = g.tree(p, per * set, per, col);
        }
      }
      again = !waited && __syncthreads_or(now.c0 != raw.c0 || now.c1 != raw.c1 || now.len != raw.len || odd);
      waited = true;
      if (again && __ldcg(p.refused)) return;  // the attention kernel wrote zeros, and no groups
    }
    if constexpr (SETS > 1) {
      s_set[sub * SETS + set][c] = out;
      for (int k = 1; k < SETS; k <<= 1) {
        __syncthreads();
        if (set % (2 * k) == 0) {
          fold_state(out, s_set[sub * SETS + set + k][c]);
          s_set[sub * SETS + set][c] = out;
        }
      }
    }
    if (mine && set == 0) write_out(p, (int64_t)row * D + col, out);
    if constexpr (SETS > 1) __syncthreads();
  }
  if (!waited) pdl_wait();
}

// ---- host side -----------------------------------------------------------------------------------

// A row has a slot for every group of the longest request, 4 dim + 8 bytes a query head.  So that the workspace stays
// bounded, a call whose rows need more takes them in several launches, a row tile's at least (8192 rows of 32 x 128
// over 131,072 tokens would take 17 GB).  Where the longest request is as long as max_len, a launch that fills this is
// milliseconds of work and the division costs nothing (8192 rows after 100k tokens: 46.1 ms, undivided 47.0); where
// it is much shorter, launches are short (2048 rows from an empty cache with a max_len of 131,072: 264 us in two
// launches, 241 undivided; 284 with half of this, 319 with a quarter).
constexpr int64_t kGroupBytes = (int64_t)1 << 32;

struct Layout {
  int rows;  // of a launch
  int RP, TQ, gmax, grid, t_slots, seg_cost;
  bool fits;  // positions on the line and rows of group results fit in 31 bits
  size_t g_acc, g_ml, t_acc, t_ml, refused, bytes;
};

template <int D>
int ctas_d(int RP) {
  switch (RP) {
    case 4: return Geo<D, 4>::kCtas;
    case 8: return Geo<D, 8>::kCtas;
    case 12: return Geo<D, 12>::kCtas;
    case 16: return Geo<D, 16>::kCtas;
    case 24: return Geo<D, 24>::kCtas;
    default: return Geo<D, 32>::kCtas;
  }
}
int ctas_per_sm(int dim, int RP) { return dim == 64 ? ctas_d<64>(RP) : dim == 128 ? ctas_d<128>(RP) : ctas_d<256>(RP); }

// Positions of the line that a segment takes besides its tiles: a new segment's
// queries have to be split before its first scores, which the tiles of its first
// CTA pay for.  Measured with 0 / 1 / 2 / 3: 32 rows, segments of 12 to 48
// tiles 222 / 210 / 202 / 202 us; 12 rows, 9 tiles 26.2 / 25.2 / 24.1 / 25.5; 24
// rows, 125 tiles 63.5 / 61.7 / 61.6 / 61.3; 4 rows, 62 tiles 53.0 / 53.3 /
// 53.6 / 54.4 (two CTAs an SM hide it).
int seg_cost(int RP) { return RP < 12 ? 0 : 2; }

Layout make_layout(int B, int T, int q_heads, int heads, int dim, int max_new, int max_len, int window) {
  Layout y;
  const int G = q_heads / heads;
  if (max_new > T) max_new = T;
  int64_t groups = ((int64_t)max_len + kGroupTokens - 1) / kGroupTokens;
  if (window > 0) {
    const int64_t span = ((int64_t)window + max_new - 2) / kGroupTokens + 2;
    if (span < groups) groups = span;
  }
  y.gmax = (int)groups;
  const int all = T;
  const int64_t row_bytes = groups > 1 ? groups * q_heads * ((int64_t)dim * 4 + 8) : 0;  // (one group: written out at once)
  if (row_bytes * T > kGroupBytes) {
    int64_t most = kGroupBytes / row_bytes;
    if (most < 32 / G) most = 32 / G;
    const int64_t launches = (T + most - 1) / most;
    T = (int)((T + launches - 1) / launches);
    if (max_new > T) max_new = T;
  }
  y.rows = T;
  // the smallest row tile that holds the step's rows of a key head, or 32 rows, and at least one token
  const int64_t hold = (int64_t)G * max_new < 32 ? (int64_t)G * max_new : 32;
  y.RP = hold <= 4 ? 4 : hold <= 8 ? 8 : hold <= 12 ? 12 : hold <= 16 ? 16 : hold <= 24 ? 24 : 32;
  y.TQ = y.RP / G;
  y.seg_cost = seg_cost(y.RP);
  // no more CTAs than tiles
  const int64_t per = ((int64_t)max_len + kTile - 1) / kTile;
  const int64_t row_tiles = most_row_tiles(B, T, y.TQ, max_new);
  y.fits = (double)row_tiles * heads * (double)(per + y.seg_cost) <= INT32_MAX && (double)y.gmax * all * q_heads <= INT32_MAX;
  if (!y.fits) return y;
  const int64_t most = row_tiles * heads * (per + y.seg_cost);
  const int full = kSms * ctas_per_sm(dim, y.RP);
  y.grid = most < full ? (int)most : full;
  const int64_t range = (most + y.grid - 1) / y.grid;
  y.t_slots = (int)(range < kGroupTiles ? range : kGroupTiles);  // a range's first seven tiles at most, and its end
  auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
  y.g_acc = 0;
  const size_t group_rows = y.gmax > 1 ? (size_t)y.gmax * T * q_heads : 0;
  y.g_ml = y.g_acc + up(group_rows * dim * 4);
  y.t_acc = y.g_ml + up(group_rows * 8);
  y.t_ml = y.t_acc + up((size_t)y.grid * y.t_slots * y.RP * dim * 4);
  y.refused = y.t_ml + up((size_t)y.grid * y.t_slots * y.RP * 8);
  y.bytes = y.refused + up(4);
  return y;
}

std::mutex g_attr_mu;
bool g_attr[64][3][33] = {};

template <int D, int RP>
cudaError_t run(const KvAttentionArgs& a, const Layout& y, Params p, int pdl, cudaStream_t s) {
  using X = Geo<D, RP>;
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(g_attr_mu);
    bool& done = g_attr[dev][D == 64 ? 0 : D == 128 ? 1 : 2][RP];
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
  for (p.t0 = 0; p.t0 < a.T; p.t0 += y.rows) {
    p.T = a.T - p.t0 < y.rows ? a.T - p.t0 : y.rows;
    p.q = a.q + p.t0 * a.q_stride;
    p.out = a.out + (int64_t)p.t0 * a.q_heads * D;
    cfg.gridDim = dim3((unsigned)y.grid);
    cfg.blockDim = dim3(X::kThreads);
    cfg.dynamicSmemBytes = (size_t)X::kSmem;
    if (cudaError_t e = cudaLaunchKernelEx(&cfg, kv_attention_kernel<D, RP>, maps, p)) return e;
    if (y.gmax == 1) continue;
    const int64_t out_rows = (int64_t)p.T * a.q_heads;
    cfg.dynamicSmemBytes = 0;
    cudaError_t e;
    if (y.gmax > 16 && out_rows * (D / 32) <= 2 * kSms) {
      cfg.gridDim = dim3((unsigned)out_rows, D / 32);
      cfg.blockDim = dim3(1024);
      e = cudaLaunchKernelEx(&cfg, kv_combine_kernel<D, 128>, p);
    } else {
      const int per4 = 256 / (D / 4) / 4;
      const int sets = y.gmax <= 8 && out_rows > 12 * kSms * per4 ? 1 : 4, per = 4 / sets * per4;  // (1: more than two rounds of 4)
      const int64_t ctas = (out_rows + per - 1) / per;
      cfg.gridDim = dim3((unsigned)(ctas < 6 * kSms ? ctas : 6 * kSms));
      cfg.blockDim = dim3(256);
      e = sets == 1 ? cudaLaunchKernelEx(&cfg, kv_combine_kernel<D, 1>, p) : cudaLaunchKernelEx(&cfg, kv_combine_kernel<D, 4>, p);
    }
    if (e) return e;
  }
  return cudaSuccess;
}

template <int D>
cudaError_t run_d(const KvAttentionArgs& a, const Layout& y, const Params& p, int pdl, cudaStream_t s) {
  switch (y.RP) {
    case 4: return run<D, 4>(a, y, p, pdl, s);
    case 8: return run<D, 8>(a, y, p, pdl, s);
    case 12: return run<D, 12>(a, y, p, pdl, s);
    case 24: return run<D, 24>(a, y, p, pdl, s);
    case 16: return run<D, 16>(a, y, p, pdl, s);
    default: return run<D, 32>(a, y, p, pdl, s);
  }
}

}  // namespace

size_t kv_attention_workspace(int B, int T, int q_heads, int kv_heads, int dim, int max_new, int max_len, int window) {
  const Layout y = make_layout(B, T, q_heads, kv_heads, dim, max_new, max_len, window);
  return y.fits ? y.bytes : 0;
}

cudaError_t launch_kv_attention(const KvAttentionArgs& a, int pdl, cudaStream_t s) {
  const Layout y = make_layout(a.B, a.T, a.q_heads, a.cache.heads, a.cache.dim, a.max_new, a.max_len, a.window);
  uint8_t* w = static_cast<uint8_t*>(a.ws);
  Params p;
  p.q_stride = a.q_stride;
  p.k_scale = a.cache.k_scale;
  p.v_scale = a.cache.v_scale;
  p.table = a.table;
  p.cu = a.cu;
  p.lens = a.lens;
  p.B = a.B;
  p.all = a.T;
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
  p.seg_cost = y.seg_cost;
  p.t_slots = y.t_slots;
  p.g_acc = reinterpret_cast<float*>(w + y.g_acc);
  p.g_ml = reinterpret_cast<float2*>(w + y.g_ml);
  p.t_acc = reinterpret_cast<float*>(w + y.t_acc);
  p.t_ml = reinterpret_cast<float2*>(w + y.t_ml);
  p.refused = reinterpret_cast<int*>(w + y.refused);
  p.arrivals = a.fault_wait ? 2 : 1;
  p.flags = a.flags;
  p.counters = a.counters;
  switch (a.cache.dim) {
    case 64: return run_d<64>(a, y, p, pdl, s);
    case 128: return run_d<128>(a, y, p, pdl, s);
    default: return run_d<256>(a, y, p, pdl, s);
  }
}

}  // namespace w4a16
