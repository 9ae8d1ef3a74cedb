// kv_attention.cu -- attention over the paged 8-bit key/value cache
// (w4a16_kv_attention; the formulas are those of include/w4a16.h "Paged
// key/value cache").
//
// One CTA per (token, query head): a thread per cached token for the scores
// of a tile of 128 tokens, then a thread per output column for the products
// with V; running maximum and sum in fp32.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv.cuh"
#include "ptx.cuh"

namespace w4a16 {
namespace {

using namespace ptx;

struct Params {
  KvAttentionArgs a;
  int shift;
};

__device__ __forceinline__ float e4m3(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

__global__ void __launch_bounds__(128) kv_attention_kernel(Params p) {
  __shared__ float s_q[256], s_p[128], s_red[4];
  __shared__ int64_t s_row[128];
  const KvAttentionArgs& a = p.a;
  const int tid = threadIdx.x, t = blockIdx.x, hq = blockIdx.y;
  const int dim = a.cache.dim, h = hq / (a.q_heads / a.cache.heads);
  pdl_wait();
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int b = lo, c0 = a.cu[b], c1 = a.cu[b + 1];
  int first = 0, last = -1;
  if (t >= c0 && t < c1) {
    const int len = a.lens[b], fresh = c1 - c0;
    if (fresh > a.max_new || len > a.max_len || len < fresh) {
      if (tid == 0) atomicOr(a.flags, W4A16_DEVICE_KV_RANGE);
    } else {
      last = len - fresh + t - c0;
      first = a.window > 0 ? max(0, last - a.window + 1) : 0;
    }
  }
  for (int d = tid; d < dim; d += 128) s_q[d] = bf16_bits_to_f32(a.q[(int64_t)t * a.q_stride + hq * dim + d]);
  __syncthreads();
  float m = -INFINITY, l = 0.f, acc[2] = {0.f, 0.f};
  for (int base = first; base <= last; base += 128) {
    const int tok = base + tid;
    float s = -INFINITY, vs = 0.f;
    int64_t row = -1;
    if (tok <= last) {
      const int blk = a.table[(int64_t)b * a.max_blocks + (tok >> p.shift)];
      if (blk >= 0 && blk < a.cache.blocks) {
        const int64_t at = (int64_t)blk * a.cache.heads + h;
        row = ((at << p.shift) + (tok & (a.cache.block - 1))) * dim;
        float dot = 0.f;
        for (int d = 0; d < dim; ++d) dot = __fmaf_rn(s_q[d], e4m3(a.cache.k[row + d]), dot);
        s = dot * a.cache.k_scale[at] * a.scale;
        vs = a.cache.v_scale[at];
      } else {
        atomicOr(a.flags, W4A16_DEVICE_KV_RANGE);
      }
    }
    float mx = s;
    for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    if ((tid & 31) == 0) s_red[tid >> 5] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    const float mn = fmaxf(m, mx), safe = mn == -INFINITY ? 0.f : mn;
    const float al = expf(m - safe);
    const float e = row >= 0 ? expf(s - safe) : 0.f;
    s_p[tid] = e * vs;
    s_row[tid] = row;
    float sum = e;
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    __syncthreads();
    if ((tid & 31) == 0) s_red[tid >> 5] = sum;
    __syncthreads();
    l = l * al + (s_red[0] + s_red[1] + s_red[2] + s_red[3]);
    m = mn;
    for (int i = 0; i < 2; ++i) {
      const int d = tid + 128 * i;
      if (d >= dim) break;
      float x = acc[i] * al;
      for (int k = 0; k < 128; ++k)
        if (s_row[k] >= 0) x = __fmaf_rn(s_p[k], e4m3(a.cache.v[s_row[k] + d]), x);
      acc[i] = x;
    }
    __syncthreads();
  }
  for (int i = 0; i < 2; ++i) {
    const int d = tid + 128 * i;
    if (d < dim) a.out[((int64_t)t * a.q_heads + hq) * dim + d] = f32_to_bf16_bits(l == 0.f ? 0.f : acc[i] / l);
  }
}

}  // namespace

size_t kv_attention_workspace(int, int, int, int, int, int, int, int) { return 0; }

cudaError_t launch_kv_attention(const KvAttentionArgs& a, int pdl, cudaStream_t s) {
  (void)pdl;
  Params p{a, __builtin_ctz((unsigned)a.cache.block)};
  kv_attention_kernel<<<dim3((unsigned)a.T, (unsigned)a.q_heads), 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace w4a16
