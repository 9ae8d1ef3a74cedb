// kv.cuh -- internal interface between the C-ABI (api.cu) and the kernels of
// the paged 8-bit key/value cache (kv.cu, kv_attention.cu).  Host-side only.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "w4a16.h"

namespace w4a16 {

struct KvPlanArgs {
  const int32_t* cached;
  const int32_t* fresh;  // new tokens per request
  int32_t* table;
  const int32_t* free_blocks;
  const int32_t* head;  // entries of free_blocks taken before this call (device), or nullptr for 0
  int32_t* cu;
  int32_t* lens;
  int32_t* slots;
  int32_t* positions;
  int32_t* head_out;
  int B, T, block, max_blocks, n_free;
  int* flags;
};
cudaError_t launch_kv_plan(const KvPlanArgs& a, int pdl, cudaStream_t s);

struct KvAppendArgs {
  const uint16_t* k;  // bf16 [T][heads][dim], tokens k_stride elements apart
  const uint16_t* v;
  int64_t k_stride, v_stride;
  const int32_t* slots;
  w4a16_kv_cache cache;
  int T;
  int* flags;
};
cudaError_t launch_kv_append(const KvAppendArgs& a, int pdl, cudaStream_t s);

struct KvAttentionArgs {
  const uint16_t* q;  // bf16 [T][q_heads][dim], tokens q_stride elements apart
  int64_t q_stride;
  w4a16_kv_cache cache;
  const int32_t* table;
  const int32_t* cu;
  const int32_t* lens;
  uint16_t* out;  // bf16 [T][q_heads][dim]
  int B, T, q_heads, max_blocks, max_new, max_len, window;
  float scale;
  void* ws;
  int* counters;
  int* flags;
  int fault_wait;  // debug (W4A16_FAULT=wait): the first CTA's first slot waits for an arrival that never comes
};
size_t kv_attention_workspace(int B, int T, int q_heads, int kv_heads, int dim, int max_new, int max_len, int window);
cudaError_t launch_kv_attention(const KvAttentionArgs& a, int pdl, cudaStream_t s);

}  // namespace w4a16
