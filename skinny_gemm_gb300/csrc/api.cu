// api.cu -- the C ABI of libw4a16.so (declared and documented in include/w4a16.h).
//
// Host-side validation happens before any launch and a rejected call writes
// nothing (fail closed, after tiny-llm "Week 2 Day 2: Keep W4 Packed",
// section "Task 2": validate inputs, reject unsupported evaluation
// explicitly).  The kernel family and its reduction order are chosen from
// (N, K) only; M only decides how many chunks of at most eight rows run.
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <string>

#include "common.cuh"
#include "fp4.cuh"
#include "kv.cuh"
#include "launch.h"
#include "stq1.cuh"
#include "stq1.h"

namespace w4a16 {
namespace {

__device__ int g_device_flags;

thread_local std::string g_last_error;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

int cuda_fail(cudaError_t e, const char* what) {
  return fail(W4A16_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

// ---- debug switches read once from the environment -----------------------------

enum Fault { kFaultNone = 0, kFaultValidate = 1, kFaultLaunch = 2, kFaultWait = 3 };

struct EnvConfig {
  int fault = kFaultNone;
  int force_kernel = W4A16_KERNEL_AUTO;
  int pdl = 2;  // W4A16_PDL: 0 plain launches, 1 overlap launches only, 2 also fetch weights early
};

std::mutex g_env_mu;
bool g_env_loaded = false;
EnvConfig g_env;

void load_env_locked() {
  EnvConfig c;
  if (const char* f = std::getenv("W4A16_FAULT")) {
    if (!std::strcmp(f, "validate")) c.fault = kFaultValidate;
    else if (!std::strcmp(f, "launch")) c.fault = kFaultLaunch;
    else if (!std::strcmp(f, "wait")) c.fault = kFaultWait;
  }
  if (const char* v = std::getenv("W4A16_PDL")) {
    if (v[0] >= '0' && v[0] <= '2' && v[1] == 0) c.pdl = v[0] - '0';
  }
  if (const char* k = std::getenv("W4A16_FORCE_KERNEL")) {
    if (!std::strcmp(k, "simt")) c.force_kernel = W4A16_KERNEL_SIMT;
    else if (!std::strcmp(k, "tc")) c.force_kernel = W4A16_KERNEL_TC;
    else if (!std::strcmp(k, "vanilla")) c.force_kernel = W4A16_KERNEL_VANILLA;
  }
  g_env = c;
  g_env_loaded = true;
}

EnvConfig env() {
  std::lock_guard<std::mutex> lk(g_env_mu);
  if (!g_env_loaded) load_env_locked();
  return g_env;
}

// ---- device flag word, one per device ------------------------------------------

constexpr int kMaxDevices = 64;
std::mutex g_flag_mu;
int* g_flag_ptr[kMaxDevices] = {};

int flag_pointer(int** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(W4A16_ERR_CUDA, "device ordinal %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_flag_mu);
  if (!g_flag_ptr[dev]) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_device_flags);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(device flags)");
    g_flag_ptr[dev] = static_cast<int*>(p);
  }
  *out = g_flag_ptr[dev];
  return W4A16_OK;
}

// ---- host threads on one stream --------------------------------------------------
//
// A call of several launches hands its workspace from one to the next.  Threads
// that launch such calls on one stream take turns, so that nothing that shares
// the workspace comes between (a stream has a workspace, and PyTorch's threads
// have one current stream).  Some streams share a turn.

constexpr int kTurns = 64;
std::mutex g_turns[kTurns];

std::mutex& turn_of(const void* stream) {
  const uint64_t h = reinterpret_cast<uintptr_t>(stream) * 0x9E3779B97F4A7C15ull;
  return g_turns[h >> 58];
}
static_assert(kTurns == 1 << (64 - 58), "the hash's bits");

// ---- validation ------------------------------------------------------------------

constexpr int kMaxDim = 1 << 30;

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

int check_nk(int N, int K) {
  if (N <= 0 || N > kMaxDim) return fail(W4A16_ERR_SHAPE, "N = %d must be in 1..2^30", N);
  if (K <= 0 || K > kMaxDim || K % kGroup) return fail(W4A16_ERR_SHAPE, "K = %d must be a positive multiple of 64", K);
  return W4A16_OK;
}

int resolve_kernel(int requested, int N, int K, w4a16_plan* plan) {
  int k = requested;
  if (k == W4A16_KERNEL_AUTO) k = env().force_kernel;
  // Default: the tensor-core family wherever it applies (K % 512 == 0, and
  // K % 512 != 0 padded to whole 512-code stages up to the K whose per-unit
  // parameter rows fit in shared memory), the CUDA-core family otherwise.
  // The choice depends on (N, K) only.
  if (k == W4A16_KERNEL_AUTO) k = tc_supported(N, K) ? W4A16_KERNEL_TC : W4A16_KERNEL_SIMT;
  switch (k) {
    case W4A16_KERNEL_SIMT: plan_simt(N, K, plan); return W4A16_OK;
    case W4A16_KERNEL_VANILLA: plan_vanilla(N, K, plan); return W4A16_OK;
    case W4A16_KERNEL_TC:
    case W4A16_KERNEL_TC_STREAM:
    case W4A16_KERNEL_TC_TILE:
    case W4A16_KERNEL_TC_PREFILL: {
      if (!tc_supported(N, K))
        return fail(W4A16_ERR_KERNEL, "K = %d is past the tensor-core kernels' K %% 512 != 0 range", K);
      if (K % 512 && k == W4A16_KERNEL_TC_PREFILL)
        return fail(W4A16_ERR_KERNEL, "the prefill kernel needs K %% 512 == 0 (K = %d)", K);
      const int path = k == W4A16_KERNEL_TC_STREAM ? 1 : k == W4A16_KERNEL_TC_TILE ? 2 : 0;
      if (path == 2 && !tc_tile_fits(N, K, 1))
        return fail(W4A16_ERR_KERNEL, "the tile kernel cannot hold K = %d in shared memory", K);
      plan_tc(N, K, path, plan);
      if (k == W4A16_KERNEL_TC_PREFILL) plan->kernel = W4A16_KERNEL_TC_PREFILL;
      return W4A16_OK;
    }
    default: return fail(W4A16_ERR_KERNEL, "unknown kernel selector %d", requested);
  }
}

int validate_mm(const void* x, const void* Wq, const void* S, const void* B, const void* y, int M, int N, int K) {
  if (M < 0 || M > kMaxDim) return fail(W4A16_ERR_SHAPE, "M = %d must be in 0..2^30", M);
  if (int rc = check_nk(N, K)) return rc;
  if (M == 0) return W4A16_OK;
  if (!x || !Wq || !S || !B || !y) return fail(W4A16_ERR_NULL, "null tensor pointer");
  if (misaligned(x, 16) || misaligned(Wq, 16)) return fail(W4A16_ERR_ALIGN, "x and Wq must be 16-byte aligned");
  if (misaligned(S, 8) || misaligned(B, 8)) return fail(W4A16_ERR_ALIGN, "scales and biases must be 8-byte aligned");
  if (misaligned(y, 2)) return fail(W4A16_ERR_ALIGN, "y must be 2-byte aligned");
  return W4A16_OK;
}

// A caller's workspace: NULL (none), or at least tc_workspace_bytes() bytes,
// 256-byte aligned.
int check_workspace(const void* ws, size_t bytes) {
  if (!ws) return W4A16_OK;
  if (misaligned(ws, 256)) return fail(W4A16_ERR_ALIGN, "the workspace must be 256-byte aligned");
  if (bytes < tc_workspace_bytes())
    return fail(W4A16_ERR_SHAPE, "a workspace of %zu bytes is too small (w4a16_workspace_bytes: %zu)", bytes,
                tc_workspace_bytes());
  return W4A16_OK;
}

int run_mm(const w4a16_bf16* x, const uint32_t* Wq, const w4a16_bf16* S, const w4a16_bf16* B, w4a16_bf16* y,
           int M, int N, int K, int kernel, void* stream, void* ws = nullptr, size_t ws_bytes = 0) {
  if (env().fault == kFaultValidate) return fail(W4A16_ERR_SHAPE, "injected validation fault (W4A16_FAULT)");
  if (int rc = validate_mm(x, Wq, S, B, y, M, N, K)) return rc;
  if (int rc = check_workspace(ws, ws_bytes)) return rc;
  w4a16_plan plan;
  if (int rc = resolve_kernel(kernel, N, K, &plan)) return rc;
  if (M == 0) return W4A16_OK;
  if (env().fault == kFaultLaunch) return fail(W4A16_ERR_CUDA, "injected launch fault (W4A16_FAULT)");
  LaunchArgs a{};
  a.x = x; a.Wq = Wq; a.S = S; a.B = B; a.y = y;
  a.N = N; a.K = K;
  a.stream = static_cast<cudaStream_t>(stream);
  a.pdl = env().pdl;
  a.tc_path = plan.kernel == W4A16_KERNEL_TC_STREAM ? 1 : plan.kernel == W4A16_KERNEL_TC_TILE ? 2
             : plan.kernel == W4A16_KERNEL_TC_PREFILL ? 3 : 0;
  a.ws = ws;
  a.ws_bytes = ws_bytes;
  a.fault_wait = env().fault == kFaultWait;
  if (int rc = flag_pointer(&a.flags)) return rc;
  const bool tc = plan.kernel == W4A16_KERNEL_TC || plan.kernel == W4A16_KERNEL_TC_STREAM ||
                  plan.kernel == W4A16_KERNEL_TC_TILE || plan.kernel == W4A16_KERNEL_TC_PREFILL;
  if (a.tc_path == 2 && !tc_tile_fits(N, K, M < kMaxChunk ? M : kMaxChunk))
    return fail(W4A16_ERR_KERNEL, "the tile kernel cannot hold K = %d for %d rows in shared memory", K,
                M < kMaxChunk ? M : kMaxChunk);
  // The tensor-core family takes all M rows at once (the tile kernel streams
  // them over resident weights, the persistent kernel launches per chunk);
  // the CUDA-core and control kernels take chunks of at most eight rows.
  for (int row0 = 0; row0 < M; row0 += tc ? M : kMaxChunk) {
    a.row0 = row0;
    a.M = tc ? M : (M - row0 < kMaxChunk) ? M - row0 : kMaxChunk;
    cudaError_t e = cudaSuccess;
    switch (plan.kernel) {
      case W4A16_KERNEL_SIMT: e = launch_simt(a, plan); break;
      case W4A16_KERNEL_TC:
      case W4A16_KERNEL_TC_STREAM:
      case W4A16_KERNEL_TC_TILE:
      case W4A16_KERNEL_TC_PREFILL: e = launch_tc(a, plan); break;
      case W4A16_KERNEL_VANILLA: e = launch_vanilla(a, plan); break;
      default: return fail(W4A16_ERR_KERNEL, "kernel %d cannot run", plan.kernel);
    }
    if (e != cudaSuccess) return cuda_fail(e, "w4a16_mm launch");
  }
  return W4A16_OK;
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

int w4a16_mm(const w4a16_bf16* x, const uint32_t* Wq, const w4a16_bf16* scales, const w4a16_bf16* biases,
             w4a16_bf16* y, int M, int N, int K, void* stream) {
  return run_mm(x, Wq, scales, biases, y, M, N, K, W4A16_KERNEL_AUTO, stream);
}

int w4a16_mm_ws(const w4a16_bf16* x, const uint32_t* Wq, const w4a16_bf16* scales, const w4a16_bf16* biases,
                w4a16_bf16* y, int M, int N, int K, void* workspace, size_t workspace_bytes, void* stream) {
  return run_mm(x, Wq, scales, biases, y, M, N, K, W4A16_KERNEL_AUTO, stream, workspace, workspace_bytes);
}

int w4a16_mm_g(const w4a16_bf16* x, const uint32_t* Wq, const w4a16_bf16* scales, const w4a16_bf16* biases,
               w4a16_bf16* y, int M, int N, int K, int group, void* workspace, size_t workspace_bytes, void* stream) {
  if (group == kGroup)
    return run_mm(x, Wq, scales, biases, y, M, N, K, W4A16_KERNEL_AUTO, stream, workspace, workspace_bytes);
  if (env().fault == kFaultValidate) return fail(W4A16_ERR_SHAPE, "injected validation fault (W4A16_FAULT)");
  if (group != 128) return fail(W4A16_ERR_SHAPE, "group = %d must be 64 or 128", group);
  if (int rc = validate_mm(x, Wq, scales, biases, y, M, N, K)) return rc;
  if (K % 512 || K > 8192)
    return fail(W4A16_ERR_SHAPE,
                "group 128 runs natively for K %% 512 == 0 up to 8192 (K = %d); expand the tables to group 64 "
                "with w4a16_expand_groups for other K", K);
  if (misaligned(scales, 16) || misaligned(biases, 16))
    return fail(W4A16_ERR_ALIGN, "group-128 scales and biases must be 16-byte aligned");
  if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
  if (M == 0) return W4A16_OK;
  if (env().fault == kFaultLaunch) return fail(W4A16_ERR_CUDA, "injected launch fault (W4A16_FAULT)");
  LaunchArgs a{};
  a.x = x; a.Wq = Wq; a.S = scales; a.B = biases; a.y = y;
  a.N = N; a.K = K; a.M = M; a.row0 = 0;
  a.stream = static_cast<cudaStream_t>(stream);
  a.pdl = env().pdl;
  a.tc_path = 1;
  a.ws = workspace;
  a.ws_bytes = workspace_bytes;
  if (int rc = flag_pointer(&a.flags)) return rc;
  cudaError_t e = launch_tc_g128(a);
  return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "w4a16_mm_g launch");
}

size_t w4a16_workspace_bytes(int N, int K) {
  if (N <= 0 || K <= 0 || K % kGroup || !tc_supported(N, K)) return 0;
  return tc_workspace_bytes();
}

int w4a16_mm_kernel(const w4a16_bf16* x, const uint32_t* Wq, const w4a16_bf16* scales, const w4a16_bf16* biases,
                    w4a16_bf16* y, int M, int N, int K, int kernel, void* stream) {
  return run_mm(x, Wq, scales, biases, y, M, N, K, kernel, stream);
}

int w4a16_mm_id(const w4a16_bf16* x, const uint32_t* Wq, const w4a16_bf16* scales, const w4a16_bf16* biases,
                const int32_t* ids, w4a16_bf16* y, int T, int N, int K, int E, void* stream) {
  return w4a16_mm_id_kernel(x, Wq, scales, biases, ids, y, T, N, K, E, W4A16_KERNEL_AUTO, stream);
}

int w4a16_mm_id_kernel(const w4a16_bf16* x, const uint32_t* Wq, const w4a16_bf16* scales,
                       const w4a16_bf16* biases, const int32_t* ids, w4a16_bf16* y, int T, int N, int K, int E,
                       int kernel, void* stream) {
  if (env().fault == kFaultValidate) return fail(W4A16_ERR_SHAPE, "injected validation fault (W4A16_FAULT)");
  if (T < 0 || T > kMaxDim) return fail(W4A16_ERR_EXPERTS, "T = %d must be in 0..2^30", T);
  if (E <= 0 || E > 65535) return fail(W4A16_ERR_EXPERTS, "E = %d must be in 1..65535", E);
  if (int rc = check_nk(N, K)) return rc;
  w4a16_plan plan;
  if (int rc = resolve_kernel(kernel, N, K, &plan)) return rc;
  if (K % 512 && plan.kernel == W4A16_KERNEL_TC_TILE)
    return fail(W4A16_ERR_KERNEL, "w4a16_mm_id with K %% 512 != 0 runs the persistent routed mode (K = %d)", K);
  if (T == 0) return W4A16_OK;
  if (!x || !Wq || !scales || !biases || !ids || !y) return fail(W4A16_ERR_NULL, "null tensor pointer");
  if (misaligned(x, 16) || misaligned(Wq, 16)) return fail(W4A16_ERR_ALIGN, "x and Wq must be 16-byte aligned");
  if (misaligned(scales, 8) || misaligned(biases, 8) || misaligned(y, 2) || misaligned(ids, 4))
    return fail(W4A16_ERR_ALIGN, "scales/biases must be 8-byte, y 2-byte and ids 4-byte aligned");
  if (plan.kernel == W4A16_KERNEL_VANILLA && T > 65535)
    return fail(W4A16_ERR_SHAPE, "the vanilla control kernel takes at most 65535 tokens");
  if (env().fault == kFaultLaunch) return fail(W4A16_ERR_CUDA, "injected launch fault (W4A16_FAULT)");
  LaunchArgs a{};
  a.x = x; a.Wq = Wq; a.S = scales; a.B = biases; a.y = y;
  a.N = N; a.K = K; a.ids = ids; a.T = T; a.E = E;
  a.stream = static_cast<cudaStream_t>(stream);
  a.pdl = env().pdl;
  a.tc_path = plan.kernel == W4A16_KERNEL_TC_STREAM ? 1 : plan.kernel == W4A16_KERNEL_TC_TILE ? 2 : 0;
  if (int rc = flag_pointer(&a.flags)) return rc;
  cudaError_t e = cudaSuccess;
  switch (plan.kernel) {
    case W4A16_KERNEL_SIMT: e = launch_simt_id(a, plan); break;
    case W4A16_KERNEL_TC:
    case W4A16_KERNEL_TC_STREAM:
    case W4A16_KERNEL_TC_TILE: e = launch_tc_id(a, plan); break;
    case W4A16_KERNEL_VANILLA: e = launch_vanilla_id(a, plan); break;
    default: return fail(W4A16_ERR_KERNEL, "kernel %d cannot run", plan.kernel);
  }
  if (e != cudaSuccess) return cuda_fail(e, "w4a16_mm_id launch");
  return W4A16_OK;
}

int w4a16_unpack(const uint32_t* Wq, uint8_t* q, int N, int K, void* stream) {
  if (N <= 0 || N > kMaxDim) return fail(W4A16_ERR_SHAPE, "N = %d must be in 1..2^30", N);
  if (K <= 0 || K > kMaxDim || K % 8) return fail(W4A16_ERR_SHAPE, "K = %d must be a positive multiple of 8", K);
  if (!Wq || !q) return fail(W4A16_ERR_NULL, "null tensor pointer");
  if (misaligned(Wq, 4) || misaligned(q, 8)) return fail(W4A16_ERR_ALIGN, "Wq must be 4-byte and q 8-byte aligned");
  cudaError_t e = launch_unpack(Wq, q, N, K, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "w4a16_unpack launch");
}

int w4a16_dequant(const uint32_t* Wq, const w4a16_bf16* scales, const w4a16_bf16* biases, float* w, int N, int K,
                  void* stream) {
  if (int rc = check_nk(N, K)) return rc;
  if (!Wq || !scales || !biases || !w) return fail(W4A16_ERR_NULL, "null tensor pointer");
  if (misaligned(Wq, 4) || misaligned(scales, 2) || misaligned(biases, 2) || misaligned(w, 16))
    return fail(W4A16_ERR_ALIGN, "Wq 4-byte, scales/biases 2-byte and w 16-byte alignment required");
  cudaError_t e = launch_dequant(Wq, scales, biases, w, N, K, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "w4a16_dequant launch");
}

int w4a16_expand_groups(const w4a16_bf16* src, w4a16_bf16* dst, int N, int K, int group, void* stream) {
  if (int rc = check_nk(N, K)) return rc;
  if (group < kGroup || group % kGroup || group > 4096 || K % group)
    return fail(W4A16_ERR_SHAPE, "group = %d must be a multiple of 64 that divides K = %d", group, K);
  if (!src || !dst) return fail(W4A16_ERR_NULL, "null tensor pointer");
  if (misaligned(src, 2) || misaligned(dst, 2)) return fail(W4A16_ERR_ALIGN, "src and dst must be 2-byte aligned");
  cudaError_t e = launch_expand_groups(src, dst, N, K, group, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "w4a16_expand_groups launch");
}

int w4a16_embed(const uint32_t* Wq, const w4a16_bf16* scales, const w4a16_bf16* biases, const int32_t* ids,
                w4a16_bf16* out, int T, int N, int K, void* stream) {
  if (env().fault == kFaultValidate) return fail(W4A16_ERR_SHAPE, "injected validation fault (W4A16_FAULT)");
  if (T < 0 || T > 65535) return fail(W4A16_ERR_SHAPE, "T = %d must be in 0..65535", T);
  if (int rc = check_nk(N, K)) return rc;
  if (T == 0) return W4A16_OK;
  if (!Wq || !scales || !biases || !ids || !out) return fail(W4A16_ERR_NULL, "null tensor pointer");
  if (misaligned(Wq, 4) || misaligned(scales, 2) || misaligned(biases, 2) || misaligned(ids, 4) || misaligned(out, 16))
    return fail(W4A16_ERR_ALIGN, "Wq and ids 4-byte, scales/biases 2-byte and out 16-byte alignment required");
  if (env().fault == kFaultLaunch) return fail(W4A16_ERR_CUDA, "injected launch fault (W4A16_FAULT)");
  int* flags = nullptr;
  if (int rc = flag_pointer(&flags)) return rc;
  cudaError_t e = launch_embed(Wq, scales, biases, ids, out, T, N, K, flags, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "w4a16_embed launch");
}

int w4a16_mm_noalloc(const w4a16_bf16* x, const uint32_t* Wq, const w4a16_bf16* scales, const w4a16_bf16* biases,
                     w4a16_bf16* y, int M, int N, int K, void* stream) {
  if (int rc = validate_mm(x, Wq, scales, biases, y, M, N, K)) return rc;
  if (!tc_supported(N, K))
    return fail(W4A16_ERR_KERNEL, "K = %d is past the tensor-core kernels' K %% 512 != 0 range", K);
  if (!tc_noalloc_fits(N, K))
    return fail(W4A16_ERR_SHAPE, "N = %d, K = %d needs more than the %zu-byte fixed scratch of w4a16_mm_noalloc", N, K,
                tc_noalloc_scratch_bytes());
  if (M == 0) return W4A16_OK;
  LaunchArgs a{};
  a.x = x; a.Wq = Wq; a.S = scales; a.B = biases; a.y = y;
  a.N = N; a.K = K;
  a.stream = static_cast<cudaStream_t>(stream);
  a.pdl = env().pdl;
  if (int rc = flag_pointer(&a.flags)) return rc;
  for (int row0 = 0; row0 < M; row0 += kMaxChunk) {
    a.row0 = row0;
    a.M = (M - row0 < kMaxChunk) ? M - row0 : kMaxChunk;
    cudaError_t e = launch_tc_noalloc(a);
    if (e == cudaErrorInvalidValue) return fail(W4A16_ERR_SHAPE, "shape exceeds the fixed scratch of w4a16_mm_noalloc");
    if (e != cudaSuccess) return cuda_fail(e, "w4a16_mm_noalloc launch");
  }
  return W4A16_OK;
}

int w4a16_mm_argmax(const w4a16_bf16* x, const uint32_t* Wq, const w4a16_bf16* scales, const w4a16_bf16* biases,
                    int32_t* idx, w4a16_bf16* val, int M, int N, int K, void* workspace, size_t workspace_bytes,
                    void* stream) {
  if (env().fault == kFaultValidate) return fail(W4A16_ERR_SHAPE, "injected validation fault (W4A16_FAULT)");
  if (int rc = validate_mm(x, Wq, scales, biases, idx, M, N, K)) return rc;
  if (M == 0) return W4A16_OK;
  if (!workspace) return fail(W4A16_ERR_NULL, "w4a16_mm_argmax needs a workspace (w4a16_workspace_bytes)");
  if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
  if (misaligned(idx, 4) || misaligned(val, 2)) return fail(W4A16_ERR_ALIGN, "idx must be 4-byte and val 2-byte aligned");
  if (K % 512)
    return fail(W4A16_ERR_KERNEL, "w4a16_mm_argmax runs the tensor-core kernel, which needs K %% 512 == 0 (K = %d)", K);
  if (env().fault == kFaultLaunch) return fail(W4A16_ERR_CUDA, "injected launch fault (W4A16_FAULT)");
  LaunchArgs a{};
  a.x = x; a.Wq = Wq; a.S = scales; a.B = biases; a.y = nullptr;
  a.N = N; a.K = K;
  a.stream = static_cast<cudaStream_t>(stream);
  a.pdl = env().pdl;
  a.tc_path = 1;
  a.ws = workspace;
  a.ws_bytes = workspace_bytes;
  if (int rc = flag_pointer(&a.flags)) return rc;
  for (int row0 = 0; row0 < M; row0 += kMaxChunk) {
    a.row0 = row0;
    a.M = (M - row0 < kMaxChunk) ? M - row0 : kMaxChunk;
    cudaError_t e = launch_tc_argmax(a, idx, val);
    if (e == cudaErrorInvalidValue) return fail(W4A16_ERR_SHAPE, "N = %d, K = %d exceeds the persistent kernel's workspace", N, K);
    if (e != cudaSuccess) return cuda_fail(e, "w4a16_mm_argmax launch");
  }
  return W4A16_OK;
}

int w4a16_mm_group(const w4a16_mm_item* items, int count, int M, int K, void* stream) {
  if (env().fault == kFaultValidate) return fail(W4A16_ERR_SHAPE, "injected validation fault (W4A16_FAULT)");
  if (count < 1 || count > W4A16_MAX_GROUP)
    return fail(W4A16_ERR_SHAPE, "count = %d must be in 1..%d", count, W4A16_MAX_GROUP);
  if (!items) return fail(W4A16_ERR_NULL, "null item array");
  int Ns[W4A16_MAX_GROUP];
  for (int i = 0; i < count; ++i) {
    const w4a16_mm_item& it = items[i];
    if (int rc = validate_mm(it.x, it.Wq, it.scales, it.biases, it.y, M, it.N, K)) return rc;
    Ns[i] = it.N;
  }
  if (M == 0) return W4A16_OK;
  if (env().force_kernel != W4A16_KERNEL_AUTO || !tc_group_supported(Ns, count, K)) {
    for (int i = 0; i < count; ++i) {
      const w4a16_mm_item& it = items[i];
      if (int rc = run_mm(it.x, it.Wq, it.scales, it.biases, it.y, M, it.N, K, W4A16_KERNEL_AUTO, stream)) return rc;
    }
    return W4A16_OK;
  }
  if (env().fault == kFaultLaunch) return fail(W4A16_ERR_CUDA, "injected launch fault (W4A16_FAULT)");
  int* flags = nullptr;
  if (int rc = flag_pointer(&flags)) return rc;
  GroupItem g[W4A16_MAX_GROUP];
  for (int i = 0; i < count; ++i)
    g[i] = GroupItem{items[i].x, items[i].Wq, items[i].scales, items[i].biases, items[i].y, items[i].N};
  cudaError_t e = launch_tc_group(g, count, M, 0, K, env().pdl, flags, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "w4a16_mm_group launch");
  return W4A16_OK;
}

int w4a16_get_plan(int N, int K, int kernel, w4a16_plan* out) {
  if (!out) return fail(W4A16_ERR_NULL, "null plan pointer");
  if (int rc = check_nk(N, K)) return rc;
  return resolve_kernel(kernel, N, K, out);
}

int w4a16_device_status(void* stream, int* flags) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  int* p = nullptr;
  if (int rc = flag_pointer(&p)) return rc;
  int v = 0;
  e = cudaMemcpy(&v, p, sizeof v, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "read device flags");
  if (flags) *flags = v;
  if (v) {
    const int zero = 0;
    e = cudaMemcpy(p, &zero, sizeof zero, cudaMemcpyHostToDevice);
    if (e != cudaSuccess) return cuda_fail(e, "clear device flags");
    return fail(W4A16_ERR_DEVICE, "a kernel reported bad input (flags 0x%x)", v);
  }
  return W4A16_OK;
}

// ---- STQ1_0 (include/stq1.h) ----------------------------------------------------

size_t stq1_packed_bytes(int N, int K) { return stq1_packed_size(N, K); }

int stq1_get_plan(int N, int K, stq1_plan* out) {
  if (!out) return fail(W4A16_ERR_NULL, "null plan pointer");
  if (!stq1_shape_ok(N, K))
    return fail(W4A16_ERR_SHAPE, "N = %d must be >= 1 and K = %d a multiple of 256 in 256..%d", N, K, STQ1_MAX_K);
  Stq1Plan p;
  stq1_make_plan(N, K, &p);
  out->ksplit = p.ks;
  out->blocks_per_slice = p.bps;
  out->rows_per_pass = p.xcap;
  return W4A16_OK;
}

int stq1_pack(const uint8_t* blocks, uint8_t* packed, int N, int K, void* stream) {
  if (!stq1_shape_ok(N, K))
    return fail(W4A16_ERR_SHAPE, "N = %d must be >= 1 and K = %d a multiple of 256 in 256..%d", N, K, STQ1_MAX_K);
  if (!blocks || !packed) return fail(W4A16_ERR_NULL, "null tensor pointer");
  if (misaligned(blocks, 2) || misaligned(packed, 16))
    return fail(W4A16_ERR_ALIGN, "blocks must be 2-byte and packed 16-byte aligned");
  cudaError_t e = launch_stq1_pack(blocks, packed, N, K, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "stq1_pack launch");
}

int stq1_mm(const float* x, const uint8_t* packed, float* y, int M, int N, int K, void* stream) {
  if (env().fault == kFaultValidate) return fail(W4A16_ERR_SHAPE, "injected validation fault (W4A16_FAULT)");
  if (M < 0 || M > kMaxDim) return fail(W4A16_ERR_SHAPE, "M = %d must be in 0..2^30", M);
  if (!stq1_shape_ok(N, K) || N > kMaxDim)
    return fail(W4A16_ERR_SHAPE, "N = %d must be in 1..2^30 and K = %d a multiple of 256 in 256..%d", N, K,
                STQ1_MAX_K);
  if (M == 0) return W4A16_OK;
  if (!x || !packed || !y) return fail(W4A16_ERR_NULL, "null tensor pointer");
  if (misaligned(x, 16) || misaligned(packed, 16) || misaligned(y, 4))
    return fail(W4A16_ERR_ALIGN, "x and packed must be 16-byte and y 4-byte aligned");
  if (env().fault == kFaultLaunch) return fail(W4A16_ERR_CUDA, "injected launch fault (W4A16_FAULT)");
  int* flags = nullptr;
  if (int rc = flag_pointer(&flags)) return rc;
  Stq1Plan pl;
  stq1_make_plan(N, K, &pl);
  for (int row0 = 0; row0 < M; row0 += pl.xcap) {
    const int rows = M - row0 < pl.xcap ? M - row0 : pl.xcap;
    cudaError_t e =
        launch_stq1_mm(x, packed, y, rows, row0, N, K, flags, env().pdl, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "stq1_mm launch");
  }
  return W4A16_OK;
}

int stq1_mm_id(const float* x, const uint8_t* packed, const int32_t* ids, float* y, int T, int N, int K, int E,
               void* stream) {
  if (env().fault == kFaultValidate) return fail(W4A16_ERR_SHAPE, "injected validation fault (W4A16_FAULT)");
  if (T < 0 || T > kMaxDim) return fail(W4A16_ERR_EXPERTS, "T = %d must be in 0..2^30", T);
  if (E <= 0 || E > 65535) return fail(W4A16_ERR_EXPERTS, "E = %d must be in 1..65535", E);
  if (!stq1_shape_ok(N, K) || N > kMaxDim)
    return fail(W4A16_ERR_SHAPE, "N = %d must be in 1..2^30 and K = %d a multiple of 256 in 256..%d", N, K,
                STQ1_MAX_K);
  if (T == 0) return W4A16_OK;
  if (!x || !packed || !ids || !y) return fail(W4A16_ERR_NULL, "null tensor pointer");
  if (misaligned(x, 16) || misaligned(packed, 16) || misaligned(y, 4) || misaligned(ids, 4))
    return fail(W4A16_ERR_ALIGN, "x and packed must be 16-byte, y and ids 4-byte aligned");
  if (env().fault == kFaultLaunch) return fail(W4A16_ERR_CUDA, "injected launch fault (W4A16_FAULT)");
  int* flags = nullptr;
  if (int rc = flag_pointer(&flags)) return rc;
  cudaError_t e =
      launch_stq1_mm_id(x, packed, ids, y, T, N, K, E, flags, env().pdl, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "stq1_mm_id launch");
}

int stq1_get_rows(const uint8_t* packed, const int32_t* ids, float* out, int T, int N, int K, void* stream) {
  if (T < 0 || T > kMaxDim) return fail(W4A16_ERR_SHAPE, "T = %d must be in 0..2^30", T);
  if (!stq1_shape_ok(N, K) || N > kMaxDim)
    return fail(W4A16_ERR_SHAPE, "N = %d must be in 1..2^30 and K = %d a multiple of 256 in 256..%d", N, K,
                STQ1_MAX_K);
  if (T == 0) return W4A16_OK;
  if (!packed || !ids || !out) return fail(W4A16_ERR_NULL, "null tensor pointer");
  if (misaligned(packed, 16) || misaligned(ids, 4) || misaligned(out, 4))
    return fail(W4A16_ERR_ALIGN, "packed must be 16-byte, ids and out 4-byte aligned");
  int* flags = nullptr;
  if (int rc = flag_pointer(&flags)) return rc;
  cudaError_t e = launch_stq1_get_rows(packed, ids, out, T, N, K, flags, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "stq1_get_rows launch");
}

// ---- paged key/value cache in 8 bits ----------------------------------------------

namespace {

bool kv_block_ok(int block) { return block == 16 || block == 32 || block == 64 || block == 128; }

int check_kv_cache(const w4a16_kv_cache* c) {
  if (!c) return fail(W4A16_ERR_NULL, "null cache");
  if (!kv_block_ok(c->block)) return fail(W4A16_ERR_SHAPE, "block = %d must be 16, 32, 64 or 128", c->block);
  if (c->dim != 64 && c->dim != 128 && c->dim != 256)
    return fail(W4A16_ERR_SHAPE, "dim = %d must be 64, 128 or 256", c->dim);
  if (c->heads < 1 || c->heads > 65535) return fail(W4A16_ERR_SHAPE, "heads = %d must be in 1..65535", c->heads);
  if (c->blocks < 1 || (int64_t)c->blocks * c->heads * c->block > INT32_MAX)
    return fail(W4A16_ERR_SHAPE, "blocks = %d: blocks * heads * block must be in 1..2^31 - 1", c->blocks);
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return fail(W4A16_ERR_NULL, "null cache pointer");
  if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->k_scale, 4) || misaligned(c->v_scale, 4))
    return fail(W4A16_ERR_ALIGN, "cache codes must be 16-byte and scales 4-byte aligned");
  return W4A16_OK;
}

}  // namespace

int w4a16_kv_plan(const int32_t* cached, const int32_t* fresh, int32_t* table, const int32_t* free_blocks,
                  const int32_t* head, int32_t* cu, int32_t* lens, int32_t* slots, int32_t* positions,
                  int32_t* head_out, int B, int T, int block, int max_blocks, int n_free, void* stream) {
  if (env().fault == kFaultValidate) return fail(W4A16_ERR_SHAPE, "injected validation fault (W4A16_FAULT)");
  if (B < 0 || B >= kMaxDim || T < 0 || T >= kMaxDim)
    return fail(W4A16_ERR_SHAPE, "B = %d and T = %d must be in 0..2^30 - 1", B, T);
  if (!kv_block_ok(block)) return fail(W4A16_ERR_SHAPE, "block = %d must be 16, 32, 64 or 128", block);
  if (max_blocks < 1 || n_free < 0)
    return fail(W4A16_ERR_SHAPE, "max_blocks = %d must be at least 1 and n_free = %d not negative", max_blocks, n_free);
  if (!cu || !head_out || (B > 0 && (!cached || !fresh || !table || !lens)) || (T > 0 && (!slots || !positions)) ||
      (n_free > 0 && !free_blocks))
    return fail(W4A16_ERR_NULL, "null array");
  if (head == head_out) return fail(W4A16_ERR_SHAPE, "head_out must not be head");
  const void* all[] = {cached, fresh, table, free_blocks, head, cu, lens, slots, positions, head_out};
  for (const void* q : all)
    if (misaligned(q, 4)) return fail(W4A16_ERR_ALIGN, "arrays must be 4-byte aligned");
  if (env().fault == kFaultLaunch) return fail(W4A16_ERR_CUDA, "injected launch fault (W4A16_FAULT)");
  KvPlanArgs a{cached, fresh, table, free_blocks, head, cu, lens, slots, positions, head_out,
               B, T, block, max_blocks, n_free, nullptr};
  // (the CTAs read all of the inputs while others write outputs)
  const struct {
    const void* p;
    int64_t n;
    const char* name;
  } arrays[] = {{cached, B, "cached"}, {fresh, B, "fresh"}, {free_blocks, n_free, "free_blocks"}, {head, head ? 1 : 0, "head"},
                {table, (int64_t)B * max_blocks, "table"}, {cu, (int64_t)B + 1, "cu"}, {lens, B, "lens"},
                {slots, T, "slots"}, {positions, T, "positions"}, {head_out, 1, "head_out"}};
  for (int i = 4; i < 10; ++i)  // what the call writes
    for (int j = 0; j < i; ++j) {
      const auto &x = arrays[i], &y = arrays[j];
      const uintptr_t at = reinterpret_cast<uintptr_t>(x.p), bt = reinterpret_cast<uintptr_t>(y.p);
      const bool in_place = i == 6 && j == 0 && lens == cached;
      if (!in_place && x.n > 0 && y.n > 0 && at < bt + 4 * (uintptr_t)y.n && bt < at + 4 * (uintptr_t)x.n)
        return fail(W4A16_ERR_SHAPE, "%s and %s overlap (only lens may be cached itself)", x.name, y.name);
    }
  if (int rc = flag_pointer(&a.flags)) return rc;
  cudaError_t e = launch_kv_plan(a, env().pdl, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "w4a16_kv_plan launch");
}

int w4a16_kv_append(const w4a16_bf16* k, int64_t k_stride, const w4a16_bf16* v, int64_t v_stride,
                    const int32_t* slots, const w4a16_kv_cache* cache, int T, void* stream) {
  if (env().fault == kFaultValidate) return fail(W4A16_ERR_SHAPE, "injected validation fault (W4A16_FAULT)");
  if (int rc = check_kv_cache(cache)) return rc;
  if (T < 0 || T >= kMaxDim) return fail(W4A16_ERR_SHAPE, "T = %d must be in 0..2^30 - 1", T);
  if (T == 0) return W4A16_OK;
  if (!k || !v || !slots) return fail(W4A16_ERR_NULL, "null tensor pointer");
  const int64_t row = (int64_t)cache->heads * cache->dim;
  if (T > 1 && (k_stride < row || v_stride < row))
    return fail(W4A16_ERR_SHAPE, "token strides must be at least heads * dim = %lld elements", (long long)row);
  if (misaligned(k, 16) || misaligned(v, 16) || k_stride % 8 || v_stride % 8 || misaligned(slots, 4))
    return fail(W4A16_ERR_ALIGN, "k and v rows must be 16-byte and slots 4-byte aligned");
  if (env().fault == kFaultLaunch) return fail(W4A16_ERR_CUDA, "injected launch fault (W4A16_FAULT)");
  KvAppendArgs a{k, v, k_stride, v_stride, slots, *cache, T, nullptr};
  if (int rc = flag_pointer(&a.flags)) return rc;
  cudaError_t e = launch_kv_append(a, env().pdl, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "w4a16_kv_append launch");
}

size_t w4a16_kv_attention_workspace_bytes(int B, int T, int q_heads, int heads, int dim, int max_new, int max_len,
                                          int window) {
  if (B < 1 || T < 1 || heads < 1 || q_heads < heads || q_heads % heads || q_heads / heads > W4A16_KV_MAX_GROUP ||
      max_new < 1 || max_len < 1 || window < 0 ||
      (dim != 64 && dim != 128 && dim != 256))
    return 0;
  return kv_attention_workspace(B, T, q_heads, heads, dim, max_new, max_len, window);
}

int w4a16_kv_attention(const w4a16_bf16* q, int64_t q_stride, const w4a16_kv_cache* cache, const int32_t* table,
                       const int32_t* cu, const int32_t* lens, w4a16_bf16* out, int B, int T, int q_heads,
                       int max_blocks, int max_new, int max_len, int window, float scale, void* workspace,
                       size_t workspace_bytes, int32_t* counters, void* stream) {
  if (env().fault == kFaultValidate) return fail(W4A16_ERR_SHAPE, "injected validation fault (W4A16_FAULT)");
  if (int rc = check_kv_cache(cache)) return rc;
  if (B < 0 || B >= kMaxDim || T < 0 || T >= kMaxDim)
    return fail(W4A16_ERR_SHAPE, "B = %d and T = %d must be in 0..2^30 - 1", B, T);
  if (T > 0 && B == 0) return fail(W4A16_ERR_SHAPE, "T = %d tokens of no request", T);
  if (q_heads < cache->heads || q_heads % cache->heads || q_heads / cache->heads > W4A16_KV_MAX_GROUP)
    return fail(W4A16_ERR_SHAPE, "q_heads = %d must be 1..%d times the cache's %d heads", q_heads, W4A16_KV_MAX_GROUP,
                cache->heads);
  if (max_blocks < 1 || max_new < 1 || max_len < 1 || window < 0 ||
      (int64_t)max_len > (int64_t)max_blocks * cache->block)
    return fail(W4A16_ERR_SHAPE,
                "max_blocks = %d and max_new = %d must be positive, window = %d not negative, max_len = %d in "
                "1..max_blocks * block", max_blocks, max_new, window, max_len);
  if (!(scale > 0.f) || scale > 3.0e38f) return fail(W4A16_ERR_SHAPE, "scale must be a positive number");
  if (T == 0) return W4A16_OK;
  if (!q || !table || !cu || !lens || !out) return fail(W4A16_ERR_NULL, "null tensor pointer");
  if (T > 1 && q_stride < (int64_t)q_heads * cache->dim)
    return fail(W4A16_ERR_SHAPE, "q_stride must be at least q_heads * dim = %lld elements",
                (long long)q_heads * cache->dim);
  if (misaligned(q, 16) || q_stride % 8 || misaligned(out, 16) || misaligned(table, 4) || misaligned(cu, 4) ||
      misaligned(lens, 4))
    return fail(W4A16_ERR_ALIGN, "q rows and out must be 16-byte, table, cu and lens 4-byte aligned");
  const size_t need = kv_attention_workspace(B, T, q_heads, cache->heads, cache->dim, max_new, max_len, window);
  if (need == 0)
    return fail(W4A16_ERR_SHAPE, "T = %d rows over max_len = %d tokens: too many for one call (2^31 tiles or group rows)",
                T, max_len);
  if (!workspace || !counters)
    return fail(W4A16_ERR_NULL, "w4a16_kv_attention needs a workspace of %zu bytes, and counters", need);
  if (misaligned(workspace, 256) || misaligned(counters, 4))
    return fail(W4A16_ERR_ALIGN, "the workspace must be 256-byte and counters 4-byte aligned");
  if (workspace_bytes < need)
    return fail(W4A16_ERR_SHAPE, "a workspace of %zu bytes is too small (%zu)", workspace_bytes, need);
  if (env().fault == kFaultLaunch) return fail(W4A16_ERR_CUDA, "injected launch fault (W4A16_FAULT)");
  KvAttentionArgs a{q, q_stride, *cache, table, cu, lens, out, B, T, q_heads, max_blocks, max_new, max_len, window,
                    scale, workspace, counters, nullptr, env().fault == kFaultWait};
  if (int rc = flag_pointer(&a.flags)) return rc;
  std::lock_guard<std::mutex> turn(turn_of(stream));
  cudaError_t e = launch_kv_attention(a, env().pdl, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "w4a16_kv_attention launch");
}

// ---- microscaled 4-bit floating point ------------------------------------------------

namespace {

constexpr int kFp4MaxExperts = 4096, kFp4MaxTop = 1024;

int check_fp4_shape(int rows, int K, int experts, int format) {
  if (format != W4A16_FP4_NV && format != W4A16_FP4_MX)
    return fail(W4A16_ERR_SHAPE, "format = %d must be W4A16_FP4_NV or W4A16_FP4_MX", format);
  if (K <= 0 || K > kMaxDim || K % 32) return fail(W4A16_ERR_SHAPE, "K = %d must be a positive multiple of 32", K);
  if (experts < 1 || experts > kFp4MaxExperts)
    return fail(W4A16_ERR_EXPERTS, "experts = %d must be in 1..%d", experts, kFp4MaxExperts);
  if (rows < 0 || (int64_t)rows * experts > kMaxDim)
    return fail(W4A16_ERR_SHAPE, "rows = %d: experts * rows must be in 0..2^30", rows);
  return W4A16_OK;
}

// A matrix with rows, its pointers there and aligned.
int check_fp4(const w4a16_fp4* m, const char* name) {
  if (!m) return fail(W4A16_ERR_NULL, "null %s", name);
  if (int rc = check_fp4_shape(m->rows, m->K, m->experts, m->format)) return rc;
  if (m->rows == 0) return W4A16_OK;
  if (!m->codes || !m->scales) return fail(W4A16_ERR_NULL, "%s: null codes or scales", name);
  if (misaligned(m->codes, 16) || misaligned(m->scales, 16) || misaligned(m->row_scale, 4))
    return fail(W4A16_ERR_ALIGN, "%s: codes and scales must be 16-byte and row_scale 4-byte aligned", name);
  return W4A16_OK;
}

int check_fp4_rows(const void* x, int64_t x_stride, int64_t rows, int K) {
  if (!x) return fail(W4A16_ERR_NULL, "null tensor pointer");
  if (rows > 1 && x_stride < K) return fail(W4A16_ERR_SHAPE, "x_stride must be at least K = %d elements", K);
  if (misaligned(x, 16) || x_stride % 8) return fail(W4A16_ERR_ALIGN, "rows of x must be 16-byte aligned");
  return W4A16_OK;
}

// CTAs write the one while others read the other.
bool fp4_overlap(const void* x, int64_t x_bytes, const void* y, int64_t y_bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  return a < b + (uintptr_t)y_bytes && b < a + (uintptr_t)x_bytes;
}
bool fp4_overlaps(const w4a16_fp4& m, const void* y, int64_t y_bytes) {
  return fp4_overlap(m.codes, (int64_t)m.experts * m.rows * (m.K / 2), y, y_bytes) ||
         fp4_overlap(m.scales, m.experts * fp4_scale_bytes(m.rows, m.K, m.format), y, y_bytes) ||
         (m.row_scale && fp4_overlap(m.row_scale, 4LL * m.experts * m.rows, y, y_bytes));
}
int64_t fp4_x_bytes(int64_t x_stride, int64_t rows, int K) { return 2 * ((rows > 1 ? (rows - 1) * x_stride : 0) + K); }
int64_t fp4_y_bytes(const w4a16_fp4* w, int64_t rows, int act) { return 2 * rows * (act == W4A16_FP4_LINEAR ? w->rows : w->rows / 2); }
int check_fp4_apart(const void* x, int64_t x_bytes, const w4a16_fp4* w, const void* y, int64_t y_bytes) {
  if (fp4_overlap(x, x_bytes, y, y_bytes)) return fail(W4A16_ERR_SHAPE, "y overlaps x");
  return fp4_overlaps(*w, y, y_bytes) ? fail(W4A16_ERR_SHAPE, "y overlaps w") : W4A16_OK;
}

int check_fp4_act(const w4a16_fp4* w, int act) {
  if (act != W4A16_FP4_LINEAR && act != W4A16_FP4_SILU && act != W4A16_FP4_GELU)
    return fail(W4A16_ERR_KERNEL, "unknown activation %d", act);
  if (w->rows < 1) return fail(W4A16_ERR_SHAPE, "a weight matrix needs rows");
  if (act != W4A16_FP4_LINEAR && w->rows % 2)
    return fail(W4A16_ERR_SHAPE, "rows = %d: gate and up rows come in pairs", w->rows);
  return W4A16_OK;
}

size_t up256(int64_t n) { return (size_t)((n + 255) / 256 * 256); }

// Workspace of quantised rows: codes, scales, row factors.
struct Fp4Space {
  size_t codes, scales, factor, place, row, tiles, count, total;
};
Fp4Space fp4_space(int64_t places, int64_t rows, int64_t tiles, int K, int format) {
  Fp4Space s = {};
  s.scales = up256(places * (K / 2));
  s.factor = s.scales + up256((places + kFp4Rows - 1) / kFp4Rows * fp4_atoms(K, format) * kFp4Atom);
  s.place = s.factor + up256(places * 4);
  if (tiles == 0) {
    s.total = s.place;
    return s;
  }
  s.row = s.place + up256(rows * 4);
  s.tiles = s.row + up256(places * 4);
  s.count = s.tiles + up256(tiles * (int64_t)sizeof(Fp4Tile));
  s.total = s.count + 256;
  return s;
}

// Routed: rows of an activation tile, and the most tiles that there can be.  Twice an expert's mean share up to 16 rows;
// then 32 rows, of which the large experts take two tiles (their weights come from L2 the second time), as a tile of 64
// has fewer slots in its ring; and from some 40 rows on the pair kernel's tile, however empty.  K = 2048, N = 1536, 64
// experts, mean rows: us with 32 / 64 / 256: 20 24.1 / 28.0 / 27.9; 31 27.8 / 31.9 / 30.9; 40 33.0 / 34.8 / 34.5; 50 37.3 /
// 39.0 / 35.9; 63 (16 experts) 19.5 / 20.9 / 20.0; 250 (16) - / 40 (of 128) / 26.
int fp4_id_tile(int64_t rows, int experts) {
  const int64_t mean = (rows + experts - 1) / experts;
  return mean > 40 ? 256 : mean > 8 ? 32 : 16;
}
int fp4_id_span(int64_t rows, int experts) { return fp4_id_tile(rows, experts) > 128 ? 256 : 128; }
int64_t fp4_id_tiles(int64_t rows, int experts) {
  // an expert with rows wastes less than one tile
  return (rows < experts ? rows : experts) + rows / fp4_id_tile(rows, experts);
}

// The workspace holds what the call's launches hand on (for routed calls, places of rows too).
int check_fp4_space(const void* ws, size_t bytes, size_t need, const void* x, int64_t x_bytes, const void* y, int64_t y_bytes) {
  if (!ws) return fail(W4A16_ERR_NULL, "the call needs a workspace of %zu bytes", need);
  if (misaligned(ws, 256)) return fail(W4A16_ERR_ALIGN, "the workspace must be 256-byte aligned");
  if (bytes < need) return fail(W4A16_ERR_SHAPE, "a workspace of %zu bytes is too small (%zu)", bytes, need);
  if (fp4_overlap(ws, (int64_t)need, x, x_bytes)) return fail(W4A16_ERR_SHAPE, "x overlaps the workspace");
  return fp4_overlap(ws, (int64_t)need, y, y_bytes) ? fail(W4A16_ERR_SHAPE, "y overlaps the workspace") : W4A16_OK;
}

}  // namespace

size_t w4a16_fp4_scale_bytes(int rows, int K, int format) {
  if (check_fp4_shape(rows, K, 1, format)) return 0;
  return (size_t)fp4_scale_bytes(rows, K, format);
}

int w4a16_fp4_quant(const w4a16_bf16* x, int64_t x_stride, const w4a16_fp4* out, void* stream) {
  if (env().fault == kFaultValidate) return fail(W4A16_ERR_SHAPE, "injected validation fault (W4A16_FAULT)");
  if (int rc = check_fp4(out, "out")) return rc;
  if (out->rows == 0) return W4A16_OK;
  if (out->format == W4A16_FP4_NV && !out->row_scale) return fail(W4A16_ERR_NULL, "out: nv needs row_scale");
  const int rows = out->rows * out->experts;
  if (int rc = check_fp4_rows(x, x_stride, rows, out->K)) return rc;
  if (fp4_overlaps(*out, x, fp4_x_bytes(x_stride, rows, out->K))) return fail(W4A16_ERR_SHAPE, "out overlaps x");
  if (env().fault == kFaultLaunch) return fail(W4A16_ERR_CUDA, "injected launch fault (W4A16_FAULT)");
  Fp4QuantArgs a{x, x_stride, out->codes, out->scales, out->row_scale, rows, out->K, out->rows, out->format};
  cudaError_t e = launch_fp4_quant(a, env().pdl, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "w4a16_fp4_quant launch");
}

int w4a16_fp4_dequant(const w4a16_fp4* w, w4a16_bf16* y, void* stream) {
  if (env().fault == kFaultValidate) return fail(W4A16_ERR_SHAPE, "injected validation fault (W4A16_FAULT)");
  if (int rc = check_fp4(w, "w")) return rc;
  if (w->rows == 0) return W4A16_OK;
  if (!y) return fail(W4A16_ERR_NULL, "null tensor pointer");
  if (misaligned(y, 16)) return fail(W4A16_ERR_ALIGN, "y must be 16-byte aligned");
  if (fp4_overlaps(*w, y, 2LL * w->experts * w->rows * w->K)) return fail(W4A16_ERR_SHAPE, "y overlaps w");
  if (env().fault == kFaultLaunch) return fail(W4A16_ERR_CUDA, "injected launch fault (W4A16_FAULT)");
  cudaError_t e = launch_fp4_dequant(*w, y, env().pdl, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "w4a16_fp4_dequant launch");
}

size_t w4a16_fp4_mm_workspace_bytes(int M, int K, int format) {
  if (check_fp4_shape(M, K, 1, format)) return 0;
  return fp4_space(M, M, 0, K, format).total;
}

int w4a16_fp4_mm(const w4a16_bf16* x, int64_t x_stride, const w4a16_fp4* w, w4a16_bf16* y, int M, int act,
                 void* workspace, size_t workspace_bytes, void* stream) {
  if (env().fault == kFaultValidate) return fail(W4A16_ERR_SHAPE, "injected validation fault (W4A16_FAULT)");
  if (int rc = check_fp4(w, "w")) return rc;
  if (int rc = check_fp4_act(w, act)) return rc;
  if (w->experts != 1) return fail(W4A16_ERR_EXPERTS, "experts = %d: w4a16_fp4_mm_id takes stacked experts", w->experts);
  if (M < 0 || M > kMaxDim) return fail(W4A16_ERR_SHAPE, "M = %d must be in 0..2^30", M);
  if (M == 0) return W4A16_OK;
  if (int rc = check_fp4_rows(x, x_stride, M, w->K)) return rc;
  if (!y) return fail(W4A16_ERR_NULL, "null tensor pointer");
  if (misaligned(y, 2)) return fail(W4A16_ERR_ALIGN, "y must be 2-byte aligned");
  const int64_t x_bytes = fp4_x_bytes(x_stride, M, w->K), y_bytes = fp4_y_bytes(w, M, act);
  if (int rc = check_fp4_apart(x, x_bytes, w, y, y_bytes)) return rc;
  const Fp4Space sp = fp4_space(M, M, 0, w->K, w->format);
  if (int rc = check_fp4_space(workspace, workspace_bytes, sp.total, x, x_bytes, y, y_bytes)) return rc;
  if (env().fault == kFaultLaunch) return fail(W4A16_ERR_CUDA, "injected launch fault (W4A16_FAULT)");
  int* flags = nullptr;
  if (int rc = flag_pointer(&flags)) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* factor = w->format == W4A16_FP4_NV ? reinterpret_cast<float*>(ws + sp.factor) : nullptr;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  Fp4MmArgs a = {};
  std::unique_lock<std::mutex> turn(turn_of(stream), std::defer_lock);
  if (fp4_mm_fuses(*w, M)) {
    a.x = x;
    a.x_stride = x_stride;
  } else {
    turn.lock();
    Fp4QuantArgs q{x, x_stride, ws, ws + sp.scales, factor, M, w->K, M, w->format};
    if (cudaError_t e = launch_fp4_quant(q, env().pdl, s)) return cuda_fail(e, "w4a16_fp4_mm launch");
  }
  a.xc = ws;
  a.xs = ws + sp.scales;
  a.xf = factor;
  a.x_rows = M;
  a.w = *w;
  a.y = y;
  a.M = M;
  a.act = act;
  a.early = true;
  a.flags = flags;
  a.fault_wait = env().fault == kFaultWait;
  cudaError_t e = launch_fp4_mm(a, env().pdl, s);
  return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "w4a16_fp4_mm launch");
}

int w4a16_fp4_mm_q(const w4a16_fp4* x, const w4a16_fp4* w, w4a16_bf16* y, int act, void* stream) {
  if (env().fault == kFaultValidate) return fail(W4A16_ERR_SHAPE, "injected validation fault (W4A16_FAULT)");
  if (int rc = check_fp4(x, "x")) return rc;
  if (int rc = check_fp4(w, "w")) return rc;
  if (int rc = check_fp4_act(w, act)) return rc;
  if (x->experts != 1 || w->experts != 1)
    return fail(W4A16_ERR_EXPERTS, "experts = %d and %d: w4a16_fp4_mm_id takes stacked experts", x->experts, w->experts);
  if (x->K != w->K || x->format != w->format)
    return fail(W4A16_ERR_SHAPE, "x has K = %d and format %d, w K = %d and format %d", x->K, x->format, w->K, w->format);
  if (x->rows == 0) return W4A16_OK;
  if (!y) return fail(W4A16_ERR_NULL, "null tensor pointer");
  if (misaligned(y, 2)) return fail(W4A16_ERR_ALIGN, "y must be 2-byte aligned");
  const int64_t y_bytes = fp4_y_bytes(w, x->rows, act);
  if (fp4_overlaps(*x, y, y_bytes) || fp4_overlaps(*w, y, y_bytes)) return fail(W4A16_ERR_SHAPE, "y overlaps x or w");
  if (env().fault == kFaultLaunch) return fail(W4A16_ERR_CUDA, "injected launch fault (W4A16_FAULT)");
  Fp4MmArgs a = {};
  a.xc = x->codes;
  a.xs = x->scales;
  a.xf = x->row_scale;
  a.x_rows = x->rows;
  a.w = *w;
  a.y = y;
  a.M = x->rows;
  a.act = act;
  if (int rc = flag_pointer(&a.flags)) return rc;
  a.fault_wait = env().fault == kFaultWait;
  cudaError_t e = launch_fp4_mm(a, env().pdl, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "w4a16_fp4_mm_q launch");
}

size_t w4a16_fp4_mm_id_workspace_bytes(int T, int top, int K, int experts, int format) {
  if (check_fp4_shape(0, K, experts, format) || T < 0 || top < 1 || top > kFp4MaxTop || (int64_t)T * top > kMaxDim) return 0;
  const int64_t rows = (int64_t)T * top, tiles = fp4_id_tiles(rows, experts);
  return rows ? fp4_space(tiles * fp4_id_span(rows, experts), rows, tiles, K, format).total : 256;
}

int w4a16_fp4_mm_id(const w4a16_bf16* x, int64_t x_stride, const w4a16_fp4* w, const int32_t* ids, w4a16_bf16* y,
                    int T, int top, int act, void* workspace, size_t workspace_bytes, void* stream) {
  if (env().fault == kFaultValidate) return fail(W4A16_ERR_SHAPE, "injected validation fault (W4A16_FAULT)");
  if (int rc = check_fp4(w, "w")) return rc;
  if (int rc = check_fp4_act(w, act)) return rc;
  if (T < 0 || top < 1 || top > kFp4MaxTop || (int64_t)T * top > kMaxDim)
    return fail(W4A16_ERR_EXPERTS, "T = %d must not be negative, top = %d in 1..%d, T * top at most 2^30", T, top, kFp4MaxTop);
  if (T == 0) return W4A16_OK;
  if (int rc = check_fp4_rows(x, x_stride, T, w->K)) return rc;
  if (!ids || !y) return fail(W4A16_ERR_NULL, "null tensor pointer");
  if (misaligned(ids, 4) || misaligned(y, 2)) return fail(W4A16_ERR_ALIGN, "ids must be 4-byte and y 2-byte aligned");
  const int64_t x_bytes = fp4_x_bytes(x_stride, T, w->K), y_bytes = fp4_y_bytes(w, (int64_t)T * top, act);
  if (int rc = check_fp4_apart(x, x_bytes, w, y, y_bytes)) return rc;
  if (fp4_overlap(ids, 4LL * T * top, y, y_bytes)) return fail(W4A16_ERR_SHAPE, "y overlaps ids");
  const int64_t rows = (int64_t)T * top, tiles = fp4_id_tiles(rows, w->experts), places = tiles * fp4_id_span(rows, w->experts);
  if (places > INT32_MAX) return fail(W4A16_ERR_EXPERTS, "T * top = %lld rows are too many for one call", (long long)rows);
  const Fp4Space sp = fp4_space(places, rows, tiles, w->K, w->format);
  if (int rc = check_fp4_space(workspace, workspace_bytes, sp.total, x, x_bytes, y, y_bytes)) return rc;
  if (env().fault == kFaultLaunch) return fail(W4A16_ERR_CUDA, "injected launch fault (W4A16_FAULT)");
  int* flags = nullptr;
  if (int rc = flag_pointer(&flags)) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* factor = w->format == W4A16_FP4_NV ? reinterpret_cast<float*>(ws + sp.factor) : nullptr;
  int32_t* place = reinterpret_cast<int32_t*>(ws + sp.place);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  Fp4RouteArgs r{ids, (int)rows, top, w->experts, fp4_id_tile(rows, w->experts), fp4_id_span(rows, w->experts), place, reinterpret_cast<int32_t*>(ws + sp.row),
                 reinterpret_cast<Fp4Tile*>(ws + sp.tiles), reinterpret_cast<int32_t*>(ws + sp.count), y,
                 act == W4A16_FP4_LINEAR ? w->rows : w->rows / 2, flags};
  Fp4MmArgs a = {};
  if (fp4_mm_id_fuses(*w, T, top)) {
    a.x = x;
    a.x_stride = x_stride;
    a.w = *w;
    a.y = y;
    a.M = T;
    a.act = act;
    a.ids = ids;
    a.top = top;
    a.flags = flags;
    a.fault_wait = env().fault == kFaultWait;
    cudaError_t e = launch_fp4_mm(a, env().pdl, s);
    return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "w4a16_fp4_mm_id launch");
  }
  Fp4QuantArgs q{x, x_stride, ws, ws + sp.scales, factor, T, w->K, T, w->format};
  std::lock_guard<std::mutex> turn(turn_of(stream));
  if (cudaError_t e = launch_fp4_route_quant(r, q, env().pdl, s)) return cuda_fail(e, "w4a16_fp4_mm_id launch");
  a.xc = ws;
  a.xs = ws + sp.scales;
  a.xf = factor;
  a.x_rows = places;
  a.w = *w;
  a.y = y;
  a.M = (int)rows;
  a.act = act;
  a.tiles = r.tiles;
  a.tile_count = r.count;
  a.row = r.row;
  a.ids = ids;
  a.early = true;
  a.max_tiles = (int)tiles;
  a.nt = r.nt;
  a.flags = flags;
  a.fault_wait = env().fault == kFaultWait;
  cudaError_t e = launch_fp4_mm(a, env().pdl, s);
  return e == cudaSuccess ? W4A16_OK : cuda_fail(e, "w4a16_fp4_mm_id launch");
}

const char* w4a16_last_error(void) { return g_last_error.c_str(); }

const char* w4a16_version(void) { return "w4a16 0.1.0 (sm_103a)"; }

void w4a16_debug_reload_env(void) {
  std::lock_guard<std::mutex> lk(g_env_mu);
  load_env_locked();
}

}  // extern "C"
