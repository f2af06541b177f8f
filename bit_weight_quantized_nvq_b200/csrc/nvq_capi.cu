// C ABI of the library: host-side argument validation, device checks and
// dispatch to the kernel launchers.  Nothing here allocates device memory.
#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

#include "nvq.h"
#include "nvq_internal.h"

namespace {

constexpr int kVersion = 10000;  // 1.0.0
constexpr int kMaxDevices = 64;

thread_local cudaError_t t_last_cuda_error = cudaSuccess;

// 0 = not yet checked, 1 = sm_100, 2 = other architecture.
std::atomic<int> g_device_ok[kMaxDevices];
std::atomic<int> g_device_sms[kMaxDevices];

bool aligned16(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

nvq_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return NVQ_OK;
  t_last_cuda_error = e;
  return NVQ_ERR_CUDA;
}

// The current device must be compute capability 10.0 (B200, sm_100a).
nvq_status check_device() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return cuda_status(e);
  }
  if (dev < 0 || dev >= kMaxDevices) return NVQ_ERR_UNSUPPORTED_DEVICE;
  int state = g_device_ok[dev].load(std::memory_order_relaxed);
  if (state == 0) {
    int major = 0, minor = 0, sms = 0;
    e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e == cudaSuccess)
      e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (e == cudaSuccess)
      e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return cuda_status(e);
    }
    state = (major == 10 && minor == 0) ? 1 : 2;
    g_device_sms[dev].store(sms, std::memory_order_relaxed);
    g_device_ok[dev].store(state, std::memory_order_relaxed);
  }
  return state == 1 ? NVQ_OK : NVQ_ERR_UNSUPPORTED_DEVICE;
}

// Shapes and pointers shared by the weight x activation entry points:
// K a positive multiple of 64, M within [m_min, m_max] (or 0), every pointer
// non-NULL and 16-byte aligned unless the product is empty (M == 0 or
// N == 0).  `need_scales` is false for the integer-sum export, which reads
// neither the weight scales nor the activation scales.
nvq_status check_dot_args(const void* codes, const void* scales, int64_t N,
                          int64_t K, const void* q, const void* d, int64_t M,
                          const void* y, int64_t m_min, int64_t m_max,
                          bool need_scales) {
  if (N < 0 || K < 0 || M < 0) return NVQ_ERR_INVALID_ARG;
  if (K == 0 || K % 64 != 0) return NVQ_ERR_BAD_SHAPE;
  if (K > (int64_t{1} << 30) || N > (int64_t{1} << 30)) return NVQ_ERR_BAD_SHAPE;
  if (M != 0 && (M < m_min || M > m_max)) return NVQ_ERR_BAD_SHAPE;
  if (N == 0 || M == 0) return NVQ_OK;
  if (!codes || !q || !y) return NVQ_ERR_INVALID_ARG;
  if (need_scales && (!scales || !d)) return NVQ_ERR_INVALID_ARG;
  if (!aligned16(codes) || !aligned16(q) || !aligned16(y)) return NVQ_ERR_MISALIGNED;
  if (need_scales && (!aligned16(scales) || !aligned16(d))) return NVQ_ERR_MISALIGNED;
  return NVQ_OK;
}

constexpr int64_t kInt32Max = INT32_MAX;

int64_t dtype_bytes(int dtype) {
  return dtype == NVQ_F32 ? 4 : dtype == NVQ_F16 || dtype == NVQ_BF16 ? 2 : 0;
}

// A packed tensor of `rows` rows of `width` elements, `stride` apart.
nvq_status check_rows(const void* p, int64_t rows, int64_t width, int64_t stride, int64_t bytes) {
  if (rows == 0) return NVQ_OK;
  if (!p) return NVQ_ERR_INVALID_ARG;
  if (stride < width || stride >= (int64_t{1} << 38)) return NVQ_ERR_BAD_SHAPE;   // below a tensor map's 2^40 bytes
  if (!aligned16(p) || stride * bytes % 16 != 0) return NVQ_ERR_MISALIGNED;
  return NVQ_OK;
}

nvq_status check_heads(int64_t heads, int64_t kv_heads, int64_t head_dim) {
  if (heads <= 0 || kv_heads <= 0) return NVQ_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return NVQ_ERR_BAD_SHAPE;
  if (heads > 65535 || kv_heads > 65535 || heads % kv_heads != 0) return NVQ_ERR_BAD_SHAPE;
  return NVQ_OK;
}

nvq_status check_cache(const nvq_kv_cache* c) {
  if (!c || !c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return NVQ_ERR_INVALID_ARG;
  if (c->n_pages <= 0 || c->page_size <= 0) return NVQ_ERR_INVALID_ARG;
  nvq_status st = check_heads(c->n_kv_heads, c->n_kv_heads, c->head_dim);
  if (st != NVQ_OK) return st;
  if (c->page_size % 16 != 0 || c->page_size > 65536 || c->n_pages > kInt32Max ||
      c->n_pages * c->n_kv_heads > kInt32Max / c->page_size)   // rows are 32-bit coordinates
    return NVQ_ERR_BAD_SHAPE;
  if (!aligned16(c->k_codes) || !aligned16(c->k_scales) || !aligned16(c->v_codes) ||
      !aligned16(c->v_scales))
    return NVQ_ERR_MISALIGNED;
  return NVQ_OK;
}

// The packed batch of nvq_kv_write and nvq_kv_read.  The index arrays hold
// int32 and need only their own alignment.
nvq_status check_kv(const nvq_kv_cache* c, const void* k, int64_t k_stride, const void* v,
                    int64_t v_stride, int dtype, const int32_t* cu, const int32_t* lens,
                    const int32_t* table, int64_t B, int64_t max_pages, int64_t rows) {
  if (B < 0 || max_pages < 0 || rows < 0 || dtype_bytes(dtype) == 0) return NVQ_ERR_INVALID_ARG;
  nvq_status st = check_cache(c);
  if (st != NVQ_OK) return st;
  if (B > kInt32Max - 1 || max_pages > kInt32Max || rows > kInt32Max) return NVQ_ERR_BAD_SHAPE;
  if (B == 0 || rows == 0) return NVQ_OK;
  if (!cu || !lens || (!table && max_pages > 0)) return NVQ_ERR_INVALID_ARG;
  const int64_t width = c->n_kv_heads * c->head_dim;
  st = check_rows(k, rows, width, k_stride, dtype_bytes(dtype));
  if (st != NVQ_OK) return st;
  return check_rows(v, rows, width, v_stride, dtype_bytes(dtype));
}

// Up to 2^64: what the kernels multiply it with before the scores (2^17 at most)
// leaves it finite.
bool good_scale(float scale) { return scale > 0.0f && scale <= 0x1p64f; }

}  // namespace

namespace nvq {
void set_last_cuda_error(cudaError_t e) { t_last_cuda_error = e; }

// SMs of the current device: cached on first use (the workspace sizes that
// depend on it are queried before any launch), 148 without a device.
int device_sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 148;
  }
  if (dev < 0 || dev >= kMaxDevices) return 148;
  int sms = g_device_sms[dev].load(std::memory_order_relaxed);
  if (sms > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      sms <= 0) {
    cudaGetLastError();
    return 148;
  }
  g_device_sms[dev].store(sms, std::memory_order_relaxed);
  return sms;
}
}  // namespace nvq

extern "C" {

int nvq_version(void) { return kVersion; }

const char* nvq_status_string(nvq_status status) {
  switch (status) {
    case NVQ_OK: return "ok";
    case NVQ_ERR_INVALID_ARG: return "invalid argument (NULL pointer, negative size or bad value)";
    case NVQ_ERR_BAD_SHAPE: return "unsupported shape (K must be a multiple of 64; M within the entry point's range)";
    case NVQ_ERR_MISALIGNED: return "device pointer not 16-byte aligned";
    case NVQ_ERR_CUDA: return "CUDA runtime error (see nvq_last_cuda_error)";
    case NVQ_ERR_UNSUPPORTED_DEVICE: return "current device is not an sm_100 (B200) GPU";
    case NVQ_ERR_WORKSPACE: return "workspace missing or smaller than nvq_gemm_workspace_size";
    default: return "unknown status";
  }
}

const char* nvq_last_cuda_error(void) { return cudaGetErrorName(t_last_cuda_error); }

nvq_status nvq_quantize_act_q8_0(const float* x, int64_t M, int64_t K,
                                 int8_t* q, uint16_t* d, void* stream) {
  if (M < 0 || K < 0) return NVQ_ERR_INVALID_ARG;
  if (K % 32 != 0) return NVQ_ERR_BAD_SHAPE;
  if (M == 0 || K == 0) return NVQ_OK;
  if (M * K > (int64_t{1} << 40)) return NVQ_ERR_BAD_SHAPE;
  if (!x || !q || !d) return NVQ_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q) || !aligned16(d)) return NVQ_ERR_MISALIGNED;
  nvq_status st = check_device();
  if (st != NVQ_OK) return st;
  return cuda_status(nvq::launch_quantize_q8_0(x, M, K, q, d,
                                               static_cast<cudaStream_t>(stream)));
}

nvq_status nvq_gemv(const uint8_t* codes, const uint8_t* scales, float g,
                    int64_t N, int64_t K, const int8_t* q, const uint16_t* d,
                    int64_t M, float* y, void* stream) {
  nvq_status st = check_dot_args(codes, scales, N, K, q, d, M, y, 1, 16, true);
  if (st != NVQ_OK) return st;
  if (!(g == g)) return NVQ_ERR_INVALID_ARG;  // NaN scale
  if (N == 0 || M == 0) return NVQ_OK;
  st = check_device();
  if (st != NVQ_OK) return st;
  return cuda_status(nvq::launch_gemv(codes, scales, g, N, K, q, d, M, y,
                                      static_cast<cudaStream_t>(stream)));
}

nvq_status nvq_gemv_requant(const uint8_t* codes, const uint8_t* scales, float g, int64_t N,
                            int64_t K, const int8_t* q, const uint16_t* d, float* y,
                            int8_t* q_out, uint16_t* d_out, int32_t* counters, void* stream) {
  nvq_status st = check_dot_args(codes, scales, N, K, q, d, 1, y, 1, 1, true);
  if (st != NVQ_OK) return st;
  if (!(g == g)) return NVQ_ERR_INVALID_ARG;
  if (N % 32 != 0) return NVQ_ERR_BAD_SHAPE;
  if (N == 0) return NVQ_OK;
  if (!q_out || !d_out || !counters) return NVQ_ERR_INVALID_ARG;
  if (!aligned16(q_out) || !aligned16(d_out) || !aligned16(counters)) return NVQ_ERR_MISALIGNED;
  st = check_device();
  if (st != NVQ_OK) return st;
  nvq::GemvTarget t = {codes, scales, g, N, y, q_out, d_out, counters};
  return cuda_status(nvq::launch_gemv_group(&t, 1, K, q, d, static_cast<cudaStream_t>(stream)));
}

nvq_status nvq_gemv_grouped(const nvq_linear* linears, int64_t count, const int8_t* q,
                            const uint16_t* d, int64_t M, float* const* ys, void* stream) {
  if (count < 0 || M < 0) return NVQ_ERR_INVALID_ARG;
  if (count == 0 || M == 0) return NVQ_OK;
  if (!linears || !ys) return NVQ_ERR_INVALID_ARG;
  const int64_t K = linears[0].K;
  int64_t rows = 0;
  for (int64_t i = 0; i < count; ++i) {
    const nvq_linear& L = linears[i];
    if (L.K != K) return NVQ_ERR_BAD_SHAPE;
    nvq_status st = check_dot_args(L.codes, L.scales, L.N, L.K, q, d, M, ys[i], 1, 16, true);
    if (st != NVQ_OK) return st;
    if (!(L.g == L.g)) return NVQ_ERR_INVALID_ARG;
    rows += L.N;
  }
  if (rows > (int64_t{1} << 30)) return NVQ_ERR_BAD_SHAPE;
  nvq_status st = check_device();
  if (st != NVQ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 1) {
    constexpr int kBatch = 16;
    nvq::GemvTarget t[kBatch];
    for (int64_t i0 = 0; i0 < count; i0 += kBatch) {
      int n = 0;
      for (int64_t i = i0; i < count && n < kBatch; ++i) {
        if (linears[i].N == 0) continue;
        t[n++] = {linears[i].codes, linears[i].scales, linears[i].g, linears[i].N, ys[i],
                  nullptr, nullptr, nullptr};
      }
      st = cuda_status(nvq::launch_gemv_group(t, n, K, q, d, s));
      if (st != NVQ_OK) return st;
    }
    return NVQ_OK;
  }
  for (int64_t i = 0; i < count; ++i) {
    const nvq_linear& L = linears[i];
    if (L.N == 0) continue;
    st = cuda_status(nvq::launch_gemv(L.codes, L.scales, L.g, L.N, K, q, d, M, ys[i], s));
    if (st != NVQ_OK) return st;
  }
  return NVQ_OK;
}

nvq_status nvq_moe_gemv(const uint8_t* codes, const uint8_t* scales, const float* g, int64_t E,
                        int64_t N, int64_t K, const int32_t* ids, int64_t T, int64_t top_k,
                        const int8_t* q, const uint16_t* d, float* y, void* stream) {
  if (E < 0 || N < 0 || K < 0 || T < 0 || top_k < 0) return NVQ_ERR_INVALID_ARG;
  if (K == 0 || K % 64 != 0) return NVQ_ERR_BAD_SHAPE;
  if (T == 0 || top_k == 0 || N == 0) return NVQ_OK;
  if (E == 0) return NVQ_ERR_INVALID_ARG;
  if (!nvq::moe_supported(K, top_k)) return NVQ_ERR_BAD_SHAPE;
  if (T > 65535 || N > (int64_t{1} << 24) || E * N > (int64_t{1} << 32)) return NVQ_ERR_BAD_SHAPE;
  if (!codes || !scales || !g || !ids || !q || !d || !y) return NVQ_ERR_INVALID_ARG;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(q) || !aligned16(d) ||
      !aligned16(y) || !aligned16(ids) || !aligned16(g))
    return NVQ_ERR_MISALIGNED;
  nvq_status st = check_device();
  if (st != NVQ_OK) return st;
  return cuda_status(nvq::launch_moe_gemv(codes, scales, g, E, N, K, ids, T, top_k, q, d, y,
                                          static_cast<cudaStream_t>(stream)));
}

size_t nvq_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || K <= 0 || N < 0) return 0;
  return nvq::gemm_workspace_size(M, N, K);
}

nvq_status nvq_gemm(const uint8_t* codes, const uint8_t* scales, float g,
                    int64_t N, int64_t K, const int8_t* q, const uint16_t* d,
                    int64_t M, float* y, void* workspace,
                    size_t workspace_bytes, void* stream) {
  nvq_status st = check_dot_args(codes, scales, N, K, q, d, M, y, 1,
                                 int64_t{1} << 24, true);
  if (st != NVQ_OK) return st;
  if (!(g == g)) return NVQ_ERR_INVALID_ARG;
  if (N == 0 || M == 0) return NVQ_OK;
  if (!workspace || workspace_bytes < nvq::gemm_workspace_size(M, N, K))
    return NVQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return NVQ_ERR_MISALIGNED;
  st = check_device();
  if (st != NVQ_OK) return st;
  return cuda_status(nvq::launch_gemm(codes, scales, g, N, K, q, d, M, y, workspace,
                                      static_cast<cudaStream_t>(stream)));
}

nvq_status nvq_gemm_noalloc(const uint8_t* codes, const uint8_t* scales, float g,
                            int64_t N, int64_t K, const int8_t* q, const uint16_t* d,
                            int64_t M, float* y, void* stream) {
  nvq_status st = check_dot_args(codes, scales, N, K, q, d, M, y, 1,
                                 int64_t{1} << 24, true);
  if (st != NVQ_OK) return st;
  if (!(g == g)) return NVQ_ERR_INVALID_ARG;
  if (N == 0 || M == 0) return NVQ_OK;
  if (nvq::gemm_workspace_size(M, N, K) > nvq::gemm_noalloc_limit()) return NVQ_ERR_WORKSPACE;
  st = check_device();
  if (st != NVQ_OK) return st;
  void* scratch = nullptr;
  cudaError_t e = nvq::gemm_noalloc_scratch(&scratch);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return cuda_status(e);
  }
  return cuda_status(nvq::launch_gemm(codes, scales, g, N, K, q, d, M, y, scratch,
                                      static_cast<cudaStream_t>(stream)));
}

size_t nvq_gemm_w4a16_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || M > 16 || K <= 0 || K % 256 != 0 || N < 0) return 0;
  return nvq::gemm_small_workspace_size(M, K);
}

nvq_status nvq_gemm_w4a16(const uint8_t* codes, const uint8_t* scales, float g, int64_t N,
                          int64_t K, const uint16_t* x, int64_t M, float* y, void* workspace,
                          size_t workspace_bytes, void* stream) {
  // x plays the part of q for the pointer checks; there is no d
  nvq_status st = check_dot_args(codes, scales, N, K, x, x, M, y, 1, 16, true);
  if (st != NVQ_OK) return st;
  if (!(g == g)) return NVQ_ERR_INVALID_ARG;
  if (K % 256 != 0) return NVQ_ERR_BAD_SHAPE;
  if (N == 0 || M == 0) return NVQ_OK;
  if (!workspace || workspace_bytes < nvq::gemm_small_workspace_size(M, K))
    return NVQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return NVQ_ERR_MISALIGNED;
  st = check_device();
  if (st != NVQ_OK) return st;
  return cuda_status(nvq::launch_gemm_small_f16(codes, scales, g, N, K, x, M, y, workspace,
                                                static_cast<cudaStream_t>(stream)));
}

nvq_status nvq_quantize_act_nvfp4(const float* x, int64_t M, int64_t K, uint8_t* codes,
                                  uint8_t* scales, float* g, void* stream) {
  if (M < 0 || K < 0) return NVQ_ERR_INVALID_ARG;
  if (K % 16 != 0) return NVQ_ERR_BAD_SHAPE;
  if (M == 0 || K == 0) return NVQ_OK;
  if (M > INT32_MAX || K > (int64_t{1} << 30)) return NVQ_ERR_BAD_SHAPE;
  if (!x || !codes || !scales || !g) return NVQ_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales) || !aligned16(g))
    return NVQ_ERR_MISALIGNED;
  nvq_status st = check_device();
  if (st != NVQ_OK) return st;
  return cuda_status(nvq::launch_quantize_nvfp4(x, M, K, codes, scales, g,
                                                static_cast<cudaStream_t>(stream)));
}

nvq_status nvq_gemm_nvf4(const uint8_t* w_codes, const uint8_t* w_scales, float g_w, int64_t N,
                         int64_t K, const uint8_t* a_codes, const uint8_t* a_scales,
                         const float* a_g, int64_t M, float* y, void* stream) {
  if (N < 0 || K < 0 || M < 0) return NVQ_ERR_INVALID_ARG;
  if (K == 0 || K % 256 != 0) return NVQ_ERR_BAD_SHAPE;
  if (K > (int64_t{1} << 30) || N > int64_t{65535} * 128 || M > INT32_MAX)
    return NVQ_ERR_BAD_SHAPE;
  if (!(g_w == g_w)) return NVQ_ERR_INVALID_ARG;
  if (N == 0 || M == 0) return NVQ_OK;
  if (!w_codes || !w_scales || !a_codes || !a_scales || !a_g || !y) return NVQ_ERR_INVALID_ARG;
  if (!aligned16(w_codes) || !aligned16(w_scales) || !aligned16(a_codes) ||
      !aligned16(a_scales) || !aligned16(a_g) || !aligned16(y))
    return NVQ_ERR_MISALIGNED;
  nvq_status st = check_device();
  if (st != NVQ_OK) return st;
  return cuda_status(nvq::launch_gemm_nvf4(w_codes, w_scales, g_w, N, K, a_codes, a_scales, a_g,
                                           M, y, static_cast<cudaStream_t>(stream)));
}

nvq_status nvq_debug_subblock_sums(const uint8_t* codes, const uint8_t* scales, float g,
                                   int64_t N, int64_t K, const int8_t* q, const uint16_t* d,
                                   int64_t M, float* y, int32_t* isum, void* stream) {
  nvq_status st = check_dot_args(codes, scales, N, K, q, d, M, y, 1, 16, true);
  if (st != NVQ_OK) return st;
  if (!(g == g)) return NVQ_ERR_INVALID_ARG;
  if (N == 0 || M == 0) return NVQ_OK;
  if (!isum) return NVQ_ERR_INVALID_ARG;
  if (!aligned16(isum)) return NVQ_ERR_MISALIGNED;
  st = check_device();
  if (st != NVQ_OK) return st;
  return cuda_status(nvq::launch_gemv_isum(codes, scales, g, N, K, q, d, M, y, isum,
                                           static_cast<cudaStream_t>(stream)));
}

nvq_status nvq_kv_write(const nvq_kv_cache* cache, const void* k, int64_t k_stride, const void* v,
                        int64_t v_stride, int dtype, const int32_t* cu_seqlens,
                        const int32_t* seq_lens, const int32_t* block_table, int64_t B,
                        int64_t max_pages, int64_t rows, void* stream) {
  nvq_status st = check_kv(cache, k, k_stride, v, v_stride, dtype, cu_seqlens, seq_lens,
                           block_table, B, max_pages, rows);
  if (st != NVQ_OK || B == 0 || rows == 0) return st;
  st = check_device();
  if (st != NVQ_OK) return st;
  const nvq::KvBatch b = {cu_seqlens, seq_lens, block_table, B, max_pages, rows};
  return cuda_status(nvq::launch_kv_write(*cache, b, k, k_stride, v, v_stride, dtype,
                                          static_cast<cudaStream_t>(stream)));
}

nvq_status nvq_kv_read(const nvq_kv_cache* cache, void* k, int64_t k_stride, void* v,
                       int64_t v_stride, int dtype, const int32_t* cu_seqlens,
                       const int32_t* seq_lens, const int32_t* block_table, int64_t B,
                       int64_t max_pages, int64_t rows, void* stream) {
  nvq_status st = check_kv(cache, k, k_stride, v, v_stride, dtype, cu_seqlens, seq_lens,
                           block_table, B, max_pages, rows);
  if (st != NVQ_OK || B == 0 || rows == 0) return st;
  st = check_device();
  if (st != NVQ_OK) return st;
  const nvq::KvBatch b = {cu_seqlens, seq_lens, block_table, B, max_pages, rows};
  return cuda_status(nvq::launch_kv_read(*cache, b, k, k_stride, v, v_stride, dtype,
                                         static_cast<cudaStream_t>(stream)));
}

size_t nvq_attn_decode_workspace_size(int64_t B, int64_t n_heads, int64_t n_kv_heads,
                                      int64_t head_dim) {
  if (B <= 0 || check_heads(n_heads, n_kv_heads, head_dim) != NVQ_OK) return 0;
  return nvq::attn_decode_workspace_size(B, n_heads, n_kv_heads, head_dim);
}

nvq_status nvq_attn_decode(const nvq_kv_cache* cache, const void* q, int64_t q_stride, int dtype,
                           const int32_t* seq_lens, const int32_t* block_table, int64_t B,
                           int64_t max_pages, int64_t n_heads, float scale, void* out,
                           int64_t out_stride, int32_t* counters, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (B < 0 || max_pages < 0 || dtype_bytes(dtype) == 0 || !good_scale(scale))
    return NVQ_ERR_INVALID_ARG;
  nvq_status st = check_cache(cache);
  if (st != NVQ_OK) return st;
  st = check_heads(n_heads, cache->n_kv_heads, cache->head_dim);
  if (st != NVQ_OK) return st;
  if (B > 65535 || max_pages > kInt32Max || max_pages * cache->page_size > kInt32Max)
    return NVQ_ERR_BAD_SHAPE;
  // the work is counted in 32 bits: 64-token tiles of every key-value head
  // (and chunk of 8 or 16 heads that share one), with room for their ends
  const int64_t share = dtype == NVQ_F32 ? 8 : 16;
  const int64_t chunks = (n_heads / cache->n_kv_heads + share - 1) / share;
  if (B * cache->n_kv_heads * chunks > kInt32Max / (max_pages * cache->page_size / 64 + 8))
    return NVQ_ERR_BAD_SHAPE;
  if (B == 0) return NVQ_OK;
  if (!seq_lens || (!block_table && max_pages > 0) || !counters) return NVQ_ERR_INVALID_ARG;
  const int64_t width = n_heads * cache->head_dim;
  st = check_rows(q, B, width, q_stride, dtype_bytes(dtype));
  if (st == NVQ_OK) st = check_rows(out, B, width, out_stride, dtype_bytes(dtype));
  if (st != NVQ_OK) return st;
  if (!workspace || workspace_bytes < nvq::attn_decode_workspace_size(B, n_heads, cache->n_kv_heads,
                                                                      cache->head_dim))
    return NVQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return NVQ_ERR_MISALIGNED;
  st = check_device();
  if (st != NVQ_OK) return st;
  return cuda_status(nvq::launch_attn_decode(*cache, seq_lens, block_table, B, max_pages, q,
                                             q_stride, n_heads, scale, dtype, out, out_stride,
                                             counters, workspace,
                                             static_cast<cudaStream_t>(stream)));
}

nvq_status nvq_attn_prefill(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                            const void* v, int64_t v_stride, int dtype, const int32_t* cu_q,
                            const int32_t* cu_k, int64_t B, int64_t total_q, int64_t total_k,
                            int64_t n_heads, int64_t n_kv_heads, int64_t head_dim, float scale,
                            int causal, void* out, int64_t out_stride, void* stream) {
  if (B < 0 || total_q < 0 || total_k < 0 || !good_scale(scale)) return NVQ_ERR_INVALID_ARG;
  if (dtype != NVQ_F16 && dtype != NVQ_BF16) return NVQ_ERR_INVALID_ARG;
  nvq_status st = check_heads(n_heads, n_kv_heads, head_dim);
  if (st != NVQ_OK) return st;
  if (B > 65535 || total_q > kInt32Max / 2 || total_k > kInt32Max / 2) return NVQ_ERR_BAD_SHAPE;
  if ((total_q / 128 + B) * n_heads > kInt32Max / 2) return NVQ_ERR_BAD_SHAPE;   // work items are counted in 32 bits
  if (B == 0 || total_q == 0) return NVQ_OK;
  if (!cu_q || !cu_k) return NVQ_ERR_INVALID_ARG;
  st = check_rows(q, total_q, n_heads * head_dim, q_stride, 2);
  if (st == NVQ_OK) st = check_rows(out, total_q, n_heads * head_dim, out_stride, 2);
  if (st == NVQ_OK) st = check_rows(k, total_k, n_kv_heads * head_dim, k_stride, 2);
  if (st == NVQ_OK) st = check_rows(v, total_k, n_kv_heads * head_dim, v_stride, 2);
  if (st != NVQ_OK) return st;
  st = check_device();
  if (st != NVQ_OK) return st;
  const nvq::PrefillArgs a = {q, k, v, out, q_stride, k_stride, v_stride, out_stride, cu_q, cu_k,
                              B, total_q, total_k, n_heads, n_kv_heads, head_dim, scale, causal};
  return cuda_status(nvq::launch_attn_prefill(a, dtype, static_cast<cudaStream_t>(stream)));
}

nvq_status nvq_error_flags(unsigned int* flags, int clear) {
  if (!flags) return NVQ_ERR_INVALID_ARG;
  nvq_status st = check_device();
  if (st != NVQ_OK) return st;
  unsigned int gemv = 0, gemm = 0, gemm_small = 0, nvf4 = 0;
  cudaError_t e = nvq::gemv_error_flags(clear != 0, &gemv);
  if (e == cudaSuccess) e = nvq::gemm_error_flags(clear != 0, &gemm);
  if (e == cudaSuccess) e = nvq::gemm_small_error_flags(clear != 0, &gemm_small);
  if (e == cudaSuccess) e = nvq::nvf4_error_flags(clear != 0, &nvf4);
  gemm |= gemm_small | nvf4;
  unsigned int kv = 0, decode = 0, prefill = 0;
  if (e == cudaSuccess) e = nvq::kv_error_flags(clear != 0, &kv);
  if (e == cudaSuccess) e = nvq::attn_decode_error_flags(clear != 0, &decode);
  if (e == cudaSuccess) e = nvq::attn_prefill_error_flags(clear != 0, &prefill);
  const unsigned int attn = kv | decode | prefill;
  if (e != cudaSuccess) {
    cudaGetLastError();
    return cuda_status(e);
  }
  *flags = ((gemv & 1u) ? NVQ_FLAG_GEMV_TIMEOUT : 0u) | (gemm ? NVQ_FLAG_GEMM_TIMEOUT : 0u) |
           (((gemv | attn) & 2u) ? NVQ_FLAG_BAD_INDEX : 0u) |
           ((attn & 1u) ? NVQ_FLAG_ATTN_TIMEOUT : 0u);
  return NVQ_OK;
}

nvq_status nvq_debug_stalled_wait(uint64_t limit_ns, int* result, void* stream) {
  if (!result) return NVQ_ERR_INVALID_ARG;
  if (limit_ns < 1000 || limit_ns > 1000000000ull) return NVQ_ERR_INVALID_ARG;
  if (!aligned16(result)) return NVQ_ERR_MISALIGNED;
  nvq_status st = check_device();
  if (st != NVQ_OK) return st;
  return cuda_status(nvq::launch_stalled_wait(limit_ns, result,
                                              static_cast<cudaStream_t>(stream)));
}

nvq_status nvq_debug_stalled_attn_wait(uint64_t limit_ns, int moving, int* result, void* stream) {
  if (!result) return NVQ_ERR_INVALID_ARG;
  if (limit_ns < 1000 || limit_ns > 1000000000ull) return NVQ_ERR_INVALID_ARG;
  if (!aligned16(result)) return NVQ_ERR_MISALIGNED;
  nvq_status st = check_device();
  if (st != NVQ_OK) return st;
  return cuda_status(nvq::launch_stalled_attn_wait(limit_ns, moving, result,
                                                   static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
