// Prompt attention: packed sequences, grouped heads, causal or not.
//
// Query i of a sequence (n queries, m keys) sees the keys j < m, with
// `causal` only j <= i + m - n (the queries are the last n positions):
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q.k_j - max);
// a query that sees no key gives 0.
//
// One warp per (row, head) with an online softmax.
#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "nvq_internal.h"

namespace nvq {
namespace {

constexpr int kWarps = 8;

__device__ unsigned int g_attn_prefill_error_flags = 0;   // bit 0: a wait timed out, bit 1: a bad index

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32)
attn_prefill_kernel(PrefillArgs a, float scale_log2) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * kWarps + (threadIdx.x >> 5), h = blockIdx.y;
  if (row >= a.total_q) return;
  const int b = dev::warp_find_seq(a.cu_q, static_cast<int>(a.B), row, lane);
  if (b >= a.B) return;
  const int hk = h / static_cast<int>(a.heads / a.kv_heads);
  const int64_t k0 = a.cu_k[b];
  int64_t m_keys = a.cu_k[b + 1] - k0;
  const int64_t i = row - a.cu_q[b], n = a.cu_q[b + 1] - a.cu_q[b];
  if (k0 < 0 || m_keys < 0 || k0 + m_keys > a.total_k || i < 0 || i >= n ||
      a.cu_q[b + 1] > a.total_q) {
    if (lane == 0) atomicOr(&g_attn_prefill_error_flags, 2u);
    m_keys = 0;
  }
  const int64_t end = a.causal ? min(m_keys, i + m_keys - n + 1) : m_keys;
  const T* q = static_cast<const T*>(a.q) + row * a.q_stride + h * D + lane * E;
  float qv[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) qv[e] = dev::to_f32(q[e]) * scale_log2, o[e] = 0.0f;
  for (int64_t j = 0; j < end; ++j) {
    const T* k = static_cast<const T*>(a.k) + (k0 + j) * a.k_stride + hk * D + lane * E;
    const T* v = static_cast<const T*>(a.v) + (k0 + j) * a.v_stride + hk * D + lane * E;
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += qv[e] * dev::to_f32(k[e]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s), c = exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = l * c + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * dev::to_f32(v[e]);
  }
  T* out = static_cast<T*>(a.out) + row * a.out_stride + h * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = dev::from_f32<T>(end <= 0 ? 0.0f : o[e] / l);
}

template <typename T>
cudaError_t prefill_t(const PrefillArgs& a, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.total_q + kWarps - 1) / kWarps), static_cast<unsigned>(a.heads));
  const float c = a.scale * 1.4426950408889634f;
  if (a.head_dim == 64)
    attn_prefill_kernel<T, 64><<<grid, kWarps * 32, 0, stream>>>(a, c);
  else
    attn_prefill_kernel<T, 128><<<grid, kWarps * 32, 0, stream>>>(a, c);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prefill(const PrefillArgs& a, int dtype, cudaStream_t stream) {
  return dtype == NVQ_F16 ? prefill_t<__half>(a, stream) : prefill_t<__nv_bfloat16>(a, stream);
}

cudaError_t attn_prefill_error_flags(bool clear, unsigned int* flags) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_attn_prefill_error_flags, sizeof(unsigned int));
  if (e == cudaSuccess && clear) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_attn_prefill_error_flags, &zero, sizeof(zero));
  }
  return e;
}

}  // namespace nvq
