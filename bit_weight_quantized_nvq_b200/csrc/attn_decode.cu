// Decode attention over the paged Q8_0 cache: one new token per sequence.
//
//   o[h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q[h].k_j - m),
//   m = max_j scale * q[h].k_j,  j < len;  an empty context gives 0.
//
// One CTA per (sequence, head).  Each warp takes every fourth token and
// keeps its own running maximum, sum and output row (online softmax); the
// four are joined at the end.
#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "nvq_internal.h"

namespace nvq {
namespace {

constexpr int kWarps = 4;

__device__ unsigned int g_attn_decode_error_flags = 0;   // bit 1: a bad index

struct DecodeArgs {
  const int8_t* kc;
  const __half* ks;
  const int8_t* vc;
  const __half* vs;
  const int32_t* lens;
  const int32_t* table;
  int max_pages, n_pages, page, kv_heads, heads;
  float scale_log2;
};

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32)
attn_decode_kernel(DecodeArgs a, const T* __restrict__ q, int64_t q_stride, T* __restrict__ out,
                   int64_t out_stride) {
  constexpr int E = D / 32;            // values of the head per lane, within one Q8_0 block
  const int b = blockIdx.y, h = blockIdx.x, hk = h / (a.heads / a.kv_heads);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float qv[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    qv[i] = dev::to_f32(q[b * q_stride + h * D + lane * E + i]) * a.scale_log2;
    o[i] = 0.0f;
  }
  int64_t len = a.lens[b];
  if (len < 0 || len > static_cast<int64_t>(a.max_pages) * a.page) {
    if (threadIdx.x == 0) atomicOr(&g_attn_decode_error_flags, 2u);
    len = len < 0 ? 0 : static_cast<int64_t>(a.max_pages) * a.page;
  }
  for (int64_t t = warp; t < len; t += kWarps) {
    int page = a.table[static_cast<int64_t>(b) * a.max_pages + t / a.page];
    if (page < 0 || page >= a.n_pages) {
      if (lane == 0) atomicOr(&g_attn_decode_error_flags, 2u);
      page = 0;
    }
    const int64_t at = ((static_cast<int64_t>(page) * a.kv_heads + hk) * a.page + t % a.page) * D + lane * E;
    const float dk = __half2float(a.ks[at / 32]), dv = __half2float(a.vs[at / 32]);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) s += qv[i] * static_cast<float>(a.kc[at + i]);
    s *= dk;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s), c = exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = l * c + p;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * c + p * dv * static_cast<float>(a.vc[at + i]);
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int i = 0; i < E; ++i) so[warp][lane * E + i] = o[i];
  __syncthreads();
  if (threadIdx.x < D) {
    float M = -INFINITY, L = 0.0f, O = 0.0f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
    for (int w = 0; w < kWarps; ++w) {
      const float c = sl[w] > 0.0f ? exp2f(sm[w] - M) : 0.0f;
      L += sl[w] * c;
      O += so[w][threadIdx.x] * c;
    }
    out[b * out_stride + h * D + threadIdx.x] = dev::from_f32<T>(len == 0 ? 0.0f : O / L);
  }
}

template <typename T>
cudaError_t decode_t(const nvq_kv_cache& c, const DecodeArgs& a, int64_t B, const void* q,
                     int64_t q_stride, void* out, int64_t out_stride, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.heads), static_cast<unsigned>(B));
  if (c.head_dim == 64)
    attn_decode_kernel<T, 64><<<grid, kWarps * 32, 0, stream>>>(a, static_cast<const T*>(q), q_stride, static_cast<T*>(out), out_stride);
  else
    attn_decode_kernel<T, 128><<<grid, kWarps * 32, 0, stream>>>(a, static_cast<const T*>(q), q_stride, static_cast<T*>(out), out_stride);
  return cudaGetLastError();
}

}  // namespace

size_t attn_decode_workspace_size(int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim) {
  return 16;
}

cudaError_t launch_attn_decode(const nvq_kv_cache& c, const int32_t* seq_lens,
                               const int32_t* block_table, int64_t B, int64_t max_pages,
                               const void* q, int64_t q_stride, int64_t heads, float scale,
                               int dtype, void* out, int64_t out_stride, int32_t* counters,
                               void* workspace, cudaStream_t stream) {
  const DecodeArgs a = {c.k_codes, reinterpret_cast<const __half*>(c.k_scales), c.v_codes,
                        reinterpret_cast<const __half*>(c.v_scales), seq_lens, block_table,
                        static_cast<int>(max_pages), static_cast<int>(c.n_pages),
                        static_cast<int>(c.page_size), static_cast<int>(c.n_kv_heads),
                        static_cast<int>(heads), scale * 1.4426950408889634f};
  switch (dtype) {
    case NVQ_F32: return decode_t<float>(c, a, B, q, q_stride, out, out_stride, stream);
    case NVQ_F16: return decode_t<__half>(c, a, B, q, q_stride, out, out_stride, stream);
    default: return decode_t<__nv_bfloat16>(c, a, B, q, q_stride, out, out_stride, stream);
  }
}

cudaError_t attn_decode_error_flags(bool clear, unsigned int* flags) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_attn_decode_error_flags, sizeof(unsigned int));
  if (e == cudaSuccess && clear) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_attn_decode_error_flags, &zero, sizeof(zero));
  }
  return e;
}

}  // namespace nvq
