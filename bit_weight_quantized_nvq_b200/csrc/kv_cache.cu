// Paged key-value cache in Q8_0: quantise rows as they are written, and read
// rows back.
//
// A cache holds keys and values as the library's Q8_0 (32 int8 codes under
// one fp16 scale; the GGML type table of the spke.com 2-bit GGUF tutorial),
// blocks running along the head.  Pages are [kv_head][token][head_dim], so
// one head's tokens of a page are one contiguous run of codes and one of
// scales, the unit that the decode attention copies.  The quantisation is
// the activation quantiser's, operation for operation (amax / 127 and
// x / d32 by IEEE division, rint, clamp; d = fp16(d32)), so a cached row is
// bit-identical to nvq_quantize_act_q8_0 of it.
//
// Both kernels are HBM-bound when they move many rows (write: e + 1.0625
// bytes per value, read: 1.0625 + e) and launch-bound for a decode step.
#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "nvq_internal.h"

namespace nvq {
namespace {

constexpr int kThreads = 256;
constexpr int kElems = 8;      // values per thread: a quarter of a Q8_0 block

__device__ unsigned int g_kv_error_flags = 0;   // bit 1: a bad index

// Where the rows of a packed batch lie in the pages.
struct Paged {
  const int32_t* cu;       // [B + 1]
  const int32_t* lens;     // [B]
  const int32_t* table;    // [B, max_pages]
  int B, rows, max_pages, n_pages, page, heads, dim;
};

// (page * heads * page_size + offset), the token's place for head 0, or -1
// for a row that has none: padding behind the last sequence, or a bad
// length or page (which raises the flag).  The whole warp calls.
__device__ __forceinline__ int64_t warp_place(const Paged& p, int row, int lane) {
  const int b = dev::warp_find_seq(p.cu, p.B, row, lane);
  if (b >= p.B) return -1;
  const int64_t pos = static_cast<int64_t>(__ldg(p.lens + b)) - __ldg(p.cu + b + 1) + row;
  int page = -1;
  if (pos >= 0 && pos < static_cast<int64_t>(p.max_pages) * p.page)
    page = __ldg(p.table + static_cast<int64_t>(b) * p.max_pages + pos / p.page);
  if (page < 0 || page >= p.n_pages) {
    if (lane == 0) atomicOr(&g_kv_error_flags, 2u);
    return -1;
  }
  return static_cast<int64_t>(page) * p.heads * p.page + pos % p.page;
}

// One CTA per group of `rpc` rows (at most one row per warp): warp w finds
// the place of row w, then every thread takes kElems values of K or V.
template <typename T>
__global__ void __launch_bounds__(kThreads)
kv_write_kernel(Paged p, int rpc, const T* __restrict__ k, int64_t k_stride,
                const T* __restrict__ v, int64_t v_stride, int8_t* __restrict__ kc,
                __half* __restrict__ ks, int8_t* __restrict__ vc, __half* __restrict__ vs) {
  __shared__ int64_t place[kThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.x * rpc;
  if (warp < rpc) {
    const int64_t at = row0 + warp < p.rows ? warp_place(p, row0 + warp, lane) : -1;
    if (lane == 0) place[warp] = at;
  }
  __syncthreads();
  const int half_row = p.heads * p.dim / kElems;      // threads of one row's K
  const int n = min(rpc, p.rows - row0) * 2 * half_row;
  // n is a multiple of 16, so the four lanes of a block run together; the
  // mask names only them
  const unsigned quad = 0xFu << (lane & 28);
  for (int t = threadIdx.x; t < n; t += kThreads) {
    const int r = t / (2 * half_row);
    int e = t - r * 2 * half_row;
    const bool is_v = e >= half_row;
    if (is_v) e -= half_row;
    const T* src = is_v ? v + (row0 + r) * v_stride : k + (row0 + r) * k_stride;
    const auto in = *reinterpret_cast<const dev::Vec<T, kElems>*>(src + static_cast<int64_t>(e) * kElems);
    float x[kElems], a = 0.0f;
#pragma unroll
    for (int i = 0; i < kElems; ++i) {
      x[i] = dev::to_f32(in.v[i]);
      a = fmaxf(a, fabsf(x[i]));
    }
    a = fmaxf(a, __shfl_xor_sync(quad, a, 1));
    a = fmaxf(a, __shfl_xor_sync(quad, a, 2));
    const float d32 = __fdiv_rn(a, 127.0f);
    uint32_t w[2] = {0u, 0u};
    if (d32 > 0.0f) {
#pragma unroll
      for (int i = 0; i < kElems; ++i) {
        int q = __float2int_rn(__fdiv_rn(x[i], d32));
        q = max(-127, min(127, q));
        w[i >> 2] |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * (i & 3));
      }
    }
    const int64_t at = place[r];
    if (at < 0) continue;
    const int h = e * kElems / p.dim;
    const int64_t o = (at + static_cast<int64_t>(h) * p.page) * p.dim + (e * kElems - h * p.dim);
    *reinterpret_cast<uint2*>((is_v ? vc : kc) + o) = make_uint2(w[0], w[1]);
    if ((lane & 3) == 0) (is_v ? vs : ks)[o / 32] = __float2half_rn(d32);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
kv_read_kernel(Paged p, int rpc, const int8_t* __restrict__ kc, const __half* __restrict__ ks,
               const int8_t* __restrict__ vc, const __half* __restrict__ vs, T* __restrict__ k,
               int64_t k_stride, T* __restrict__ v, int64_t v_stride) {
  __shared__ int64_t place[kThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.x * rpc;
  if (warp < rpc) {
    const int64_t at = row0 + warp < p.rows ? warp_place(p, row0 + warp, lane) : -1;
    if (lane == 0) place[warp] = at;
  }
  __syncthreads();
  const int half_row = p.heads * p.dim / kElems;
  const int n = min(rpc, p.rows - row0) * 2 * half_row;
  for (int t = threadIdx.x; t < n; t += kThreads) {
    const int r = t / (2 * half_row);
    int e = t - r * 2 * half_row;
    const bool is_v = e >= half_row;
    if (is_v) e -= half_row;
    const int64_t at = place[r];
    if (at < 0) continue;
    const int h = e * kElems / p.dim;
    const int64_t o = (at + static_cast<int64_t>(h) * p.page) * p.dim + (e * kElems - h * p.dim);
    const auto q = *reinterpret_cast<const dev::Vec<int8_t, kElems>*>((is_v ? vc : kc) + o);
    // code * scale has at most 18 significant bits: exact in fp32, rounded once
    const float d = __half2float((is_v ? vs : ks)[o / 32]);
    dev::Vec<T, kElems> out;
#pragma unroll
    for (int i = 0; i < kElems; ++i) out.v[i] = dev::from_f32<T>(static_cast<float>(q.v[i]) * d);
    T* dst = is_v ? v + (row0 + r) * v_stride : k + (row0 + r) * k_stride;
    *reinterpret_cast<dev::Vec<T, kElems>*>(dst + static_cast<int64_t>(e) * kElems) = out;
  }
}

Paged paged_of(const nvq_kv_cache& c, const KvBatch& b) {
  return {b.cu_seqlens, b.seq_lens, b.block_table, static_cast<int>(b.B), static_cast<int>(b.rows),
          static_cast<int>(b.max_pages), static_cast<int>(c.n_pages), static_cast<int>(c.page_size),
          static_cast<int>(c.n_kv_heads), static_cast<int>(c.head_dim)};
}

// rows per CTA: as many as fill its threads, at most one per warp
int rows_per_cta(const nvq_kv_cache& c) {
  const int64_t per_row = 2 * c.n_kv_heads * c.head_dim / kElems;
  return static_cast<int>(per_row >= kThreads ? 1 : kThreads / per_row > 8 ? 8 : kThreads / per_row);
}

cudaLaunchConfig_t config(int64_t rows, int rpc, cudaStream_t stream, cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + rpc - 1) / rpc));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <typename T>
cudaError_t write_t(const nvq_kv_cache& c, const KvBatch& b, const void* k, int64_t k_stride,
                    const void* v, int64_t v_stride, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  const int rpc = rows_per_cta(c);
  const cudaLaunchConfig_t cfg = config(b.rows, rpc, stream, &attr);
  return cudaLaunchKernelEx(&cfg, kv_write_kernel<T>, paged_of(c, b), rpc, static_cast<const T*>(k),
                            k_stride, static_cast<const T*>(v), v_stride, c.k_codes,
                            reinterpret_cast<__half*>(c.k_scales), c.v_codes,
                            reinterpret_cast<__half*>(c.v_scales));
}

template <typename T>
cudaError_t read_t(const nvq_kv_cache& c, const KvBatch& b, void* k, int64_t k_stride, void* v,
                   int64_t v_stride, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  const int rpc = rows_per_cta(c);
  const cudaLaunchConfig_t cfg = config(b.rows, rpc, stream, &attr);
  return cudaLaunchKernelEx(&cfg, kv_read_kernel<T>, paged_of(c, b), rpc,
                            static_cast<const int8_t*>(c.k_codes),
                            reinterpret_cast<const __half*>(c.k_scales),
                            static_cast<const int8_t*>(c.v_codes),
                            reinterpret_cast<const __half*>(c.v_scales), static_cast<T*>(k),
                            k_stride, static_cast<T*>(v), v_stride);
}

}  // namespace

cudaError_t launch_kv_write(const nvq_kv_cache& c, const KvBatch& b, const void* k,
                            int64_t k_stride, const void* v, int64_t v_stride, int dtype,
                            cudaStream_t stream) {
  switch (dtype) {
    case NVQ_F32: return write_t<float>(c, b, k, k_stride, v, v_stride, stream);
    case NVQ_F16: return write_t<__half>(c, b, k, k_stride, v, v_stride, stream);
    default: return write_t<__nv_bfloat16>(c, b, k, k_stride, v, v_stride, stream);
  }
}

cudaError_t launch_kv_read(const nvq_kv_cache& c, const KvBatch& b, void* k, int64_t k_stride,
                           void* v, int64_t v_stride, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case NVQ_F32: return read_t<float>(c, b, k, k_stride, v, v_stride, stream);
    case NVQ_F16: return read_t<__half>(c, b, k, k_stride, v, v_stride, stream);
    default: return read_t<__nv_bfloat16>(c, b, k, k_stride, v, v_stride, stream);
  }
}

cudaError_t kv_error_flags(bool clear, unsigned int* flags) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_kv_error_flags, sizeof(unsigned int));
  if (e == cudaSuccess && clear) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_kv_error_flags, &zero, sizeof(zero));
  }
  return e;
}

}  // namespace nvq
