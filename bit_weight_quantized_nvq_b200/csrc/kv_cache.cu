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
constexpr int kElems = 16;     // values per thread: half a Q8_0 block
constexpr int kMaxRows = kThreads / 32;

__device__ unsigned int g_kv_error_flags = 0;   // bit 1: a bad index

// Where the rows of a packed batch lie in the pages.
struct Paged {
  const int32_t* cu;       // [B + 1]
  const int32_t* lens;     // [B]
  const int32_t* table;    // [B, max_pages]
  int B, rows, max_pages, n_pages, page, heads, dim_shift;
  int per_row;             // threads of one row: its K, then its V
};

// (page * heads * page_size + offset), the token's place for head 0, or -1
// for a row that has none: padding behind the last sequence, or a bad
// length or page (which raises the flag).  The whole warp calls.
__device__ __forceinline__ int64_t warp_place(const Paged& p, int row, int lane) {
  const int b = dev::warp_find_seq(p.cu, p.B, row, lane);
  if (b >= p.B) return -1;
  const int64_t pos = static_cast<int64_t>(__ldg(p.lens + b)) - __ldg(p.cu + b + 1) + row;
  int page = -1, off = 0;
  if (pos >= 0 && pos < static_cast<int64_t>(p.max_pages) * p.page) {
    // below 2^47: an exact quotient needs 64 bits only for contexts over 2^31
    const int col = pos <= INT32_MAX ? static_cast<int>(pos) / p.page : static_cast<int>(pos / p.page);
    off = static_cast<int>(pos - static_cast<int64_t>(col) * p.page);
    page = __ldg(p.table + static_cast<int64_t>(b) * p.max_pages + col);
  }
  if (page < 0 || page >= p.n_pages) {
    if (lane == 0) atomicOr(&g_kv_error_flags, 2u);
    return -1;
  }
  return static_cast<int64_t>(page) * p.heads * p.page + off;
}

// One CTA per `rpc` rows: warp w finds the place of row w, then thread t takes
// the CTA's 16-value pieces t, t + 256, ..  A piece is in K or V of one row.
struct Piece {
  int64_t at;        // row's place (-1: none)
  int64_t cached;    // its first value in the codes
  int row, elem;     // packed row, first element of the row
  bool is_v;
};
__device__ __forceinline__ Piece piece_of(const Paged& p, const int64_t* place, int row0, int t) {
  Piece x;
  const int r = t / p.per_row;
  int e = t - r * p.per_row;
  x.is_v = 2 * e >= p.per_row;
  if (x.is_v) e -= p.per_row / 2;
  x.row = row0 + r;
  x.elem = e * kElems;
  x.at = place[r];
  const int h = x.elem >> p.dim_shift;
  x.cached = ((x.at + static_cast<int64_t>(h) * p.page) << p.dim_shift) + (x.elem - (h << p.dim_shift));
  return x;
}
__device__ __forceinline__ int find_places(const Paged& p, int rpc, int64_t* place) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.x * rpc;
  if (warp < rpc) {
    const int64_t at = row0 + warp < p.rows ? warp_place(p, row0 + warp, lane) : -1;
    if (lane == 0) place[warp] = at;
  }
  __syncthreads();
  return min(rpc, p.rows - row0) * p.per_row;       // pieces
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
kv_write_kernel(const Paged p, int rpc, const T* __restrict__ k, int64_t k_stride,
                const T* __restrict__ v, int64_t v_stride, int8_t* __restrict__ kc,
                __half* __restrict__ ks, int8_t* __restrict__ vc, __half* __restrict__ vs) {
  __shared__ int64_t place[kMaxRows];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = find_places(p, rpc, place);
  // n is even, so both lanes of a block run together; the mask names only them
  const unsigned pair = 3u << (threadIdx.x & 30);
  for (int t = threadIdx.x; t < n; t += kThreads) {
    const Piece x = piece_of(p, place, blockIdx.x * rpc, t);
    const T* src = (x.is_v ? v + x.row * v_stride : k + x.row * k_stride) + x.elem;
    const auto in = *reinterpret_cast<const dev::Vec<T, kElems>*>(src);
    float f[kElems], a = 0.0f;
#pragma unroll
    for (int i = 0; i < kElems; ++i) {
      f[i] = dev::to_f32(in.v[i]);
      a = fmaxf(a, fabsf(f[i]));
    }
    a = fmaxf(a, __shfl_xor_sync(pair, a, 1));
    const float d32 = __fdiv_rn(a, 127.0f);
    uint32_t w[kElems / 4] = {};
    if (d32 > 0.0f) {
#pragma unroll
      for (int i = 0; i < kElems; ++i) {
        int q = __float2int_rn(__fdiv_rn(f[i], d32));
        q = max(-127, min(127, q));
        w[i >> 2] |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * (i & 3));
      }
    }
    if (x.at < 0) continue;
    *reinterpret_cast<uint4*>((x.is_v ? vc : kc) + x.cached) = make_uint4(w[0], w[1], w[2], w[3]);
    if ((t & 1) == 0) (x.is_v ? vs : ks)[x.cached / 32] = __float2half_rn(d32);
  }
}

template <typename T>
__device__ __forceinline__ void read_piece(const uint4 q, float d, T* dst) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  dev::Vec<T, kElems> out;
#pragma unroll
  for (int i = 0; i < kElems; ++i) {
    // 0x4B0000bb is 2^23 + code + 128.  code * scale has at most 18
    // significant bits: exact in fp32, rounded once
    const uint32_t u = __byte_perm(w[i >> 2] ^ 0x80808080u, 0x4B000000u, 0x7440 + (i & 3));
    out.v[i] = dev::from_f32<T>((__uint_as_float(u) - 8388736.0f) * d);
  }
  *reinterpret_cast<dev::Vec<T, kElems>*>(dst) = out;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
kv_read_kernel(const Paged p, int rpc, const int8_t* __restrict__ kc, const __half* __restrict__ ks,
               const int8_t* __restrict__ vc, const __half* __restrict__ vs, T* __restrict__ k,
               int64_t k_stride, T* __restrict__ v, int64_t v_stride) {
  __shared__ int64_t place[kMaxRows];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = find_places(p, rpc, place);
  // four pieces' loads in flight before the first is used
  for (int t0 = threadIdx.x; t0 < n; t0 += 4 * kThreads) {
    uint4 q[4];
    __half d[4];
    T* dst[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + i * kThreads;
      dst[i] = nullptr;
      if (t < n) {
        const Piece x = piece_of(p, place, blockIdx.x * rpc, t);
        if (x.at >= 0) {
          dst[i] = (x.is_v ? v + x.row * v_stride : k + x.row * k_stride) + x.elem;
          q[i] = __ldcs(reinterpret_cast<const uint4*>((x.is_v ? vc : kc) + x.cached));
          d[i] = (x.is_v ? vs : ks)[x.cached / 32];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (dst[i] != nullptr) read_piece(q[i], __half2float(d[i]), dst[i]);
  }
}

Paged paged_of(const nvq_kv_cache& c, const KvBatch& b) {
  return {b.cu_seqlens, b.seq_lens, b.block_table, static_cast<int>(b.B), static_cast<int>(b.rows),
          static_cast<int>(b.max_pages), static_cast<int>(c.n_pages), static_cast<int>(c.page_size),
          static_cast<int>(c.n_kv_heads), c.head_dim == 64 ? 6 : 7,
          static_cast<int>(2 * c.n_kv_heads * c.head_dim / kElems)};
}

// Rows per CTA, one per warp at most: the look-ups of a row's place are a
// chain of four loads, so a CTA makes several at once, but few rows are
// spread over the SMs.
int rows_per_cta(const KvBatch& b) {
  const int64_t r = b.rows / (4 * static_cast<int64_t>(device_sm_count()));
  return static_cast<int>(r < 1 ? 1 : r > kMaxRows ? kMaxRows : r);
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
  const int rpc = rows_per_cta(b);
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
  const int rpc = rows_per_cta(b);
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
