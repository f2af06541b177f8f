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
// Both kernels have to move e + 1.0625 bytes per value, and are launch-bound for
// a decode step.  The read of many rows is HBM-bound: 80052 rows of 8 x 128 as
// fp16, cold L2, 88 us (5.7 TB/s).  The write is not: 7000 such rows take 25 us
// for 6.6 us of bytes.  A warp's chain of four dependent look-ups, its loads of
// K, K's quantisation and only then V's loads is hidden by the 24 to 40 other
// warps that its registers leave room for on an SM (48 to 76 a thread), in two to
// three waves of CTAs.  Rows of one or two heads leave lanes idle: 12000 rows of
// 1 x 128 in fp16 are written in 18 us (1.5 us of bytes).
#include <cstring>

#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "nvq_internal.h"

namespace nvq {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;      // pieces of a lane whose loads are in flight together

__device__ unsigned int g_kv_error_flags = 0;   // bit 1: a bad index

// Where the rows of a packed batch lie in the pages.
struct Paged {
  const int32_t* cu;       // [B + 1]
  const int32_t* lens;     // [B]
  const int32_t* table;    // [B, max_pages]
  int B, rows, max_pages, n_pages, page, heads, dim_shift;
  int parts;               // warps that share a row
};

// (page * heads * page_size + offset), the token's place for head 0, or -1
// for a row that has none: padding behind the last sequence, or a bad
// length or page (which raises the flag).  The whole warp calls.
__device__ __forceinline__ int64_t warp_place(const Paged& p, int row, int lane) {
  const int b = dev::warp_find_seq(p.cu, p.B, row, lane);
  if (b >= p.B) return -1;
  const int64_t pos = static_cast<int64_t>(p.lens[b]) - p.cu[b + 1] + row;
  int page = -1, off = 0;
  if (pos >= 0 && pos < static_cast<int64_t>(p.max_pages) * p.page) {
    const int col = static_cast<int>(static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.page));   // a length is below 2^31
    off = static_cast<int>(pos) - col * p.page;
    page = p.table[static_cast<int64_t>(b) * p.max_pages + col];
  }
  if (page < 0 || page >= p.n_pages) {
    if (lane == 0) atomicOr(&g_kv_error_flags, 2u);
    return -1;
  }
  return static_cast<int64_t>(page) * p.heads * p.page + off;
}

// A warp's share of a row: the 16-byte pieces of the packed side (4 or 8
// values) lane, lane + 32, .. of K and then of V, so that both sides are
// read and written in whole lines.  The look-up of the row's place is a
// chain of four loads, hidden by the other warps.
template <typename T>
struct Share {
  static constexpr int kElems = 16 / sizeof(T);
  int row, e0, e1;         // elements of K and V of the row: e0 .. e1 - 1
  int64_t at;
  __device__ __forceinline__ bool find(const Paged& p) {
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    row = static_cast<int>(w / p.parts);
    if (row >= p.rows) return false;
    const int part = static_cast<int>(w - static_cast<int64_t>(row) * p.parts);
    // shares are whole warps' pieces (the width is a multiple of 64)
    const int pieces = (p.heads << p.dim_shift) / kElems;
    const int each = (pieces + 32 * p.parts - 1) / (32 * p.parts) * 32;
    e0 = min(part * each, pieces) * kElems;
    e1 = min((part + 1) * each, pieces) * kElems;
    at = warp_place(p, row, lane);
    return at >= 0;
  }
  // the first code of the piece that starts at element e
  __device__ __forceinline__ int64_t code(const Paged& p, int e) const {
    const int h = e >> p.dim_shift;
    return ((at + static_cast<int64_t>(h) * p.page) << p.dim_shift) + (e - (h << p.dim_shift));
  }
};
// kElems codes as one word or two.
template <int N> struct Codes;
template <> struct Codes<4> { using type = uint32_t; };
template <> struct Codes<8> { using type = uint2; };

// Codes of N values with scale d32, rint(x / d32) of the correctly rounded
// quotient: x * (1 / d32) is within 2^-22 of it, relatively, and below 128, so
// where it is not within 2^-14 of a tie it rounds to the same number; else,
// and where the reciprocal may leave the normal range, by the division itself.
// Adding 1.5 * 2^23 rounds to the nearest even whole number and leaves it in
// the low bits, which spares the conversion units.
template <int N>
__device__ __forceinline__ void quantise(const float (&f)[N], float d32, uint32_t (&w)[N / 4]) {
  constexpr float kRound = 12582912.0f;
  const float inv = __frcp_rn(d32);
  bool exact = !(d32 >= 0x1p-100f && d32 <= 0x1p100f);
  uint32_t q[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float t = f[i] * inv, u = t + kRound;
    exact |= fabsf(t - (u - kRound)) > 0.5f - 0x1p-14f;
    q[i] = __float_as_uint(u);
  }
  if (exact) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = max(-127, min(127, __float2int_rn(__fdiv_rn(f[i], d32))));
  }
#pragma unroll
  for (int i = 0; i < N; i += 4)
    w[i / 4] = __byte_perm(__byte_perm(q[i], q[i + 1], 0x0040), __byte_perm(q[i + 2], q[i + 3], 0x0040), 0x5410);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
kv_write_kernel(const Paged p, const T* k, int64_t k_stride, const T* v, int64_t v_stride,
                int8_t* kc, __half* ks, int8_t* vc, __half* vs) {
  constexpr int N = Share<T>::kElems, kLanes = 32 / N;      // lanes of a Q8_0 block
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Share<T> x;
  if (!x.find(p)) return;                 // whole warps leave together
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int is_v = 0; is_v < 2; ++is_v) {
    const T* src = is_v ? v + x.row * v_stride : k + x.row * k_stride;
    int8_t* codes = is_v ? vc : kc;
    __half* scales = is_v ? vs : ks;
    for (int e0 = x.e0 + lane * N; e0 - lane * N < x.e1; e0 += kBatch * 32 * N) {
      dev::Vec<T, N> in[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int e = e0 + i * 32 * N;
        if (e < x.e1) in[i] = *reinterpret_cast<const dev::Vec<T, N>*>(src + e);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int e = e0 + i * 32 * N;
        // the lanes of a block are inside the share together
        const unsigned mask = __ballot_sync(0xffffffffu, e < x.e1);
        if (e >= x.e1) continue;
        float f[N], a = 0.0f;
#pragma unroll
        for (int u = 0; u < N; ++u) {
          f[u] = dev::to_f32(in[i].v[u]);
          a = fmaxf(a, fabsf(f[u]));
        }
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) a = fmaxf(a, __shfl_xor_sync(mask, a, o));
        const float d32 = __fdiv_rn(a, 127.0f);
        uint32_t w[N / 4] = {};
        if (d32 > 0.0f) quantise<N>(f, d32, w);
        const int64_t at = x.code(p, e);
        typename Codes<N>::type word;
        memcpy(&word, w, sizeof(w));
        *reinterpret_cast<typename Codes<N>::type*>(codes + at) = word;
        if (lane % kLanes == 0) scales[at / 32] = __float2half_rn(d32);
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
kv_read_kernel(const Paged p, const int8_t* kc, const __half* ks, const int8_t* vc,
               const __half* vs, T* k, int64_t k_stride, T* v, int64_t v_stride) {
  constexpr int N = Share<T>::kElems;
  using Word = typename Codes<N>::type;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Share<T> x;
  if (!x.find(p)) return;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int is_v = 0; is_v < 2; ++is_v) {
    T* dst = is_v ? v + x.row * v_stride : k + x.row * k_stride;
    const int8_t* codes = is_v ? vc : kc;
    const __half* scales = is_v ? vs : ks;
    for (int e0 = x.e0 + lane * N; e0 < x.e1; e0 += kBatch * 32 * N) {
      Word q[kBatch];
      __half d[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int e = e0 + i * 32 * N;
        if (e < x.e1) {
          const int64_t at = x.code(p, e);
          q[i] = __ldcs(reinterpret_cast<const Word*>(codes + at));
          d[i] = scales[at / 32];
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int e = e0 + i * 32 * N;
        if (e >= x.e1) continue;
        uint32_t w[N / 4];
        memcpy(w, &q[i], sizeof(w));
        const float scale = __half2float(d[i]);
        dev::Vec<T, N> out;
#pragma unroll
        for (int u = 0; u < N; ++u) {
          // 0x4B0000bb is 2^23 + code + 128.  code * scale has at most 18
          // significant bits: exact in fp32, rounded once
          const uint32_t b = __byte_perm(w[u / 4] ^ 0x80808080u, 0x4B000000u, 0x7440 + (u % 4));
          out.v[u] = dev::from_f32<T>((__uint_as_float(b) - 8388736.0f) * scale);
        }
        *reinterpret_cast<dev::Vec<T, N>*>(dst + e) = out;
      }
    }
  }
}

// Warps that share a row: one where there are rows enough for 48 warps per SM,
// more for a decode step's few rows, as far as a warp still has a piece of K and
// of V for each of its lanes.  48 lies between what the two kernels want (24 to
// 40 warps are resident of the write, 64 of the read); us with 24, 48 and 96:
//                                   write               read back
//   4000 rows of 40 x 128, bf16     66   59   60        37   31   31
//   4000 rows of 40 x 128, fp32     59   57   55        55   45   45
//   4000 rows of 8 x 128, fp16      16   18   22        14   12   14
//   7000 rows of 8 x 128, bf16      25   29   39        16   17   21
Paged paged_of(const nvq_kv_cache& c, const KvBatch& b, int elems) {
  const int64_t width = c.n_kv_heads * c.head_dim;
  int parts = 1;
  while (b.rows * parts < 48 * static_cast<int64_t>(device_sm_count()) && 32 * elems * 2 * parts <= width) parts *= 2;
  return {b.cu_seqlens, b.seq_lens, b.block_table, static_cast<int>(b.B), static_cast<int>(b.rows),
          static_cast<int>(b.max_pages), static_cast<int>(c.n_pages), static_cast<int>(c.page_size),
          static_cast<int>(c.n_kv_heads), c.head_dim == 64 ? 6 : 7, parts};
}

cudaLaunchConfig_t config(const Paged& p, cudaStream_t stream, cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int64_t warps = static_cast<int64_t>(p.rows) * p.parts;
  cfg.gridDim = dim3(static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32)));
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
  const Paged p = paged_of(c, b, 16 / sizeof(T));
  const cudaLaunchConfig_t cfg = config(p, stream, &attr);
  return cudaLaunchKernelEx(&cfg, kv_write_kernel<T>, p, static_cast<const T*>(k),
                            k_stride, static_cast<const T*>(v), v_stride, c.k_codes,
                            reinterpret_cast<__half*>(c.k_scales), c.v_codes,
                            reinterpret_cast<__half*>(c.v_scales));
}

template <typename T>
cudaError_t read_t(const nvq_kv_cache& c, const KvBatch& b, void* k, int64_t k_stride, void* v,
                   int64_t v_stride, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  const Paged p = paged_of(c, b, 16 / sizeof(T));
  const cudaLaunchConfig_t cfg = config(p, stream, &attr);
  return cudaLaunchKernelEx(&cfg, kv_read_kernel<T>, p, static_cast<const int8_t*>(c.k_codes),
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
