// Prompt attention: packed sequences, grouped heads, causal or not.
//
// Query i of a sequence (n queries, m keys) sees the keys j < m, with
// `causal` only j <= i + m - n (the queries are the last n positions):
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q.k_j - max);
// a query that sees no key gives 0.  One pass over the keys with a running
// maximum and sum.
//
// Two bounds are equally near at head_dim 128: a block of 128 queries and 128
// keys takes the tensor core 2 x 512 cycles (S = Q K^T and O += P V) and the
// special-function units 1024 cycles (16384 exponentials at 16 a cycle).  So
// a persistent CTA per SM works on two query tiles at once, and each tile has
// two S buffers of 64 keys: while the exponentials of one are formed the tensor
// core has the other, and the other tile's.
//
//   warps 0-3   softmax of tile 0, one thread per query row: read S from
//               tensor memory, write P = exp2(..) over it as the left operand
//               of the next product; at the end O / sum -> out
//   warps 4-7   the same for tile 1
//   warps 8, 9  issue the MMAs of tile 0 and of tile 1: O += P V of a buffer,
//               then the S of two steps later into it.  One issuing thread takes
//               about as long for a small MMA as the tensor core for one of
//               N = 128, so each tile has its own
//   warp 10     TMA: both Q tiles, then K and V blocks of 128 keys into a ring
//   warp 11     cleans V blocks that some query does not see all of (below)
//
// The two tiles share K and V: two heads of one key-value head with the same
// 128 queries where the group is even, else 256 queries of one head.  Work
// items are (sequence, tile, heads), the later tiles of a sequence (more
// keys) first, dealt to the CTAs forwards and backwards in turn.
//
// The running maximum is a reference point only: the maximum of the first step
// with a finite score, kept while no later step's exponentials add up to more
// than 2^8 times the reference's (then none of them is above that).  So a step costs no search for its maximum and no
// rescaling of O; where a row passes the mark, its warp searches, waits for the
// product before, rescales O and forms the step again.
//
// A key behind a query's last one gets p = 0, but 0 * NaN is not 0: before a
// block with such keys is used, its rows of V behind the sequence's end are
// zeroed in shared memory, and NaN and infinities in rows that only some of
// the queries see are replaced by 0 and added to those queries' results at
// the end.  A warp of its own does it ahead of the products; done by the
// softmax warps, 2048 tokens of 40 heads took 80 us instead of 71.
//
// Measured, cold L2: 8192 tokens, 40 over 8 heads of 128, bf16, causal, 625
// to 640 us by machine (1075 to 1100 TFLOP/s; 710 to 730 back to back, at the
// power limit); 2048 tokens, 40 heads, fp16, 68 to 70 us.
#include <algorithm>
#include <climits>
#include <mutex>
#include <type_traits>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "nvq_device.cuh"
#include "nvq_internal.h"
#include "tcgen05.cuh"

namespace nvq {
namespace {

constexpr int kTile = 128;           // queries of a tile, keys of a block
constexpr int kStep = 64;            // keys of a step: half a block
constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kLoadWarp = 10, kCleanWarp = 11;
constexpr int kRaw = 4;              // V blocks on their way to be cleaned (the ring holds no more)
constexpr uint64_t kWaitLimitNs = 4000000000ull;
// How far a step's exponentials may add up before the reference moves.  With
// fp16 they are 2^7 times as large, so that probabilities down to 2^-32 of the
// reference's count instead of 2^-25: behind one key that stands out, 100000 keys
// of 2^-25 are 0.3 % of the sum.  With bf16 they are 2^-24 times as large: the
// products with its largest values then add up below fp32's largest number.
constexpr float kLazy = 256.0f;
template <bool BF16> constexpr float kShift = BF16 ? -24.0f : 7.0f;                  // a power of two
template <bool BF16> constexpr float kMark = kLazy * (BF16 ? 0x1p-24f : 0x1p7f);    // fp16: below 65504
constexpr float kLarge = 1024.0f;     // exponents from here on are formed as differences first

__device__ unsigned int g_attn_prefill_error_flags = 0;   // bit 0: a wait timed out, bit 1: a bad index

template <int D>
struct Cfg {
  static constexpr int kSub = kTile * 128;              // a 64-wide, 128-byte swizzled sub-tile
  static constexpr int kSubs = D / 64;
  static constexpr int kBlock = kSubs * kSub;           // bytes of a Q tile, K or V block
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kOffRing = 2 * kBlock;
  static constexpr int kOffBars = kOffRing + kStages * kBlock;
  static constexpr int kBars = 2 * kStages + 2 + 4 + 4 + 2 + 2 + 1 + kRaw;
  static constexpr int kOffMisc = kOffBars + 8 * kBars;
  static constexpr int kSmem = kOffMisc + 16 + 1024;
};

struct Args {
  const void* v;
  void* out;
  int64_t v_stride, out_stride;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int B, total_q, total_k, group, heads, pairs, max_items;
  float scale_log2;
  int causal, two_heads;
};

// One item: a sequence's rows, and what each of its two tiles does.
struct Item {
  int q0, n, k0, m;          // packed rows of the sequence: queries, keys
  int row[2], head[2];       // first query and head of each tile
  int steps[2];              // steps of 64 keys of each (0: it sees none)
  bool on[2];                // whether the tile has queries
  int clean_from;            // the first key that some query does not see
  int scan = 0, before = 0;  // where the search for the next one starts: sequence, tiles before it
  __device__ int blocks() const { return (max(steps[0], steps[1]) + 1) / 2; }   // K and V blocks loaded
  // keys that query i (of the sequence) sees
  __device__ int limit(int i, int causal) const { return causal ? min(m, i + m - n + 1) : m; }
};

__device__ __forceinline__ void sequence(const Args& a, int b, int& q0, int& n, int& k0, int& m) {
  q0 = a.cu_q[b];
  int q1 = a.cu_q[b + 1], k1 = a.cu_k[b + 1];
  k0 = a.cu_k[b];
  if (q0 < 0 || q1 < q0 || q1 > a.total_q || k0 < 0 || k1 < k0 || k1 > a.total_k) {
    // no keys; the rows that lie inside give zeros
    atomicOr(&g_attn_prefill_error_flags, 2u);
    q0 = min(max(q0, 0), a.total_q);
    q1 = min(max(q1, q0), a.total_q);
    k0 = k1 = 0;
  }
  n = q1 - q0;
  m = k1 - k0;
}

// Item of this CTA's turn t: every second round is dealt backwards, so that no
// CTA always gets the longest of a round.
__device__ __forceinline__ int item_of(int t) {
  const int G = gridDim.x;
  return t * G + (t & 1 ? G - 1 - static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x));
}
// The item's sequence, tile and heads; the whole warp calls.  false: there is
// no such item.
__device__ __forceinline__ bool find_item(const Args& a, int x, int lane, Item& it) {
  const int rows = a.two_heads ? kTile : 2 * kTile;
  // a CTA's items come in order, so the search goes on where it was
  for (int& b0 = it.scan; b0 < a.B; b0 += 32) {
    int q0 = 0, n = 0, k0 = 0, m = 0;
    if (b0 + lane < a.B) sequence(a, b0 + lane, q0, n, k0, m);
    const int tiles = (n + rows - 1) / rows;
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    const int at = x / a.pairs - it.before;
    const unsigned hit = __ballot_sync(0xffffffffu, incl > at);
    if (hit != 0) {
      const int src = __ffs(hit) - 1;
      it.q0 = __shfl_sync(0xffffffffu, q0, src);
      it.n = __shfl_sync(0xffffffffu, n, src);
      it.k0 = __shfl_sync(0xffffffffu, k0, src);
      it.m = __shfl_sync(0xffffffffu, m, src);
      // the sequence's later tiles first
      const int tile = __shfl_sync(0xffffffffu, incl, src) - 1 - at;
      const int pair = x % a.pairs;
      it.clean_from = INT_MAX;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        it.row[s] = a.two_heads ? tile * kTile : (2 * tile + s) * kTile;
        it.head[s] = a.two_heads ? 2 * pair + s : pair;
        it.on[s] = it.row[s] < it.n;
        const int last_row = min(it.row[s] + kTile, it.n) - 1;
        it.steps[s] = it.on[s] ? (max(0, it.limit(last_row, a.causal)) + kStep - 1) / kStep : 0;
        if (it.steps[s] > 0) it.clean_from = min(it.clean_from, max(0, it.limit(it.row[s], a.causal)));
      }
      return true;
    }
    it.before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// D[tmem] (+)= A[smem] * B[smem]^T, kind::f16.
__device__ __forceinline__ void mma_f16_ss(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Descriptor of a right operand stored with its columns contiguous (MN-major,
// V as it lies): 64 columns in a 128-byte swizzled row, 8-row groups 1024
// bytes apart (stride offset), the next 64 columns a sub-tile further on
// (leading offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr, uint32_t sub_bytes) {
  uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(sub_bytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// Wait for this thread's tensor-memory loads; the values pass through, so
// that nothing that uses them moves in front of the wait.
__device__ __forceinline__ void wait_ld_32(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                 "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                 "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                 "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void wait_ld_16(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}
// Pairs of fp32 values in one instruction.
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float2 split2(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// The largest of three; NaN if one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 32 bytes, a whole sector, from one lane.
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  return dev::h2_bits(__floats2half2_rn(lo, hi));
}

// One warp: rows `from`.. of a V block in shared memory; those from `end` on are
// set to zero, in the others NaN and infinities.  Returns whether this lane
// met one.  Eight lanes take a row of 128 bytes; the swizzle only permutes it.
template <int SUBS, bool BF16>
__device__ __noinline__ bool clean_values(unsigned char* block, int sub_bytes, int from, int end, int lane) {
  constexpr uint32_t kExp = BF16 ? 0x7F807F80u : 0x7C007C00u, kOne = BF16 ? 0x00800080u : 0x04000400u;
  bool any = false;
  // whole rows of zeros first, then the check, several loads in flight
  for (int row = max(from, end) + (lane >> 3); row < kTile; row += 4)
#pragma unroll
    for (int i = 0; i < SUBS; ++i)
      reinterpret_cast<uint4*>(block + i * sub_bytes + row * 128)[lane & 7] = make_uint4(0, 0, 0, 0);
  constexpr int kBatch = 4;
  for (int row0 = from + (lane >> 3); row0 < min(end, kTile); row0 += 4 * kBatch) {
    uint4 w[kBatch][SUBS];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
#pragma unroll
      for (int i = 0; i < SUBS; ++i) {
        const int row = row0 + 4 * k;
        w[k][i] = row < min(end, kTile) ? reinterpret_cast<const uint4*>(block + i * sub_bytes + row * 128)[lane & 7]
                                        : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
#pragma unroll
      for (int i = 0; i < SUBS; ++i) {
        uint32_t u[4] = {w[k][i].x, w[k][i].y, w[k][i].z, w[k][i].w}, hits = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) hits |= ((u[e] & kExp) + kOne) & 0x80008000u;     // exponent all ones
        if (hits != 0) {
          any = true;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t hit = ((u[e] & kExp) + kOne) & 0x80008000u;
            if (hit & 0x8000u) u[e] &= 0xFFFF0000u;
            if (hit & 0x80000000u) u[e] &= 0x0000FFFFu;
          }
          reinterpret_cast<uint4*>(block + i * sub_bytes + (row0 + 4 * k) * 128)[lane & 7] = make_uint4(u[0], u[1], u[2], u[3]);
        }
      }
  }
  return any;
}

// The whole warp waits (one lane then acts; see the prefill GEMM).  The limit
// holds from the last block that was loaded on: a warp may wait through any
// number of items that need nothing of it (the cleaner through those without
// unseen keys, a tile's softmax through those with one tile).  The blocks are
// counted in `issued`, so the waits still end.  false, and the flag: no block
// came for the limit, or another warp gave up.
__device__ __forceinline__ bool counted_wait(uint32_t bar, uint32_t parity, volatile int* issued,
                                             volatile int* abort_flag, uint64_t limit_ns) {
  if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
  for (int before = __shfl_sync(0xffffffffu, *issued, 0);;) {
    const bool got = ptx::mbar_wait_bounded(bar, parity, abort_flag, limit_ns);
    if (__all_sync(0xffffffffu, got)) return true;
    const int now = __shfl_sync(0xffffffffu, *issued, 0);
    if (now == before || __any_sync(0xffffffffu, *abort_flag != 0)) break;
    before = now;
  }
  *abort_flag = 1;
  atomicOr(&g_attn_prefill_error_flags, 1u);
  return false;
}

// Test-only: warp 0 waits as above for a phase that warp 1 completes after two
// limits, having counted a block every half of one (`moving`), or never.
__global__ void __launch_bounds__(64) stalled_attn_wait_kernel(uint64_t limit_ns, int moving, int* result) {
  __shared__ __align__(8) uint64_t bar_s;
  __shared__ int issued_s, abort_s;
  volatile int* issued = &issued_s;
  volatile int* abort_flag = &abort_s;
  const uint32_t bar = ptx::smem_addr(&bar_s);
  if (threadIdx.x == 0) {
    ptx::mbar_init(bar, 1);
    *issued = *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  const uint64_t t0 = ptx::globaltimer_ns();
  if (threadIdx.x < 32) {
    const bool got = counted_wait(bar, 0, issued, abort_flag, limit_ns);
    const uint64_t us = (ptx::globaltimer_ns() - t0) / 1000;
    if (threadIdx.x == 0) {
      result[0] = got ? 1 : 0;
      result[1] = us > 0x7fffffffull ? 0x7fffffff : static_cast<int>(us);
    }
  } else if (moving && threadIdx.x == 32) {
    for (int r = 1; r <= 4; ++r) {
      // at most 2^21 sleeps of a microsecond, whatever the clock says
      for (int i = 0; i < (1 << 21) && ptx::globaltimer_ns() - t0 < r * limit_ns / 2; ++i) __nanosleep(1000);
      *issued = r;
    }
    ptx::mbar_arrive(bar);
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
attn_prefill_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                    const __grid_constant__ CUtensorMap v_map, const Args a) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw);
  unsigned char* smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
  const uint32_t base = ptx::smem_addr(smem);
  auto bar = [&](int i) { return base + C::kOffBars + 8u * i; };
  auto kv_full = [&](int s) { return bar(s); };
  auto kv_empty = [&](int s) { return bar(C::kStages + s); };
  const uint32_t q_full = bar(2 * C::kStages), q_empty = bar(2 * C::kStages + 1);
  auto s_full = [&](int s, int b) { return bar(2 * C::kStages + 2 + 2 * s + b); };
  auto p_full = [&](int s, int b) { return bar(2 * C::kStages + 6 + 2 * s + b); };
  auto o_done = [&](int s) { return bar(2 * C::kStages + 10 + s); };
  auto o_full = [&](int s) { return bar(2 * C::kStages + 12 + s); };
  const uint32_t mma_done = bar(2 * C::kStages + 14);
  auto v_raw = [&](int i) { return bar(2 * C::kStages + 15 + i % kRaw); };
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  volatile int* issued = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
  volatile int* found = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 12);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(kv_full(s), 1);
      ptx::mbar_init(kv_empty(s), 2);      // both tiles
    }
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(q_empty, 2);
    for (int s = 0; s < 2; ++s) {
      for (int b = 0; b < 2; ++b) {
        ptx::mbar_init(s_full(s, b), 1);
        ptx::mbar_init(p_full(s, b), 4);
      }
      ptx::mbar_init(o_done(s), 1);
      ptx::mbar_init(o_full(s), 1);
    }
    ptx::mbar_init(mma_done, 2);
    for (int i = 0; i < kRaw; ++i) ptx::mbar_init(v_raw(i), 1);
    *abort_flag = 0;
    *issued = 0;
    *found = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&q_map);
    ptx::prefetch_tensormap(&k_map);
    ptx::prefetch_tensormap(&v_map);
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_addr(tmem_holder), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  auto warp_wait = [&](uint32_t b, uint32_t parity) -> bool {
    return counted_wait(b, parity, issued, abort_flag, kWaitLimitNs);
  };
  // tensor memory: S (and P) of tile s, buffer b at 128 s + 64 b, O at 256 + 128 s

  if (warp == kLoadWarp) {
    // --------------------------------- copies ---------------------------------
    int g = 0;                 // K and V blocks issued
    int raws = 0;              // V blocks to be cleaned
    bool ok = true;
    Item it;
    // a V block to be cleaned is announced to the warp that does it, which
    // announces it as full
    auto block = [&](const CUtensorMap* map, int col, int row, bool clean) {
      const int s = g % C::kStages;
      if (!warp_wait(kv_empty(s), ((g / C::kStages) & 1) ^ 1)) return false;
      if (lane == 0) {
        const uint32_t b = clean ? v_raw(raws) : kv_full(s);
        ptx::mbar_arrive_expect_tx(b, C::kBlock);
        for (int i = 0; i < C::kSubs; ++i)
          ptx::tma_load_2d(base + C::kOffRing + s * C::kBlock + i * C::kSub, map, col + 64 * i, row, b);
        *issued = g + 1;
      }
      __syncwarp();
      ++g;
      raws += clean;
      return true;
    };
    int items = 0;
    for (int t = 0, x; ok && (x = item_of(t), t * static_cast<int>(gridDim.x) < a.max_items); ++t) {
      if (!find_item(a, x, lane, it) || it.blocks() == 0) continue;
      ok = warp_wait(q_empty, (items & 1) ^ 1);
      if (!ok) break;
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(q_full, (it.steps[0] > 0 ? C::kBlock : 0) + (it.steps[1] > 0 ? C::kBlock : 0));
#pragma unroll
        for (int s = 0; s < 2; ++s)
          if (it.steps[s] > 0)
            for (int i = 0; i < C::kSubs; ++i)
              ptx::tma_load_2d(base + s * C::kBlock + i * C::kSub, &q_map, it.head[s] * D + 64 * i, it.q0 + it.row[s], q_full);
      }
      __syncwarp();
      ++items;
      const int col = it.head[0] / a.group * D;
      for (int j = 0; ok && j < it.blocks(); ++j)
        ok = block(&k_map, col, it.k0 + j * kTile, false) &&
             block(&v_map, col, it.k0 + j * kTile, (j + 1) * kTile > it.clean_from);
    }
    if (*abort_flag) {
      // the MMAs may have stopped: wait for the copies in flight
      if (items > 0) ptx::mbar_wait_bounded(q_full, (items - 1) & 1, nullptr, kWaitLimitNs);
      for (int i = max(0, raws - kRaw); i < raws; ++i)
        ptx::mbar_wait_bounded(v_raw(i), (i / kRaw) & 1, nullptr, kWaitLimitNs);
      for (int i = max(0, g - C::kStages); i < g; ++i)
        ptx::mbar_wait_bounded(kv_full(i % C::kStages), (i / C::kStages) & 1, nullptr, kWaitLimitNs);
    }
  } else if (warp == kCleanWarp) {
    // ------------------------ V blocks with unseen keys ------------------------
    int g = 0, items = 0, raws = 0;
    bool ok = true;
    Item it;
    for (int t = 0, x; ok && (x = item_of(t), t * static_cast<int>(gridDim.x) < a.max_items); ++t) {
      if (!find_item(a, x, lane, it) || it.blocks() == 0) continue;
      for (int j = max(0, it.clean_from / kTile); ok && j < it.blocks(); ++j) {
        const int v = g + 2 * j + 1;
        ok = warp_wait(v_raw(raws), (raws / kRaw) & 1);
        ++raws;
        if (!ok) break;
        const bool met = clean_values<C::kSubs, BF16>(smem + C::kOffRing + (v % C::kStages) * C::kBlock, C::kSub,
                                                      max(0, it.clean_from - j * kTile), it.m - j * kTile, lane);
        // the number of the last such item, however far ahead: an item before
        // it then looks for values to add back and, where it has none, adds none
        if (met) *found = items + 1;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(kv_full(v % C::kStages));
      }
      g += 2 * it.blocks();
      ++items;
    }
  } else if (warp >= kMmaWarp) {
    // ------------------------------ MMAs of tile s ------------------------------
    constexpr uint32_t kFmt = BF16 ? (1u << 7) | (1u << 10) : 0u;
    constexpr uint32_t idesc_s = ptx::idesc_f16_f32(kTile, kStep) | kFmt;
    constexpr uint32_t idesc_o = ptx::idesc_f16_f32(kTile, D) | kFmt | (1u << 16);   // V: columns contiguous
    const int s = warp - kMmaWarp;
    const uint32_t t_s = tmem + 128 * s, t_o = tmem + 256 + 128 * s;
    const uint64_t q = ptx::sw128_kmajor_desc(base + s * C::kBlock);
    int g = 0, items = 0;
    uint32_t p_par = 0;          // parity of each buffer's next P
    bool ok = true;
    Item it;
    auto ring = [&](int i) { return base + C::kOffRing + (i % C::kStages) * C::kBlock; };
    auto wait_block = [&](int i) { return warp_wait(kv_full(i % C::kStages), (i / C::kStages) & 1); };
    for (int t = 0, x; ok && (x = item_of(t), t * static_cast<int>(gridDim.x) < a.max_items); ++t) {
      if (!find_item(a, x, lane, it) || it.blocks() == 0) continue;
      const int N = it.blocks(), steps = s ? it.steps[1] : it.steps[0];
      ok = warp_wait(q_full, items & 1);
      if (!ok) break;
      auto scores = [&](int i) {       // S of step i
        const int k = g + (i & ~1);
        if (!(i & 1) && !wait_block(k)) return false;
        if (lane == 0) {
          ptx::tc_fence_after();
          const uint64_t kd = ptx::sw128_kmajor_desc(ring(k) + (i & 1) * kStep * 128);
#pragma unroll
          for (int e = 0; e < D / 16; ++e) {
            const uint32_t off = ((e / 4) * C::kSub + (e % 4) * 32) >> 4;
            mma_f16_ss(t_s + kStep * (i & 1), q + off, kd + off, idesc_s, e > 0);
          }
          ptx::mma_commit(s_full(s, i & 1));
          if ((i & 1) || i + 1 == steps) ptx::mma_commit(kv_empty(k % C::kStages));
          if (i + 1 == steps) ptx::mma_commit(q_empty);
        }
        __syncwarp();
        return true;
      };
      if (steps > 0) ok = scores(0);
      if (ok && steps > 1) ok = scores(1);
      for (int i = 0; ok && i < steps; ++i) {
        const int v = g + (i | 1), b = i & 1;
        ok = (b || wait_block(v)) && warp_wait(p_full(s, b), (p_par >> b) & 1);
        if (!ok) break;
        p_par ^= 1u << b;
        if (lane == 0) {
          ptx::tc_fence_after();
          const uint64_t vd = sw128_mnmajor_desc(ring(v) + b * kStep * 128, C::kSub);
#pragma unroll
          for (int e = 0; e < kStep / 16; ++e)
            ptx::mma_f16_ts(t_o, t_s + kStep * b + 8 * e, vd + ((e * 16 * 128) >> 4), idesc_o, i > 0 || e > 0);
          ptx::mma_commit(o_done(s));                       // every step, and
          if (i + 1 == steps) ptx::mma_commit(o_full(s));   // every item
          if (b || i + 1 == steps) ptx::mma_commit(kv_empty(v % C::kStages));
        }
        __syncwarp();
        if (i + 2 < steps) ok = scores(i + 2);
      }
      // blocks that only the other tile uses
      for (int i = g + 2 * ((steps + 1) / 2); ok && i < g + 2 * N; ++i) {
        ok = wait_block(i);
        if (ok && lane == 0) ptx::mbar_arrive(kv_empty(i % C::kStages));
        __syncwarp();
      }
      if (ok && steps == 0 && lane == 0) ptx::mbar_arrive(q_empty);
      g += 2 * N;
      ++items;
    }
    // no MMA may still use shared or tensor memory when they are released
    if (lane == 0) ptx::mma_commit(mma_done);
    __syncwarp();
    ptx::mbar_wait_bounded(mma_done, 0, nullptr, kWaitLimitNs);
  } else {
    // --------------------------------- softmax ---------------------------------
    const int s = warp >> 2;                       // tile
    const int r = threadIdx.x & 127;               // row of the tile
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + 128 * s, t_o = tmem + lanes + 256 + 128 * s;
    const float c = a.scale_log2;
    const bool sectors = ((reinterpret_cast<uintptr_t>(a.out) | (2 * a.out_stride)) & 31) == 0;
    int items = 0;
    uint32_t s_par = 0;                            // parity of each buffer's next S
    int sent = 0, o_count = 0;                     // steps handed on, results taken, over all items
    bool ok = true;
    Item it;
    for (int t = 0, x; ok && (x = item_of(t), t * static_cast<int>(gridDim.x) < a.max_items); ++t) {
      if (!find_item(a, x, lane, it)) continue;
      const int item = items;
      if (it.blocks() > 0) ++items;
      // this tile's values (selected, so that they stay in registers)
      if (!(s ? it.on[1] : it.on[0])) continue;
      const int row = (s ? it.row[1] : it.row[0]) + r;       // query of the sequence
      const int steps = s ? it.steps[1] : it.steps[0], head = s ? it.head[1] : it.head[0];
      const int limit = it.limit(row, a.causal);
      float ref = 0.0f, l = 0.0f;                  // reference (a score); sum
      bool fresh = limit > 0;                      // no reference yet
      for (int i = 0; ok && i < steps; ++i) {
        const int b = i & 1;
        ok = warp_wait(s_full(s, b), (s_par >> b) & 1);
        if (!ok) break;
        s_par ^= 1u << b;
        ptx::tc_fence_after();
        const int seen = limit - i * kStep;        // keys of the step that the row sees
        uint32_t v[2][32];
        ptx::tmem_ld_32cols(t_s + kStep * b, v[0]);
        ptx::tmem_ld_32cols(t_s + kStep * b + 32, v[1]);
        wait_ld_32(v[0]);
        wait_ld_32(v[1]);
        // rows see more keys the later they are: lane 0 the fewest, and only
        // the columns that it does not see are looked at
        const int least = __shfl_sync(0xffffffffu, seen, 0);
        if (least < kStep) {
#pragma unroll
          for (int q = 0; q < kStep; q += 8)
            if (least < q + 8) {
#pragma unroll
              for (int e = q; e < q + 8; ++e)
                if (e >= seen) v[e / 32][e % 32] = 0xFF800000u;       // -infinity
            }
        }
        // the step's maximum (NaN if a score is); it is not needed as a rule
        auto largest = [&]() -> float {
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < kStep; e += 2)
            top[e / 2 % 4] = max3_nan(top[e / 2 % 4], __uint_as_float(v[e / 32][e % 32]), __uint_as_float(v[e / 32][e % 32 + 1]));
          return max3_nan(max3_nan(top[0], top[1], top[2]), top[3], top[3]);
        };
        // the first step with a score above -infinity has a row's reference
        if (__any_sync(0xffffffffu, fresh)) {
          const float top = largest();
          if (fresh && !(top == -INFINITY)) {
            if (fabsf(top) < INFINITY) ref = top;
            fresh = false;
          }
        }
        // The exponentials against the reference, and their sum.  Where a row's
        // scores are large the difference comes first: it is exact near the
        // maximum.  Each row goes by its own reference (fma(x + -0, c, n) is
        // fma(x, c, n)), so that no other row of the warp changes its bits.
        auto form = [&](auto large) -> float {
          F2 sum0 = f2(0.0f), sum1 = f2(0.0f);
          const bool own = decltype(large)::value && fabsf(ref * c) > kLarge;
          const F2 m2 = f2(own ? -ref : -0.0f), n2 = f2(own ? kShift<BF16> : fmaf(-ref, c, kShift<BF16>)), c2 = f2(c);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const F2 x = f2(__uint_as_float(v[h][e]), __uint_as_float(v[h][e + 1]));
              const float2 u = split2(fma2(decltype(large)::value ? add2(x, m2) : x, c2, n2));
              const float2 y = make_float2(exp2_approx(u.x), exp2_approx(u.y));
              (e & 2 ? sum1 : sum0) = add2(e & 2 ? sum1 : sum0, f2(y.x, y.y));
              p[e / 2] = pack2<BF16>(y.x, y.y);
            }
            ptx::tmem_st_16cols(t_s + kStep * b + 16 * h, p);
          }
          const float2 sum = split2(add2(sum0, sum1));
          return sum.x + sum.y;
        };
        using Yes = std::integral_constant<bool, true>;
        using No = std::integral_constant<bool, false>;
        // No exponential is above their sum: while that stays below 2^8 the
        // reference may lag.  Else (NaN among them) the step's maximum becomes
        // the reference, and the step is formed again.
        float sum;
        for (int round = 0;; ++round) {
          sum = __any_sync(0xffffffffu, fabsf(ref * c) > kLarge) ? form(Yes{}) : form(No{});
          const bool grow = !(sum <= kMark<BF16>);
          if (round > 0 || !__any_sync(0xffffffffu, grow)) break;
          ptx::tmem_wait_st();       // stores to one place are not kept in order by themselves
          const float top = largest();
          const float f = grow ? exp2_approx((ref - top) * c) : 1.0f;
          if (grow) ref = top;
          l *= f;
          if (i > 0) {
            // O holds the steps before, once the last of their products is
            // done (the one before that is: this S was formed after it)
            ok = warp_wait(o_done(s), (sent - 1) & 1);
            if (!ok) break;
            ptx::tc_fence_after();
#pragma unroll
            for (int q = 0; q < D / 16; ++q) {
              uint32_t w[16];
              ptx::tmem_ld_16cols(t_o + 16 * q, w);
              wait_ld_16(w);
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * f);
              ptx::tmem_st_16cols(t_o + 16 * q, w);
            }
          }
        }
        if (!ok) break;
        l += sum;
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(p_full(s, b));
        ++sent;
      }
      if (!ok) break;
      // -------- the tile's results
      const bool some = steps > 0;
      if (some) {
        ok = warp_wait(o_full(s), o_count++ & 1);
        if (!ok) break;
        ptx::tc_fence_after();
      }
      const float inv = l > 0.0f ? __fdividef(1.0f, l) : l;       // nothing seen: 0; NaN stays
      const bool patch = some && *found > item;
      using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
      T* out = static_cast<T*>(a.out) + (static_cast<int64_t>(it.q0) + row) * a.out_stride + head * D;
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t v[32];
        if (some) {
          ptx::tmem_ld_32cols(t_o + 32 * q, v);
          wait_ld_32(v);
        }
        float e[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) e[i] = some && l != 0.0f ? __uint_as_float(v[i]) * inv : 0.0f;
        if (patch) {
          // the NaN and infinities that this row sees among the cleaned keys
          for (int k = it.clean_from; k < limit; ++k) {
            const T* src = static_cast<const T*>(a.v) + (static_cast<int64_t>(it.k0) + k) * a.v_stride +
                           head / a.group * D + 32 * q;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float f = dev::to_f32(src[i]);
              if (!(fabsf(f) <= 3.4e38f)) e[i] += f;
            }
          }
        }
        if (row < it.n) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack2<BF16>(e[2 * i], e[2 * i + 1]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // a lane's row is its own, so every store goes to 32 places: whole
            // sectors where the rows allow it
            if (sectors) {
              const uint32_t x8[8] = {w[8 * h], w[8 * h + 1], w[8 * h + 2], w[8 * h + 3],
                                      w[8 * h + 4], w[8 * h + 5], w[8 * h + 6], w[8 * h + 7]};
              store32(out + 32 * q + 16 * h, x8);
            } else {
              uint4* to = reinterpret_cast<uint4*>(out + 32 * q + 16 * h);
              to[0] = make_uint4(w[8 * h], w[8 * h + 1], w[8 * h + 2], w[8 * h + 3]);
              to[1] = make_uint4(w[8 * h + 4], w[8 * h + 5], w[8 * h + 6], w[8 * h + 7]);
            }
          }
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, 512);
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Packed rows as [rows][width] 16-bit elements, boxes of 64 columns and 128 rows.
bool row_map(CUtensorMap* map, const void* p, int64_t rows, int64_t width, int64_t stride, bool bf16) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[2] = {64, kTile};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BF16>
cudaError_t prefill_t(const PrefillArgs& p, cudaStream_t stream) {
  using C = Cfg<D>;
  CUtensorMap q_map, k_map, v_map;
  const bool keys = p.total_k > 0;      // without any, no key is loaded
  if (!row_map(&q_map, p.q, p.total_q, p.heads * D, p.q_stride, BF16) ||
      !row_map(&k_map, keys ? p.k : p.q, keys ? p.total_k : 1, keys ? p.kv_heads * D : D, keys ? p.k_stride : D, BF16) ||
      !row_map(&v_map, keys ? p.v : p.q, keys ? p.total_k : 1, keys ? p.kv_heads * D : D, keys ? p.v_stride : D, BF16))
    return cudaErrorInvalidValue;
  static SmemAttrOnce attr;
  cudaError_t e = attr.ensure(attn_prefill_kernel<D, BF16>, C::kSmem);
  if (e != cudaSuccess) return e;
  Args a = {};
  a.v = p.v;
  a.out = p.out;
  a.v_stride = p.v_stride;
  a.out_stride = p.out_stride;
  a.cu_q = p.cu_q;
  a.cu_k = p.cu_k;
  a.B = static_cast<int>(p.B);
  a.total_q = static_cast<int>(p.total_q);
  a.total_k = static_cast<int>(p.total_k);
  a.heads = static_cast<int>(p.heads);
  a.group = static_cast<int>(p.heads / p.kv_heads);
  a.two_heads = a.group % 2 == 0;
  a.pairs = a.two_heads ? a.heads / 2 : a.heads;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.causal = p.causal != 0;
  // at most one ragged tile per sequence
  const int64_t rows = a.two_heads ? kTile : 2 * kTile;
  const int64_t items = (p.total_q / rows + p.B) * a.pairs;
  if (items > INT32_MAX / 2) return cudaErrorInvalidValue;
  a.max_items = static_cast<int>(items);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(device_sm_count(), items)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_prefill_kernel<D, BF16>, q_map, k_map, v_map, a);
}

}  // namespace

cudaError_t launch_attn_prefill(const PrefillArgs& a, int dtype, cudaStream_t stream) {
  if (a.head_dim == 64)
    return dtype == NVQ_F16 ? prefill_t<64, false>(a, stream) : prefill_t<64, true>(a, stream);
  return dtype == NVQ_F16 ? prefill_t<128, false>(a, stream) : prefill_t<128, true>(a, stream);
}

cudaError_t launch_stalled_attn_wait(uint64_t limit_ns, int moving, int* result, cudaStream_t stream) {
  stalled_attn_wait_kernel<<<1, 64, 0, stream>>>(limit_ns, moving, result);
  return cudaGetLastError();
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
