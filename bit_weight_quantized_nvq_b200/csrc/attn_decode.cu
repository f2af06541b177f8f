// Decode attention over the paged Q8_0 cache: one new token per sequence.
//
//   o[h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q[h].k_j - m),
//   m = max_j scale * q[h].k_j,  j < len;  an empty context gives 0.
//
// One pass over the cache with a running maximum and sum.  The floor is the
// cache's bytes, 2 * 1.0625 per key-value pair of elements, so everything is
// arranged around the copy stream; what comes next is the instruction issue
// (int8 to floating point), hence the layouts below.
//
// Work split.  A unit is (sequence, key-value head, chunk of the heads that
// share it); its context is cut into tiles of 64 tokens.  The tiles of all
// units, in order, are split evenly over a fixed grid of persistent CTAs, so
// one long sequence and many ragged ones balance alike.  A unit that falls
// on several CTAs leaves (m, l, o) parts in the workspace; the CTA that
// arrives last at the unit's counter joins them in the order of the tiles
// (the result does not depend on timing) and sets the counter back to 0.
//
// Copies.  Four warps take 16 tokens of each tile, and each warp has a ring
// of its own in shared memory, which it fills by 16-byte cp.async and waits
// for by itself: no barrier inside a unit, any page size that is a multiple
// of 16 alike.  The chunks are swizzled so that both read patterns below are
// free of bank conflicts.  (One warp issuing TMA boxes for all four was the
// first form: with pages of 16 tokens, 16 small copies a tile, the copies alone
// took 66 us for 162 MB; with pages of 128, 127 us for 706 MB.
// Each warp issuing TMA boxes of its own: 174 us for the 706 MB, against 156
// with cp.async then.)
//
// Scores (m16n8k16, fp16 operands): A holds the queries, B the codes of 8
// tokens, which are exact in fp16.  (As code + 128, without the subtraction
// that takes the 128 off again, the partial sums were as large as 128 sum |q|
// whatever the codes: with one large key channel per block, at which the query
// is 0, fp32 results were off by up to 4 times their bound.)  Each query row
// is scaled by a power of two to just below 2^14 before it is rounded, so
// 16-bit queries are exact and fp32 ones become a pair hi + lo of at least 22
// bits, in rows g and g + 8 of the same fragment (both down to 2^-39 of the
// row's largest element).  Two MMAs cover one block of 32 values; its scale is
// then applied in fp32.
//
// Values (m16n8k8, tf32 operands), transposed, o^T = V^T p^T: A holds 16 dims of
// 8 tokens, exact, B = p_j * scale_j of 8 heads, in tf32 because the scales
// need fp32's range (fp32 rows: hi, then lo).  The accumulators of the
// scores are, in the same lanes, this B; and with 8 heads the sums take half
// the registers that heads as rows of 16 would.
//
// These are warp-level MMAs: there are at most 16 query rows per key-value
// head, an eighth of the smallest tcgen05 tile, and the operands change
// with every tile, so the tensor pipe is not what bounds this kernel.
//
// Measured, cold L2: 64 sequences of 2048..8192 tokens, 64 over 8 heads of 128,
// fp16, 158 us (4.5 TB/s); one of 131072, fp32, 85 us (3.4); 24 of 1..6000 with
// pages of 16, bf16, 53 us (3.0); 24 of 1..6000, 64 over 4 heads, fp16, 61 us
// (1.3).  Copies alone take 125 us of the 158; the issue slots are 61 % full.
#include <algorithm>

#include <cuda_fp16.h>

#include "kv_device.cuh"
#include "nvq_device.cuh"
#include "nvq_internal.h"
#include "tcgen05.cuh"

namespace nvq {
namespace {

constexpr int kTile = 64;            // tokens of a tile
constexpr int kWarps = 4;            // 16 tokens of a tile each
constexpr int kThreads = 32 * kWarps;
constexpr int kUnitCost = 3;         // a unit's start and end, in tiles
constexpr int kFlush = 4;            // tiles between additions of the accumulators, with fp32
constexpr float kLazy = 8.0f;        // the running maximum may lag by this power of two
// The running maximum before any finite score: a finite number, so that a
// score of -infinity (its value is below fp32's range) gets the weight 0
// where no finite one came before it, instead of exp2(-inf - -inf).
constexpr float kNone = -3.402823466e38f;

// How the 16 rows of an MMA are used: fp32 heads as hi (rows 0-7) and lo
// (rows 8-15); up to 8 heads of a 16-bit type; up to 16 of them.
enum Rows { kSplit = 0, kOne = 1, kTwo = 2 };

__device__ unsigned int g_attn_decode_error_flags = 0;   // bit 1: a bad index

struct DecodeArgs {
  const int8_t* kc;
  const int8_t* vc;
  const __half* ks;
  const __half* vs;
  const int32_t* lens;
  const int32_t* table;
  const void* q;
  void* out;
  int64_t q_stride, out_stride;
  int* counters;
  float* part;             // [2 * grid][rows][D + 4]: o, then m and l
  int B, max_pages, n_pages, page, kv_heads, group, chunks, rows, dtype;
  float scale_log2;
};

template <int D, Rows R>
struct Cfg {
  static constexpr int kHeads = R == kTwo ? 16 : 8;          // heads of a chunk
  static constexpr int kBlocks = D / 32;
  static constexpr int kStages = R == kSplit ? 6 : 4;
  static constexpr int kCodes = 16 * D;                      // bytes of 16 tokens' codes
  static constexpr int kScales = 16 * kBlocks * 2;
  static constexpr int kStage = 2 * kCodes + 2 * kScales;    // K, V, scales of K, of V
  static constexpr int kRing = kStages * kStage;             // of one warp
  static constexpr int kPart = D + 4;                        // floats of a part's row: o, m, l
  static constexpr int kOffMl = kWarps * kRing;
  static constexpr int kSmem = kOffMl + kWarps * kHeads * 8;
  static constexpr int kCtas = R == kOne ? 3 : 2;            // per SM
};

// The work in order: sequence by sequence, unit by unit, each as kUnitCost
// places for its start and end and then one for each tile, so that a CTA that
// gets many short units gets fewer tiles.
struct Walk {
  int b, unit, at, n;      // sequence, unit in it, place in the unit; n: the unit's tiles
  int left;                // places of this CTA from here on
  // tiles of the unit that are this CTA's: [first, last)
  __device__ int first() const { return max(0, at - kUnitCost); }
  __device__ int last() const { return max(0, min(n + kUnitCost, at + left) - kUnitCost); }
};

__device__ __forceinline__ int clamp_len(const DecodeArgs& a, int b) {
  return max(0, min(a.lens[b], a.max_pages * a.page));
}
__device__ __forceinline__ int tiles_of(const DecodeArgs& a, int b) {
  return static_cast<int>((clamp_len(a, b) + int64_t{kTile - 1}) / kTile);
}
__device__ __forceinline__ int places(int tiles) { return tiles > 0 ? tiles + kUnitCost : 0; }

// Split of W places over G CTAs: the first W % G have one more.
struct Split {
  unsigned base, rem;
  __device__ int start(int c) const { return c * base + min(static_cast<unsigned>(c), rem); }
  __device__ int owner(int at) const {
    const unsigned x = at, big = rem * (base + 1);
    return x < big ? x / (base + 1) : rem + (x - big) / base;
  }
};

__device__ __forceinline__ int warp_sum_int(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ int warp_scan_int(int v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// On to the next unit.
__device__ __forceinline__ void next_unit(const DecodeArgs& a, Walk& w, int U) {
  w.left -= w.n + kUnitCost - w.at;
  w.at = 0;
  if (w.left <= 0 || ++w.unit < U) return;
  w.unit = 0;
  do {
    if (++w.b >= a.B) {     // not met while places are left
      w.left = 0;
      return;
    }
    w.n = tiles_of(a, w.b);
  } while (w.n == 0);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                        float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// Four int8 codes as fp16 (u = code + 128 per byte): 0x64bb is 1024 + u, and
// 1152 off it is exact.
__device__ __forceinline__ void codes_to_h2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 off = dev::bits_h2(0x64806480u);
  lo = dev::h2_bits(__hsub2(dev::bits_h2(__byte_perm(u, 0x64646464u, 0x4140)), off));
  hi = dev::h2_bits(__hsub2(dev::bits_h2(__byte_perm(u, 0x64646464u, 0x4342)), off));
}
// The same as fp32: 0x4B0000bb is 2^23 + u.  The differences are exact.
__device__ __forceinline__ void codes_to_f32(uint32_t w, uint32_t (&f)[4]) {
  const uint32_t u = w ^ 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; i += 2)
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=r"(f[i]), "=r"(f[i + 1])
        : "r"(__byte_perm(u, 0x4B000000u, 0x7440 + i)), "r"(__byte_perm(u, 0x4B000000u, 0x7441 + i)),
          "r"(0xCB000080u));    // -(2^23 + 128)
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void store4(void* p, int64_t at, int dtype, float4 v) {
  if (dtype == NVQ_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = v;
  } else if (dtype == NVQ_F16) {
    *reinterpret_cast<uint2*>(static_cast<__half*>(p) + at) =
        make_uint2(dev::h2_bits(__floats2half2_rn(v.x, v.y)), dev::h2_bits(__floats2half2_rn(v.z, v.w)));
  } else {
    const __nv_bfloat162 u = __floats2bfloat162_rn(v.x, v.y), w = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&w));
  }
}

// The words of a query row that lane j holds: 8 elements of each block, at
// 32 * block + 8 * j; zeros for a row that is none.
template <int D, bool F32>
struct Raw {
  uint4 w[D / 32 * (F32 ? 2 : 1)];
  __device__ __forceinline__ void load(const void* q, int64_t at, bool on, int j) {
#pragma unroll
    for (int bl = 0; bl < D / 32; ++bl) {
      if (F32) {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(q) + at + 32 * bl + 8 * j);
        w[2 * bl] = on ? *s : make_uint4(0, 0, 0, 0);
        w[(2 * bl + 1) % (sizeof(w) / 16)] = on ? s[1] : make_uint4(0, 0, 0, 0);
      } else {
        w[bl] = on ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(q) + at + 32 * bl + 8 * j)
                   : make_uint4(0, 0, 0, 0);
      }
    }
  }
  __device__ __forceinline__ void values(int dtype, float (&x)[D / 4]) const {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(w) / 16); ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (F32) {
          x[(4 * i + k) % (D / 4)] = __uint_as_float(u[k]);
        } else {
          const float2 f = dtype == NVQ_F16 ? __half22float2(dev::bits_h2(u[k]))
                                            : make_float2(__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xFFFF0000u));
          x[(8 * i + 2 * k) % (D / 4)] = f.x, x[(8 * i + 2 * k + 1) % (D / 4)] = f.y;
        }
      }
    }
  }
};

// The row as operands: scaled by a power of two so that its largest lies in
// [2^13, 2^14), then rounded to fp16, and the remainder for `lo`.  Returns
// the two factors that turn the MMA's sums into powers of two.
template <int D, bool F32, bool LO>
__device__ __forceinline__ float2 query_row(const Raw<D, F32>& raw, int dtype, float scale_log2,
                                           uint32_t (&hi)[D / 8], uint32_t (&lo)[D / 8]) {
  float x[D / 4], top = 0.0f;
  raw.values(dtype, x);
#pragma unroll
  for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(x[i]));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // 2^(13 - exponent), kept within fp32's normal range (zeros and subnormals)
  const int k = min(126, 140 - static_cast<int>(__float_as_uint(top) >> 23));
  const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const float u = x[2 * i] * up, v = x[2 * i + 1] * up;
    const __half2 h = __floats2half2_rn(u, v);
    hi[i] = dev::h2_bits(h);
    if (LO) {
      const float2 f = __half22float2(h);
      lo[i] = dev::h2_bits(__floats2half2_rn(u - f.x, v - f.y));
    }
  }
  // 2^-k is up to 2^115, even for infinities: in one factor with the scale only
  // up to 2^16, so that neither factor overflows for a scale of up to 2^64, nor
  // the product of a sum (below 2^44) and the first one.  A sum of 0 stays 0,
  // and a score is finite where its value is.
  const int e1 = min(-k, 16);
  return make_float2(scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e1) << 23),
                     __uint_as_float(static_cast<uint32_t>(127 - k - e1) << 23));
}

template <int D, Rows R>
__global__ void __launch_bounds__(kThreads, (Cfg<D, R>::kCtas))
attn_decode_kernel(const DecodeArgs a) {
  using C = Cfg<D, R>;
  extern __shared__ __align__(128) unsigned char smem[];
  float* ml = reinterpret_cast<float*>(smem + C::kOffMl);            // [warp][head][m, l]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // what only the walk and the ends of units need stays out of the registers
  // of the main loop
  struct Seg {
    int b, unit, n, start;      // a unit that other CTAs have parts of; start: its first place
  };
  __shared__ Split split_s;
  __shared__ Walk pw_s[kWarps];  // each warp's copies' position
  __shared__ Seg seg_s[2];
  __shared__ int last_s[2];
  const int U = a.kv_heads * a.chunks;
  const int G = gridDim.x, cta = blockIdx.x;
  // every warp finds the CTA's first place for itself (no hand-over): the sum
  // of all places, then the sequence that holds the first one
  int total = 0, mine = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    mine = b0 + lane < a.B ? tiles_of(a, b0 + lane) : 0;
    total += places(mine);
  }
  total = warp_sum_int(total) * U;
  const Split split = {static_cast<unsigned>(total) / G, static_cast<unsigned>(total) % G};
  Walk w = {0, 0, 0, 0, split.start(cta + 1) - split.start(cta)};
  int unit_start = 0;           // the first place of the unit of `w`
  if (w.left > 0) {
    const int first = split.start(cta);
    int before = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      if (a.B > 32) mine = b0 + lane < a.B ? tiles_of(a, b0 + lane) : 0;
      const int incl = warp_scan_int(places(mine), lane);
      const unsigned hit = __ballot_sync(0xffffffffu, (before + incl) * U > first);
      if (hit != 0) {
        const int at = __ffs(hit) - 1;
        w.b = b0 + at;
        w.n = __shfl_sync(0xffffffffu, mine, at);
        before += __shfl_sync(0xffffffffu, incl - places(mine), at);
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    const int r = first - before * U;
    w.unit = static_cast<unsigned>(r) / static_cast<unsigned>(w.n + kUnitCost);
    w.at = r - w.unit * (w.n + kUnitCost);
    unit_start = first - w.at;
  }
  if (threadIdx.x == 0) split_s = split;
  if (lane == 0) pw_s[warp] = w;
  __syncwarp();

  // ------------------------------- the copies -------------------------------
  // This warp's 16 tokens of the tiles ahead.  Their place in the table moves
  // on by a tile at a time; the page is read one tile ahead of its copies.
  const int step_page = kTile / a.page, step_off = kTile % a.page;
  const uint32_t ring = ptx::smem_addr(smem) + warp * C::kRing;
  // chunk (of 16 bytes) lane + 32 i of the codes: row (lane + 32 i) / (D / 16),
  // exchanged within the row's 128 (or 64) bytes
  constexpr int kRowChunks = D / 16;
  auto swz = [](int r) { return D == 128 ? r & 7 : (r >> 1) & 3; };
  const int r0 = lane / kRowChunks;
  const uint32_t to0 = r0 * D + (((lane % kRowChunks) ^ swz(r0)) << 4);
  int p_s = 0;                  // ring slot of the next tile
  int p_left = 0;               // tiles of the unit not issued yet (0: none is left at all)
  int p_rem = 0;                // this warp's tokens from the next tile on, the other warps' included
  int p_idx = 0, p_off = 0;     // column of the table, token in the page
  int p_page = 0;
  int p_head = 0;
  const int32_t* p_table = nullptr;
  auto begin_unit = [&]() {     // from pw_s, at some tile of a unit
    const Walk pw = pw_s[warp];
    p_left = pw.left > 0 ? pw.last() - pw.first() : 0;
    if (p_left <= 0) {
      p_left = 0;
      return;
    }
    const int pos0 = pw.first() * kTile + 16 * warp;
    p_rem = clamp_len(a, pw.b) - pos0;
    p_idx = pos0 / a.page;
    p_off = pos0 % a.page;
    p_head = pw.unit / a.chunks;
    p_table = a.table + static_cast<int64_t>(pw.b) * a.max_pages;
    if (p_rem > 0) p_page = p_table[p_idx];
  };
  auto issue = [&]() {
    if (p_left > 0) {
      if (p_rem > 0) {
        if (p_page < 0 || p_page >= a.n_pages) {
          if (lane == 0) atomicOr(&g_attn_decode_error_flags, 2u);
          p_page = 0;
        }
        const int64_t row = (p_page * a.kv_heads + p_head) * a.page + p_off;     // below 2^31
        const int8_t* k = a.kc + row * D + 16 * lane;
        const int8_t* v = a.vc + row * D + 16 * lane;
        const uint32_t to = ring + p_s * C::kStage;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          // 4 rows of 128 bytes, or 8 of 64, further on: the exchange differs
          // by a constant
          const uint32_t t = to + (to0 ^ (D == 128 ? (i & 1) << 6 : 0)) + 512 * i;
          ptx::cp_async_16(t, k + 512 * i, 16);
          ptx::cp_async_16(t + C::kCodes, v + 512 * i, 16);
        }
        constexpr int kN = C::kScales / 16;
        if (lane < 2 * kN)
          ptx::cp_async_16(to + 2 * C::kCodes + 16 * lane,
                           reinterpret_cast<const uint8_t*>((lane < kN ? a.ks : a.vs) + row * C::kBlocks) + 16 * (lane % kN), 16);
      }
      p_s = p_s + 1 == C::kStages ? 0 : p_s + 1;
      if (--p_left > 0) {
        p_rem -= kTile;
        p_idx += step_page;
        p_off += step_off;
        if (p_off >= a.page) {
          p_off -= a.page;
          ++p_idx;
        }
        if (p_rem > 0) p_page = p_table[p_idx];
      } else {
        Walk pw = pw_s[warp];
        next_unit(a, pw, U);
        __syncwarp();
        if (lane == 0) pw_s[warp] = pw;
        __syncwarp();
        begin_unit();
      }
    }
    ptx::cp_async_commit();      // one group a tile, empty ones included
  };
  begin_unit();
  for (int i = 0; i < C::kStages - 1; ++i) issue();

  // -------------------------------- the tokens -------------------------------
  const int gq = lane >> 2, j = lane & 3;
  // Token order inside a tile of 8: column n of the score MMA is token
  // perm(n).  It makes the four rows that a half-warp reads (K), and the
  // four that the lanes j read (V), fall on different banks.
  constexpr uint32_t kPerm = D == 128 ? 0x57136420u : 0x67235410u;
  auto perm = [](int n) { return static_cast<int>((kPerm >> (4 * n)) & 7u); };
  const int tk = perm(gq), ta = perm(2 * j), tb = perm(2 * j + 1);
  const uint32_t off_k = tk * D + (((j >> 1) ^ swz(tk)) << 4) + (j & 1) * 8;
  const uint32_t off_va = ta * D + (((gq >> 2) ^ swz(ta)) << 4) + (gq & 3) * 4;
  const uint32_t off_vb = tb * D + (((gq >> 2) ^ swz(tb)) << 4) + (gq & 3) * 4;
  constexpr int kH = R == kTwo ? 2 : 1;      // heads of this lane: gq, and gq + 8

  // sequences without tokens: zeros
  for (int b = cta; b < a.B; b += G) {
    const int64_t len = a.lens[b];
    if (threadIdx.x == 0 && (len < 0 || len > static_cast<int64_t>(a.max_pages) * a.page))
      atomicOr(&g_attn_decode_error_flags, 2u);
    if (clamp_len(a, b) == 0) {
      const int n = a.kv_heads * a.group * D;
      for (int i = 4 * threadIdx.x; i < n; i += 4 * kThreads)
        store4(a.out, b * a.out_stride + i, a.dtype, make_float4(0.f, 0.f, 0.f, 0.f));
    }
  }

  Raw<D, R == kSplit> raw[kH];
  auto load_queries = [&]() {
    const int hk = w.unit / a.chunks, chunk = w.unit - hk * a.chunks;
    const int hc = min(C::kHeads, a.group - chunk * C::kHeads);
    const int64_t at = w.b * a.q_stride + static_cast<int64_t>(hk * a.group + chunk * C::kHeads) * D;
#pragma unroll
    for (int h = 0; h < kH; ++h) raw[h].load(a.q, at + (gq + 8 * h) * D, gq + 8 * h < hc, j);
  };
  constexpr int kVecs = D / 4;
  int s_last = 0;               // ring slot used last
  // Row (warp x, head h) of eight heads' sums, in the codes of the ring slot
  // that was used last (it is filled again only by the next tile's issue):
  // D floats, its float4s exchanged by the head so that the four heads that
  // lanes j write fall on different banks.
  auto red = [&](int x, int h, int d4) -> float4* {
    unsigned char* at = smem + x * C::kRing + s_last * C::kStage;
    return reinterpret_cast<float4*>(at) + (h * (D / 4) + (d4 ^ (((h >> 1) & 3) << 1)));
  };
  // Sum of the four warps' rows of the chunk's heads 8 n + h; the result, or a part.
  auto join4 = [&](int b, int unit, int n, float* part) {
    const int hk = unit / a.chunks, chunk = unit - hk * a.chunks;
    const int hc = min(C::kHeads, a.group - chunk * C::kHeads);
    const int64_t to_out = b * a.out_stride + static_cast<int64_t>(hk * a.group + chunk * C::kHeads) * D;
    for (int i = threadIdx.x; i < min(8, hc - 8 * n) * kVecs; i += kThreads) {
      const int h = i / kVecs, d4 = i - h * kVecs, hn = 8 * n + h;
      float top = -INFINITY, L = 0.0f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) top = fmaxf(top, ml[2 * (x * C::kHeads + hn)]);
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float c = exp2_approx(ml[2 * (x * C::kHeads + hn)] - top);
        L = fmaf(c, ml[2 * (x * C::kHeads + hn) + 1], L);
        const float4 v = *red(x, h, d4);
        O.x = fmaf(c, v.x, O.x), O.y = fmaf(c, v.y, O.y), O.z = fmaf(c, v.z, O.z), O.w = fmaf(c, v.w, O.w);
      }
      if (part == nullptr) {
        const float inv = __fdividef(1.0f, L);
        store4(a.out, to_out + hn * D + 4 * d4, a.dtype, make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv));
      } else {
        float* to = part + hn * C::kPart;
        __stcg(reinterpret_cast<float4*>(to + 4 * d4), O);
        if (d4 == 0) __stcg(reinterpret_cast<float2*>(to + D), make_float2(top, L));
      }
    }
  };
  const int64_t part_floats = static_cast<int64_t>(a.rows) * C::kPart;

  int g_s = 0;                  // ring slot of the next tile to be used
  int segs = 0;                 // units here that other CTAs have parts of
  if (w.left > 0 && w.last() <= w.first()) w.left = 0;      // places of a unit's cost alone
  while (w.left > 0) {
    // ------------------------- one unit (or a part of it) -------------------------
    const int b = w.b, unit = w.unit, tile0 = w.first(), n_here = w.last() - tile0;
    const bool whole = n_here == w.n;
    // tokens from the first tile of this part on; only the last tile's matter
    int rem = clamp_len(a, b) - tile0 * kTile;
    load_queries();
    uint32_t qh[D / 8], ql[D / 8];
    float2 factor[kH];
    factor[0] = query_row<D, R == kSplit, R == kSplit>(raw[0], a.dtype, a.scale_log2, qh, ql);
    if constexpr (R == kTwo) {
      uint32_t none[D / 8];
      factor[kH - 1] = query_row<D, false, false>(raw[kH - 1], a.dtype, a.scale_log2, ql, none);
    }

    // o[n][2 * bl + x]: heads 8 n + 2 j (elements 0, 2) and 8 n + 2 j + 1 (1, 3),
    // dims 32 bl + 4 gq + 2 x (0, 1) and the next one (2, 3)
    float o[kH][D / 16][4], m[kH], l[kH];
#pragma unroll
    for (int n = 0; n < kH; ++n)
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
#pragma unroll
    for (int h = 0; h < kH; ++h) m[h] = kNone, l[h] = 0.0f;

    // The tensor core adds to its accumulators by truncation, so with fp32 they
    // hold kFlush tiles at a time and are added up here (131072 tokens: 2.6e-6
    // of error without it).
    float sum[R == kSplit ? D / 16 : 1][4] = {};
    uint32_t odd = 0;             // fp16 pair: the largest |value scale| seen by this lane
    for (int t = n_here; t > 0; --t, rem -= kTile) {
      if (R == kSplit && (n_here - t) % kFlush == kFlush - 1) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            sum[i % (R == kSplit ? D / 16 : 1)][u] += o[0][i][u];
            o[0][i][u] = 0.0f;
          }
      }
      issue();                                  // into the slot of the tile before
      ptx::cp_async_wait<C::kStages - 1>();
      __syncwarp();
      const int valid = rem - 16 * warp;        // this warp's tokens (16 or more: all)
      if (valid > 0) {
        const uint32_t kb = ring + g_s * C::kStage, vb = kb + C::kCodes;
        const uint32_t ksb = kb + 2 * C::kCodes, vsb = ksb + C::kScales;
        // ---- scores of the lane's tokens ta, tb, 8 + ta, 8 + tb
        float p[kH][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float da[C::kBlocks], db[C::kBlocks];
          if constexpr (D == 128) {
            const uint2 u = lds64(ksb + (8 * x + ta) * 8), v = lds64(ksb + (8 * x + tb) * 8);
            const float2 u0 = __half22float2(dev::bits_h2(u.x)), u1 = __half22float2(dev::bits_h2(u.y));
            const float2 v0 = __half22float2(dev::bits_h2(v.x)), v1 = __half22float2(dev::bits_h2(v.y));
            da[0] = u0.x, da[1] = u0.y, da[2] = u1.x, da[3] = u1.y;
            db[0] = v0.x, db[1] = v0.y, db[2] = v1.x, db[3] = v1.y;
          } else {
            const float2 u = __half22float2(dev::bits_h2(lds32(ksb + (8 * x + ta) * 4)));
            const float2 v = __half22float2(dev::bits_h2(lds32(ksb + (8 * x + tb) * 4)));
            da[0] = u.x, da[1] = u.y, db[0] = v.x, db[1] = v.y;
          }
          float sa[kH] = {}, sb[kH] = {};
#pragma unroll
          for (int bl = 0; bl < C::kBlocks; ++bl) {
            const uint2 c8 = lds64(kb + 8 * x * D + (off_k ^ (32u * bl)));
            uint32_t b0, b1, b2, b3;
            codes_to_h2(c8.x, b0, b1);
            codes_to_h2(c8.y, b2, b3);
            float acc[4];
            const uint32_t z = 0;
            mma_f16(acc, qh[4 * bl], R == kOne ? z : ql[4 * bl], qh[4 * bl + 1], R == kOne ? z : ql[4 * bl + 1], b0, b1, 0.0f, 0.0f, 0.0f, 0.0f);
            mma_f16(acc, qh[4 * bl + 2], R == kOne ? z : ql[4 * bl + 2], qh[4 * bl + 3], R == kOne ? z : ql[4 * bl + 3], b2, b3,
                    acc[0], acc[1], acc[2], acc[3]);
            if (R == kSplit) acc[0] += acc[2], acc[1] += acc[3];
            sa[0] = fmaf(da[bl], acc[0], sa[0]);
            sb[0] = fmaf(db[bl], acc[1], sb[0]);
            if (R == kTwo) {
              sa[kH - 1] = fmaf(da[bl], acc[2], sa[kH - 1]);
              sb[kH - 1] = fmaf(db[bl], acc[3], sb[kH - 1]);
            }
          }
#pragma unroll
          for (int h = 0; h < kH; ++h) {
            p[h][2 * x] = sa[h] * factor[h].x * factor[h].y;
            p[h][2 * x + 1] = sb[h] * factor[h].x * factor[h].y;
          }
        }
        if (valid < 16) {        // the last tile
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((i >> 1) * 8 + (i & 1 ? tb : ta) >= valid)
#pragma unroll
              for (int h = 0; h < kH; ++h) p[h][i] = -INFINITY;
        }
        // ---- running maximum (the same in the four lanes of a head) and sum.
        // The maximum is only a reference point: it may lag while no exponent
        // passes 2^8, so most tiles need no more than this vote.
        float top[kH];
        bool grow = false;
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          top[h] = fmaxf(fmaxf(p[h][0], p[h][1]), fmaxf(p[h][2], p[h][3]));
          grow |= top[h] > m[h] + kLazy;
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int h = 0; h < kH; ++h) {
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
            const float mn = fmaxf(m[h], top[h]);
            const float c = m[h] == mn ? 1.0f : exp2_approx(m[h] - mn);
            m[h] = mn;
            l[h] *= c;
            // the factors of the heads whose sums this lane holds
            const float c0 = __shfl_sync(0xffffffffu, c, 8 * j), c1 = __shfl_sync(0xffffffffu, c, 8 * j + 4);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[h][i][0] *= c0, o[h][i][1] *= c1, o[h][i][2] *= c0, o[h][i][3] *= c1;
              if constexpr (R == kSplit) sum[i][0] *= c0, sum[i][1] *= c1, sum[i][2] *= c0, sum[i][3] *= c1;
            }
          }
        }
#pragma unroll
        for (int h = 0; h < kH; ++h) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[h][i] = exp2_approx(p[h][i] - m[h]);
            l[h] += p[h][i];
          }
        }
        // ---- values: one block of 32 at a time
        if constexpr (R != kSplit) {
          // one word of them a lane: the largest |scale| of its two blocks
          uint32_t w = 4 * lane < C::kScales && 2 * lane / C::kBlocks < valid ? lds32(vsb + 4 * lane) : 0u;
          odd = __vmaxu2(odd, w & 0x7FFF7FFFu);
        }
        uint2 sc[4];     // the tokens' value scales
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = (i >> 1) * 8 + (i & 1 ? tb : ta);
          sc[i] = D == 128 ? lds64(vsb + tok * 8) : make_uint2(lds32(vsb + tok * 4), 0u);
        }
        if (valid < 16) {        // whatever lies behind the last token
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((i >> 1) * 8 + (i & 1 ? tb : ta) >= valid) sc[i] = make_uint2(0u, 0u);
        }
#pragma unroll
        for (int bl = 0; bl < C::kBlocks; ++bl) {
          uint32_t hi[kH][4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 d2 = __half22float2(dev::bits_h2(bl < 2 ? sc[i].x : sc[i].y));
            const float d = (bl & 1) ? d2.y : d2.x;
#pragma unroll
            for (int h = 0; h < kH; ++h) {
              const float x = p[h][i] * d;
              if (R == kSplit) {
                hi[h][i] = __float_as_uint(x) & 0xFFFFE000u;              // tf32, exactly
                lo[i] = __float_as_uint(x - __uint_as_float(hi[h][i]));
              } else {
                // to nearest: the MMA drops 13 bits.  A NaN's carry goes into
                // its sign; `odd` brings it back at the unit's end (64
                // sequences of 2048..8192: 156 us without it, 158 with it, 162
                // with cvt.rna here)
                hi[h][i] = __float_as_uint(x) + 0x1000u;
              }
            }
          }
          const uint32_t x32 = 32u * bl;
#pragma unroll
          for (int x = 0; x < 2; ++x) {      // tokens 0-7, tokens 8-15
            uint32_t va[4], vc[4];
            codes_to_f32(lds32(vb + 8 * x * D + (off_va ^ x32)), va);
            codes_to_f32(lds32(vb + 8 * x * D + (off_vb ^ x32)), vc);
#pragma unroll
            for (int n = 0; n < kH; ++n) {
              mma_tf32(o[n][2 * bl], va[0], va[1], vc[0], vc[1], hi[n][2 * x], hi[n][2 * x + 1]);
              mma_tf32(o[n][2 * bl + 1], va[2], va[3], vc[2], vc[3], hi[n][2 * x], hi[n][2 * x + 1]);
            }
            if (R == kSplit) {
              mma_tf32(o[0][2 * bl], va[0], va[1], vc[0], vc[1], lo[2 * x], lo[2 * x + 1]);
              mma_tf32(o[0][2 * bl + 1], va[2], va[3], vc[2], vc[3], lo[2 * x], lo[2 * x + 1]);
            }
          }
        }
      }
      __syncwarp();                             // all lanes have left the slot
      g_s = g_s + 1 == C::kStages ? 0 : g_s + 1;
    }

    if constexpr (R == kSplit) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) o[0][i][u] += sum[i][u];
    }
    if constexpr (R != kSplit) {
      // A value block with a NaN scale gives NaN; with an infinite one what it
      // is, but NaN where its weight underflowed
      if (__any_sync(0xffffffffu, __vcmpgeu2(odd, 0x7C007C00u) != 0)) {
#pragma unroll
        for (int i = C::kBlocks / 2; i < 32; i <<= 1) odd = __vmaxu2(odd, __shfl_xor_sync(0xffffffffu, odd, i));
#pragma unroll
        for (int bl = 0; bl < C::kBlocks; ++bl) {
          const uint32_t top = (__shfl_sync(0xffffffffu, odd, bl / 2) >> (16 * (bl & 1))) & 0xFFFFu;
#pragma unroll
          for (int n = 0; n < kH; ++n)
#pragma unroll
            for (int i = 2 * bl; i < 2 * bl + 2; ++i)
#pragma unroll
              for (int u = 0; u < 4; ++u)
                if (top > 0x7C00u || (top == 0x7C00u && fabsf(o[n][i][u]) < INFINITY)) o[n][i][u] = __uint_as_float(0x7FFFFFFFu);
        }
      }
    }
    // ------------------ the four warps' parts of the unit, joined ------------------
    // Eight heads at a time.  A part goes to this CTA's slot of the workspace:
    // the second one if it starts the unit (then it is the CTA's last), else
    // the first.
    s_last = g_s == 0 ? C::kStages - 1 : g_s - 1;
    float* part = whole ? nullptr : a.part + (2 * static_cast<int64_t>(cta) + (tile0 == 0 ? 1 : 0)) * part_floats;
    if (!whole) {
      if (threadIdx.x == 0) seg_s[segs] = {b, unit, w.n, unit_start};
      ++segs;
    }
    unit_start += w.n + kUnitCost;
    next_unit(a, w, U);
    if (w.left > 0 && w.last() <= w.first()) w.left = 0;
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (j == 0) {
        ml[2 * (warp * C::kHeads + gq + 8 * h)] = m[h];
        ml[2 * (warp * C::kHeads + gq + 8 * h) + 1] = l[h];
      }
      __syncthreads();      // every warp has left the tile's codes, or the heads before
#pragma unroll
      for (int bl = 0; bl < C::kBlocks; ++bl) {
        const float(&u)[4] = o[h][2 * bl];
        const float(&v)[4] = o[h][2 * bl + 1];
        *red(warp, 2 * j, 8 * bl + gq) = make_float4(u[0], u[2], v[0], v[2]);
        *red(warp, 2 * j + 1, 8 * bl + gq) = make_float4(u[1], u[3], v[1], v[3]);
      }
      __syncthreads();
      join4(b, unit, h, part);
    }
    __syncthreads();      // the slot goes back to the copies, ml to the next unit
  }

  // ----------------------- units that several CTAs have parts of -----------------------
  // All arrivals are made here, so that no stream of copies waits for one; the
  // CTA that arrives last adds up the unit's parts, in tile order.
  if (segs == 0) return;
  const Split sp = split_s;
  auto owners = [&](const Seg& x, int& c0, int& c1) {
    c0 = sp.owner(x.start + kUnitCost);
    c1 = sp.owner(x.start + kUnitCost + x.n - 1);
  };
  if (threadIdx.x < segs) {
    const Seg x = seg_s[threadIdx.x];
    int c0, c1;
    owners(x, c0, c1);
    int* counter = a.counters + static_cast<int64_t>(x.b) * U + x.unit;
    __threadfence();      // the parts of this CTA, seen through the barrier, come first
    const int old = atomicAdd(counter, 1);
    __threadfence();
    last_s[threadIdx.x] = old == c1 - c0;
    if (old == c1 - c0) *counter = 0;
  }
  __syncthreads();
  for (int i = 0; i < segs; ++i) {
    if (!last_s[i]) continue;
    const Seg x = seg_s[i];
    int c0, c1;
    owners(x, c0, c1);
    const int parts = c1 - c0 + 1, chunk = x.unit % a.chunks;
    const int hc = min(C::kHeads, a.group - chunk * C::kHeads);
    const float* from = a.part + (2 * static_cast<int64_t>(c0) + 1) * part_floats;      // part 0, then every second slot from c0 + 1 on
    for (int n = 0; n < kH; ++n) {
      // each warp adds a quarter of the parts, every load of eight of them at once
      for (int e = lane; e < min(8, hc - 8 * n) * kVecs; e += 32) {
        const int h = e / kVecs, d4 = e - h * kVecs, hn = 8 * n + h;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
        float top = -INFINITY, L = 0.0f;
        for (int k0 = warp; k0 < parts; k0 += 8 * kWarps) {
          float2 y[8];
          float4 v[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int k = k0 + u * kWarps;
            const float* at = from + (k == 0 ? 0 : 2 * k - 1) * part_floats + hn * C::kPart;
            y[u] = k < parts ? __ldcg(reinterpret_cast<const float2*>(at + D)) : make_float2(-INFINITY, 0.0f);
            v[u] = k < parts ? __ldcg(reinterpret_cast<const float4*>(at + 4 * d4)) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
          float mn = top;
#pragma unroll
          for (int u = 0; u < 8; ++u) mn = fmaxf(mn, y[u].x);
          const float c = exp2_approx(top - mn);      // mn is at least kNone: k0 is a part
          top = mn;
          L *= c, O.x *= c, O.y *= c, O.z *= c, O.w *= c;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const float f = exp2_approx(y[u].x - mn);
            L = fmaf(f, y[u].y, L);
            O.x = fmaf(f, v[u].x, O.x), O.y = fmaf(f, v[u].y, O.y), O.z = fmaf(f, v[u].z, O.z), O.w = fmaf(f, v[u].w, O.w);
          }
        }
        *red(warp, h, d4) = O;
        if (d4 == 0) {
          ml[2 * (warp * C::kHeads + hn)] = top;
          ml[2 * (warp * C::kHeads + hn) + 1] = L;
        }
      }
      __syncthreads();
      join4(x.b, x.unit, n, nullptr);
      __syncthreads();
    }
  }
}

template <int D, Rows R>
cudaError_t decode_launch(const nvq_kv_cache& c, DecodeArgs a, cudaStream_t stream) {
  using C = Cfg<D, R>;
  static SmemAttrOnce attr;
  cudaError_t e = attr.ensure(attn_decode_kernel<D, R>, C::kSmem);
  if (e != cudaSuccess) return e;
  a.chunks = (a.group + C::kHeads - 1) / C::kHeads;
  a.rows = std::min(a.group, C::kHeads);
  // no more CTAs than the tables can hold tiles
  const int64_t cap = (static_cast<int64_t>(a.max_pages) * a.page + kTile - 1) / kTile;
  const int64_t tiles = std::max<int64_t>(1, a.B * cap) * a.kv_heads * a.chunks;
  const int64_t grid = std::min<int64_t>(static_cast<int64_t>(device_sm_count()) * C::kCtas, tiles);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_decode_kernel<D, R>, a);
}

}  // namespace

// Two parts per CTA, up to 16 rows of head_dim + 4 floats.
size_t attn_decode_workspace_size(int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim) {
  const int64_t rows = std::min<int64_t>(16, heads / kv_heads);
  return static_cast<size_t>(device_sm_count()) * 3 * 2 * rows * (head_dim + 4) * sizeof(float);
}

cudaError_t launch_attn_decode(const nvq_kv_cache& c, const int32_t* seq_lens,
                               const int32_t* block_table, int64_t B, int64_t max_pages,
                               const void* q, int64_t q_stride, int64_t heads, float scale,
                               int dtype, void* out, int64_t out_stride, int32_t* counters,
                               void* workspace, cudaStream_t stream) {
  DecodeArgs a = {};
  a.kc = c.k_codes;
  a.vc = c.v_codes;
  a.ks = reinterpret_cast<const __half*>(c.k_scales);
  a.vs = reinterpret_cast<const __half*>(c.v_scales);
  a.lens = seq_lens;
  a.table = block_table;
  a.q = q;
  a.out = out;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.counters = counters;
  a.part = static_cast<float*>(workspace);
  a.B = static_cast<int>(B);
  a.max_pages = static_cast<int>(max_pages);
  a.n_pages = static_cast<int>(c.n_pages);
  a.page = static_cast<int>(c.page_size);
  a.kv_heads = static_cast<int>(c.n_kv_heads);
  a.group = static_cast<int>(heads / c.n_kv_heads);
  a.dtype = dtype;
  a.scale_log2 = scale * 1.4426950408889634f;
  const Rows r = dtype == NVQ_F32 ? kSplit : a.group <= 8 ? kOne : kTwo;
  if (c.head_dim == 64)
    return r == kSplit ? decode_launch<64, kSplit>(c, a, stream)
           : r == kOne ? decode_launch<64, kOne>(c, a, stream)
                       : decode_launch<64, kTwo>(c, a, stream);
  return r == kSplit ? decode_launch<128, kSplit>(c, a, stream)
         : r == kOne ? decode_launch<128, kOne>(c, a, stream)
                     : decode_launch<128, kTwo>(c, a, stream);
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
