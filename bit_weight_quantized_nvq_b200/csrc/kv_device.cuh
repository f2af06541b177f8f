// Device helpers shared by the paged-cache and attention kernels (sm_100a):
// 16- and 32-bit element types, sequence lookup in a packed batch, and page
// addresses.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "nvq_internal.h"

namespace nvq {
namespace dev {

// Element types of the packed rows: conversion to and from fp32 (one
// rounding, to nearest even).
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// N consecutive elements as one or more 16-byte accesses.
template <typename T, int N>
struct alignas(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Vec {
  T v[N];
};

// The kernels of the cache and the decode attention are launched while the
// kernel before them on the stream may still run and write what they read
// (programmatic launch; they wait before their first load).  So their loads are
// ordinary ones: the non-coherent path is for data that nothing writes from a
// kernel's launch on, and may hold what another kernel read there before.

// The number of entries of the non-decreasing cu[1..B] that are <= row, i.e.
// the sequence that holds packed row `row` (B: behind the last sequence).
// The whole warp searches: each round probes 32 evenly spaced entries, so a
// batch of up to 32 takes one dependent load and one of up to 1024 two.  A
// table that is not sorted gives some value in 0..B.
__device__ __forceinline__ int warp_find_seq(const int32_t* cu, int B, int row,
                                             int lane) {
  int lo = 0, n = B;
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = (lane + 1) * step - 1;
    const bool le = i < n && cu[1 + lo + i] <= row;
    const int cnt = __popc(__ballot_sync(0xffffffffu, le));
    lo += cnt * step;
    n = min(step - 1, max(0, n - cnt * step));
  }
  return min(lo, B);
}

}  // namespace dev
}  // namespace nvq
