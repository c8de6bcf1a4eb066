// Constants and conversions that the kernels around the grouped products share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "gmm_kernel.cuh"

namespace gmm {

constexpr uint32_t kStatusBadSlot = 16u;   // a slot_rows / row_slots value outside its range
constexpr uint32_t kStatusBadLogit = 32u;  // a router's logit that is NaN (or, under a softmax, +infinity)

constexpr int kRouteMaxTopK = 32;          // a token's slots are held one per lane
constexpr int kRouteMaxExperts = 4096;     // one group per expert: the grouped kernels' limit

template <class T>
__device__ __forceinline__ T route_from_float(float x);
template <>
__device__ __forceinline__ float route_from_float(float x) { return x; }
template <>
__device__ __forceinline__ __half route_from_float(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 route_from_float(float x) { return __float2bfloat16_rn(x); }

// Division by a number that the host knows: for n < 2^31 and m = floor(2^(31 + l) / d) + 1 with 2^l >= d,
// n / d = n * m >> (31 + l).  d = 1 has mul = 0.
struct Divisor {
  uint32_t d, mul, shift;
  __host__ static Divisor of(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    return d == 1 ? Divisor{1, 0, 0} : Divisor{d, static_cast<uint32_t>((1ull << (31 + l)) / d + 1), l - 1};
  }
  __device__ __forceinline__ uint32_t quotient(uint32_t n) const { return mul == 0u ? n : __umulhi(n, mul) >> shift; }
};

}  // namespace gmm
