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

}  // namespace gmm
