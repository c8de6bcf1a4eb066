// Sixteen consecutive elements of bf16, fp16 or fp32 as the quantisers load and look at them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

#include "sm103_ptx.cuh"

namespace gmm {

// 16 consecutive elements as fp32 bit patterns' source: raw loads, then values.
template <class T>
struct QuantRaw;
template <>
struct QuantRaw<float> { uint32_t w[16]; };
template <>
struct QuantRaw<__half> { uint32_t w[8]; };
template <>
struct QuantRaw<__nv_bfloat16> { uint32_t w[8]; };

// kAlign: what the address is a multiple of, 32 (whole sectors by one load), 16, or the
// element's size.
template <class T, int kAlign>
__device__ __forceinline__ QuantRaw<T> quant_load(const uint8_t *p) {
  QuantRaw<T> r;
  constexpr int kWords = sizeof(r.w) / 4;
  if constexpr (kAlign == 32) {
#pragma unroll
    for (int i = 0; i < kWords / 8; ++i) ld_global_nc_v8(p + 32 * i, *reinterpret_cast<uint32_t(*)[8]>(&r.w[8 * i]));
  } else if constexpr (kAlign == 16) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
      r.w[4 * i] = v.x;
      r.w[4 * i + 1] = v.y;
      r.w[4 * i + 2] = v.z;
      r.w[4 * i + 3] = v.w;
    }
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) r.w[i] = __ldg(reinterpret_cast<const uint32_t *>(p) + i);
  } else {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const unsigned short *h = reinterpret_cast<const unsigned short *>(p) + 2 * i;
      r.w[i] = static_cast<uint32_t>(__ldg(h)) | (static_cast<uint32_t>(__ldg(h + 1)) << 16);
    }
  }
  return r;
}

// The largest magnitude of 16 elements as an fp32 bit pattern.  Magnitudes are compared as
// integers (the order of the bit patterns without the sign), so a NaN ends up largest.
template <class T>
__device__ __forceinline__ uint32_t quant_amax(const QuantRaw<T> &r) {
  if constexpr (sizeof(T) == 4) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, r.w[i] & 0x7fffffffu);
    return m;
  } else {
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m2 = __vmaxu2(m2, r.w[i] & 0x7fff7fffu);
    const unsigned short m = static_cast<unsigned short>(max(m2 & 0xffffu, m2 >> 16));
    if constexpr (std::is_same_v<T, __half>) return __float_as_uint(__half2float(__ushort_as_half(m)));
    else return static_cast<uint32_t>(m) << 16;
  }
}

// The 16 elements negated, in fp32 (see the kernel: in these signs a -0 stays -0).
template <class T>
__device__ __forceinline__ void quant_negated(const QuantRaw<T> &r, float (&v)[16]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r.w[i] ^ 0x80000000u);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = r.w[i] ^ 0x80008000u;
      if constexpr (std::is_same_v<T, __half>) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      } else {
        v[2 * i] = __uint_as_float(w << 16);
        v[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
      }
    }
  }
}

}  // namespace gmm
