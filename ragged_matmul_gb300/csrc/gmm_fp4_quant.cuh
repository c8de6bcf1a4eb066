// Microscaled 4-bit floating point: quantisation and its inverse, for sm_103a.
//
// A value is e2m1 (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) times
// the scale of its block of consecutive K:
//   nvfp4   block 16, scale s e4m3, times an optional fp32 global scale g (1 without it):
//             s = e4m3( amax / (6 g) ),  d = s g
//   mxfp4   block 32, scale a power of two (e8m0, code = exponent + 127):
//             d = 2^( floor(log2 amax) - 2 )   (code 0 for amax = 0 or below 2^-124)
//   q = e2m1( x / d ), both roundings to nearest even, saturating at 448 and 6; d = 0: q = 0.
// A block whose largest magnitude is infinite or NaN gets a NaN scale (0x7F / 0xFF) and
// zero codes, so that it stands for NaN.
// Packed: element k in nibble k % 2 (low nibble first) of byte k / 2.  A row's scale bytes
// are padded with zeros to a multiple of 16.
//
// The quotient x / d decides ties between neighbouring codes, and inputs of few mantissa
// bits over a scale of few mantissa bits hit them often, so it is the correctly rounded
// quotient and not x times a rounded reciprocal.  A division per element would cost more
// than the memory traffic; with r = 1 / d rounded once per block, y = x r and the exact
// remainder e = y d - x (one fused multiply-add), y - e r is the correctly rounded quotient
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990): three instructions.  Scales and quotients so small or large that a step could leave
// the normal range take the division itself.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "gmm_route.cuh"

namespace gmm {

constexpr int kQuantThreads = 256;
constexpr int kQuantPer = 2;     // 16-element blocks a thread, quantisation
constexpr int kDequantPer = 4;   // and its inverse
constexpr uint32_t kE4m3Nan = 0x7Fu, kE8m0Nan = 0xFFu;

struct QuantParams {
  const uint8_t *x;           // quantise: [*, K], row pitch x_pitch; dequantise: the output
  uint8_t *packed;            // [rows, K / 2]
  uint8_t *scales;            // [rows, scale_pitch]
  const int32_t *row_slots;   // quantise: source row = row_slots[r] / top_k, or null (row r)
  const float *global_scale;  // one value, or null (1)
  long long x_pitch;          // bytes
  int row0;                   // this launch's rows: row0 .. row0 + rows - 1
  int rows;
  uint32_t div_mul;           // block / (K / 16) = umulhi(block, div_mul) >> div_shift, for block < 2^31
  uint32_t div_shift;
  int src_rows;               // rows of x
  int K;
  int scale_pitch;
  int top_k;
  uint32_t *status;
};

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

// Eight values to eight e2m1 codes, the first in the lowest nibble.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float *v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

__device__ __forceinline__ uint32_t float_to_e4m3(float x) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(x));
  return r & 0xffu;
}

__device__ __forceinline__ float e4m3_to_float(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(code)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xffffu)));
}

// 2^(code - 127); code 0 is 2^-127 (a subnormal), 255 is NaN.
__device__ __forceinline__ float e8m0_to_float(uint32_t code) {
  return __uint_as_float(code == 0 ? 0x00400000u : (code == kE8m0Nan ? 0x7fffffffu : code << 23));
}

// Where 16-element block `idx` of the call lies, and whether there is one.
struct QuantAt {
  int row;        // row of packed and scales
  int src;        // row of x (-1: none)
  uint32_t blk;   // 16-element block within the row
  bool live;
};

__device__ __forceinline__ QuantAt quant_at(const QuantParams &p, uint32_t idx, uint32_t per_row) {
  QuantAt a;
  const uint32_t row = __umulhi(idx, p.div_mul) >> p.div_shift;
  const bool in = row < static_cast<uint32_t>(p.rows);
  a.row = p.row0 + static_cast<int>(in ? row : 0u);
  a.blk = idx - row * per_row;
  a.src = a.row;
  if (in && p.row_slots != nullptr) {
    const int s = __ldg(p.row_slots + a.row);
    a.src = s < 0 ? -1 : s / p.top_k;
    if (a.src >= p.src_rows) {
      atomicOr(p.status, kStatusBadSlot);
      a.src = -1;
    }
  }
  a.live = in && a.src >= 0;
  return a;
}

// Bound by the bytes of x and the codes (32768 rows of 4096 bf16 to mxfp4 and back in 105 us,
// 6.5 TB/s; nvfp4's arithmetic takes a fifth more).  A thread takes kQuantPer blocks of 16 elements,
// kQuantThreads apart, with their loads in flight together (one left 49 KB of an SM's loads in
// flight, at the limit of the latency); the two threads of an mxfp4 block exchange their maxima.
template <class T, bool kMx, int kAlign>
__global__ void __launch_bounds__(kQuantThreads) gmm_quantize_fp4_kernel(const __grid_constant__ QuantParams p) {
  const uint32_t per_row = static_cast<uint32_t>(p.K) / 16u;   // K is a multiple of 32: even
  const uint32_t idx0 = blockIdx.x * (kQuantThreads * kQuantPer) + threadIdx.x;
  QuantAt at[kQuantPer];
  QuantRaw<T> raw[kQuantPer];
#pragma unroll
  for (int u = 0; u < kQuantPer; ++u) {   // both threads of a block agree on it: they share the row
    at[u] = quant_at(p, idx0 + static_cast<uint32_t>(u) * kQuantThreads, per_row);
    raw[u] = QuantRaw<T>{};
    if (at[u].live)
      raw[u] = quant_load<T, kAlign>(p.x + at[u].src * p.x_pitch + static_cast<long long>(at[u].blk) * 16 * sizeof(T));
  }
  const float g = !kMx && p.global_scale != nullptr ? __ldg(p.global_scale) : 1.0f;
#pragma unroll
  for (int u = 0; u < kQuantPer; ++u) {
    const uint32_t blk = at[u].blk;
    uint32_t amax = quant_amax<T>(raw[u]);
    if (kMx) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    if (!at[u].live) continue;
    float v[16], y[16];   // -x, and x / d
    quant_negated<T>(raw[u], v);
    uint32_t code;
    if (amax >= 0x7f800000u) {
      code = kMx ? kE8m0Nan : kE4m3Nan;
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = 0.0f;
    } else if constexpr (kMx) {
      // floor(log2 amax) is the exponent field less 127; a subnormal's field is 0.
      const uint32_t field = amax >> 23;
      code = field > 2u ? field - 2u : 0u;
      // 1 / d is a power of two too, and x / d is x with another exponent.
      const float inv = __uint_as_float((254u - code) << 23);   // code is at most 252
#pragma unroll
      for (int i = 0; i < 16; i += 2) mul_f32x2(y[i], y[i + 1], -inv, v[i], v[i + 1]);
    } else {
      code = float_to_e4m3(__fdiv_rn(__uint_as_float(amax), 6.0f * g));
      const float d = e4m3_to_float(code) * g;
      const float r = __frcp_rn(d);
      if (d > 1e-30f && d < 1e30f && __uint_as_float(amax) * r < 1e30f) {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          mul_f32x2(y[i], y[i + 1], -r, v[i], v[i + 1]);      // y = x r
          fma_f32x2(v[i], v[i + 1], d, y[i], y[i + 1]);       // e = y d - x
          fma_f32x2(y[i], y[i + 1], -r, v[i], v[i + 1]);      // y - e r
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = d == 0.0f ? 0.0f : __fdiv_rn(-v[i], d);
      }
    }
    const uint2 w = make_uint2(pack_e2m1x8(y), pack_e2m1x8(y + 8));
    reinterpret_cast<uint2 *>(p.packed + static_cast<size_t>(at[u].row) * (p.K / 2))[blk] = w;
    uint8_t *srow = p.scales + static_cast<size_t>(at[u].row) * p.scale_pitch;
    if (kMx) {
      if ((blk & 1u) == 0) srow[blk >> 1] = static_cast<uint8_t>(code);
    } else {
      srow[blk] = static_cast<uint8_t>(code);
    }
    if (blk == per_row - 1)   // the row's padding
      for (int i = static_cast<int>(kMx ? per_row / 2 : per_row); i < p.scale_pitch; ++i) srow[i] = 0;
  }
}

// One byte (two e2m1 codes) to two fp32 values.
__device__ __forceinline__ float2 e2m1x2_to_float2(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 b, x, y, z;\n\tmov.b32 {b, x, y, z}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
      : "=r"(h)
      : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// y = q * (s * g), the product of the scales rounded to fp32 once, then once to T.  Bound by
// the bytes of y; a thread takes kDequantPer blocks of 16 elements.
template <class T, bool kMx, int kAlign>
__global__ void __launch_bounds__(kQuantThreads) gmm_dequantize_fp4_kernel(const __grid_constant__ QuantParams p) {
  const uint32_t per_row = static_cast<uint32_t>(p.K) / 16u;
  const uint32_t idx0 = blockIdx.x * (kQuantThreads * kDequantPer) + threadIdx.x;
  const float g = !kMx && p.global_scale != nullptr ? __ldg(p.global_scale) : 1.0f;
  uint2 w[kDequantPer];
  uint32_t code[kDequantPer];
#pragma unroll
  for (int u = 0; u < kDequantPer; ++u) {
    const uint32_t idx = idx0 + static_cast<uint32_t>(u) * kQuantThreads, q = __umulhi(idx, p.div_mul) >> p.div_shift;
    if (q >= static_cast<uint32_t>(p.rows)) continue;
    const uint32_t blk = idx - q * per_row;
    const size_t row = static_cast<size_t>(p.row0) + q;
    w[u] = __ldg(reinterpret_cast<const uint2 *>(p.packed + row * (p.K / 2)) + blk);
    code[u] = __ldg(p.scales + row * p.scale_pitch + (kMx ? blk >> 1 : blk));
  }
#pragma unroll
  for (int u = 0; u < kDequantPer; ++u) {
    const uint32_t idx = idx0 + static_cast<uint32_t>(u) * kQuantThreads, q = __umulhi(idx, p.div_mul) >> p.div_shift;
    if (q >= static_cast<uint32_t>(p.rows)) continue;
    const uint32_t blk = idx - q * per_row;
    const size_t row = static_cast<size_t>(p.row0) + q;
    float d;
    if constexpr (kMx) d = e8m0_to_float(code[u]);
    else d = e4m3_to_float(code[u]) * g;
    alignas(32) T y[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = e2m1x2_to_float2(((i < 4 ? w[u].x : w[u].y) >> (8 * (i & 3))) & 0xffu);
      y[2 * i] = route_from_float<T>(f.x * d);
      y[2 * i + 1] = route_from_float<T>(f.y * d);
    }
    T *out = reinterpret_cast<T *>(const_cast<uint8_t *>(p.x) + row * p.x_pitch) + static_cast<size_t>(blk) * 16;
    if constexpr (kAlign == 32) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
        st_global_v8(reinterpret_cast<uint8_t *>(out) + 32 * i, reinterpret_cast<const uint32_t *>(y) + 8 * i);
    } else if constexpr (kAlign == 16) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)); ++i)
        reinterpret_cast<uint4 *>(out)[i] = reinterpret_cast<const uint4 *>(y)[i];
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) out[i] = y[i];
    }
  }
}

}  // namespace gmm
