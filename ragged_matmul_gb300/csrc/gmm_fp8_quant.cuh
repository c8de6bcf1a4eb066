// Quantisation to 8-bit floating point (e4m3) with a scale for each block of 128, for sm_103a.
//
//   q = e4m3( x / s ),  s = amax / 448 (fp32), or with power-of-two scales the smallest 2^i >=
//   amax / 448 (i from -127); amax the block's largest magnitude, every step rounded to nearest
//   even, s = 0 gives q = 0.  A block that holds an infinity or a NaN gets a NaN scale and zero
//   codes, so that it stands for NaN.
// Blocks:
//   rows    128 consecutive elements of a row (the last block of a row may be shorter);
//   tiles   128 x 128 of a weight matrix (the last ones smaller);
//   cols    128 rows of one group and one column, stored transposed: q_t[c, at(r)] with the
//           group's blocks of 128 rows at columns that are multiples of 128,
//             at(r) = (first_g / 128 + g) * 128 + (r - first_g)       (first_g: the group's first row),
//           zeros behind a group's last row up to the block's end, scales always powers of two as
//           their exponent codes (i + 127).  first_g / 128 + g rises by at least the group's
//           blocks from group to group, so no prefix sum is needed, and each group's rows are a
//           K-major operand of its own for the weight gradient's MMA.
//
// All three read and write every byte once and are bound by that: tiles of 64 matrices of 2816 x 2048 bf16
// 155 us (7.1 TB/s); rows in both forms, 32768 x 4096 bf16, 93 us (5.8 TB/s; 17 instructions an element, of
// which the exact quotients of the rows take a tenth).  Quotients are the correctly
// rounded ones, as for the 4-bit formats (see gmm_fp4_quant.cuh), and powers of two divide exactly.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

#include "gmm_common.cuh"
#include "gmm_quant_raw.cuh"

namespace gmm {

constexpr int kQ8Threads = 256;
constexpr int kQ8Block = 128;
constexpr int kQ8RowLanes = 4;    // rows: lanes that share a row's block, two runs of 16 elements each
constexpr int kQ8Lanes = kQ8Block / 16;   // tiles: lanes that share a row's block
constexpr int kQ8TileRuns = kQ8Block * kQ8Lanes / kQ8Threads;   // 16-element runs of a tile a thread holds

struct Quant8Params {
  const uint8_t *x;           // rows, cols: [src_rows, width], row pitch x_pitch; tiles: [batch, rows, width] contiguous
  uint8_t *q;                 // [rows, width] (tiles: [batch, rows, width]); cols: or null
  float *scales;              // [rows, blocks] (tiles: [batch, row blocks, blocks]); cols: or null
  uint8_t *q_t;               // cols: [width, pitch]
  uint8_t *t_scales;          // cols: [pitch / 128, width]
  const uint32_t *a_offsets;  // cols: [groups + 1]
  const int32_t *row_slots;   // source row = row_slots[r] / top_k, or null (row r)
  long long x_pitch;          // bytes
  Divisor by_blocks;          // rows: units (a row's block) are numbered row by row
  Divisor by_top_k;
  int row0;                   // rows: this launch's first row
  int rows;
  int src_rows;
  int width;
  int blocks;                 // ceil(width / 128)
  int row_blocks;             // tiles: ceil(rows / 128)
  int groups;
  int pitch;                  // cols: bytes of a row of q_t, a multiple of 128
  uint32_t *status;
};

// Two e4m3 codes, `lo` in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  return pack_e4m3x2(a, b) | (pack_e4m3x2(c, d) << 16);
}

// Exponent code i + 127 of the smallest 2^i that is at least amax / 448 = amax / (1.75 * 2^8), for a
// finite amax given by its bits (a subnormal amax: 0).
__device__ __forceinline__ uint32_t pow2_code(uint32_t amax) {
  const int field = static_cast<int>(amax >> 23) - ((amax & 0x7fffffu) <= 0x600000u ? 8 : 7);
  return static_cast<uint32_t>(max(field, 0));
}
__device__ __forceinline__ float pow2_inverse(uint32_t code) {   // 2^(127 - code), code below 254
  return __uint_as_float((254u - code) << 23);
}
__device__ __forceinline__ float pow2_value(uint32_t code) { return __uint_as_float(code == 0u ? 0x00400000u : code << 23); }

// A block's scale and how to divide by it.
struct Quant8Scale {
  float s;      // the scale (NaN, 0 among them)
  float r;      // what to multiply by
  int how;      // 0: all codes are zero, 1: multiply, 2: multiply and correct, 3: divide
};

template <bool kPow2>
__device__ __forceinline__ Quant8Scale quant8_scale(uint32_t amax) {
  Quant8Scale c;
  c.how = 0;
  c.r = 0.0f;
  if (amax >= 0x7f800000u) {
    c.s = __uint_as_float(0x7fffffffu);
  } else if (amax == 0u) {
    c.s = 0.0f;
  } else if constexpr (kPow2) {
    const uint32_t code = pow2_code(amax);
    c.s = pow2_value(code);
    c.r = pow2_inverse(code);
    c.how = 1;
  } else {
    const float a = __uint_as_float(amax);
    if (amax >= 37u << 23) {   // 2^-90 and above: s > 1e-30
      // The correctly rounded a / 448: a product corrected by its remainder, compared with the
      // division for every mantissa of a.
      const float y = a * (1.0f / 448.0f);
      c.s = __fmaf_rn(__fmaf_rn(-448.0f, y, a), 1.0f / 448.0f, y);
      c.how = 2;
    } else {
      c.s = __fdiv_rn(a, 448.0f);
      c.how = c.s > 1e-30f ? 2 : (c.s > 0.0f ? 3 : 0);
    }
    if (c.how == 2) c.r = __frcp_rn(c.s);
  }
  return c;
}

// 16 elements over their block's scale, as codes.
template <class T, bool kPow2>
__device__ __forceinline__ uint4 quant8_codes(const QuantRaw<T> &raw, const Quant8Scale &c) {
  float v[16], y[16];   // -x, and x / s
  quant_negated<T>(raw, v);
  if (kPow2 && c.how == 1) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) mul_f32x2(y[i], y[i + 1], -c.r, v[i], v[i + 1]);
  } else if (!kPow2 && c.how == 2) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      mul_f32x2(y[i], y[i + 1], -c.r, v[i], v[i + 1]);      // y = x r
      fma_f32x2(v[i], v[i + 1], c.s, y[i], y[i + 1]);       // e = y s - x
      fma_f32x2(y[i], y[i + 1], -c.r, v[i], v[i + 1]);      // y - e r
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = c.how == 3 ? __fdiv_rn(-v[i], c.s) : 0.0f;
  }
  return make_uint4(pack_e4m3x4(y[0], y[1], y[2], y[3]), pack_e4m3x4(y[4], y[5], y[6], y[7]),
                    pack_e4m3x4(y[8], y[9], y[10], y[11]), pack_e4m3x4(y[12], y[13], y[14], y[15]));
}

__device__ __forceinline__ int quant8_source(const Quant8Params &p, int row) {
  if (p.row_slots == nullptr) return row;
  const int s = __ldg(p.row_slots + row);
  if (s < 0) return -1;
  const int src = static_cast<int>(p.by_top_k.quotient(static_cast<uint32_t>(s)));
  if (src < p.src_rows) return src;
  atomicOr(p.status, kStatusBadSlot);
  return -1;
}

// Rows: four lanes a block, two runs of 16 elements each (64 apart): what a block costs beside its elements (its
// place, its source row, its scale) is shared by 32 of a lane (65536 gathered rows of 2048 bf16 73 -> 56 us, 16384
// x 4096 37 -> 32, 6.2 TB/s; two blocks a lane 55 and 33, and 8 rows 2.9 us instead of 2.5).
template <class T, bool kPow2, int kAlign>
__global__ void __launch_bounds__(kQ8Threads) gmm_quantize_fp8_kernel(const __grid_constant__ Quant8Params p) {
  const uint32_t unit = blockIdx.x * (kQ8Threads / kQ8RowLanes) + threadIdx.x / kQ8RowLanes;
  const uint32_t r = p.by_blocks.quotient(unit), blk = unit - r * p.by_blocks.d;
  const uint32_t part = threadIdx.x % kQ8RowLanes, col = blk * kQ8Block + part * 16u, width = static_cast<uint32_t>(p.width);
  const uint32_t row = static_cast<uint32_t>(p.row0) + r;
  const int src = r < static_cast<uint32_t>(p.rows) ? quant8_source(p, static_cast<int>(row)) : -1;
  const uint8_t *from = p.x + src * p.x_pitch + static_cast<size_t>(col) * sizeof(T);
  QuantRaw<T> raw[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    raw[h] = QuantRaw<T>{};
    if (src >= 0 && col + 64u * h < width) raw[h] = quant_load<T, kAlign>(from + 64 * h * sizeof(T));
  }
  uint32_t amax = max(quant_amax<T>(raw[0]), quant_amax<T>(raw[1]));
#pragma unroll
  for (int o = kQ8RowLanes / 2; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (src < 0) return;
  const Quant8Scale c = quant8_scale<kPow2>(amax);
  if (part == 0) p.scales[static_cast<size_t>(row) * p.by_blocks.d + blk] = c.s;
  uint8_t *to = p.q + static_cast<size_t>(row) * width + col;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (col + 64u * h < width) *reinterpret_cast<uint4 *>(to + 64 * h) = quant8_codes<T, kPow2>(raw[h], c);
}

// Tiles: a CTA holds one in registers.
template <class T, bool kPow2, int kAlign>
__global__ void __launch_bounds__(kQ8Threads) gmm_quantize_fp8_tiles_kernel(const __grid_constant__ Quant8Params p) {
  __shared__ uint32_t warp_max[kQ8Threads / 32];
  const uint32_t per = static_cast<uint32_t>(p.blocks) * p.row_blocks;
  const uint32_t b = blockIdx.x / per, in = blockIdx.x - b * per, rb = in / p.blocks, cb = in - rb * p.blocks;
  const uint32_t col = cb * kQ8Block + threadIdx.x % kQ8Lanes * 16u, row0 = rb * kQ8Block + threadIdx.x / kQ8Lanes;
  const size_t base = static_cast<size_t>(b) * p.rows;
  QuantRaw<T> raw[kQ8TileRuns];
  uint32_t amax = 0;
#pragma unroll
  for (int u = 0; u < kQ8TileRuns; ++u) {
    const uint32_t row = row0 + static_cast<uint32_t>(u) * (kQ8Threads / kQ8Lanes);
    raw[u] = QuantRaw<T>{};
    if (row < static_cast<uint32_t>(p.rows) && col < static_cast<uint32_t>(p.width))
      raw[u] = quant_load<T, kAlign>(p.x + ((base + row) * p.width + col) * sizeof(T));
  }
#pragma unroll
  for (int u = 0; u < kQ8TileRuns; ++u) amax = max(amax, quant_amax<T>(raw[u]));
  amax = __reduce_max_sync(0xffffffffu, amax);
  if ((threadIdx.x & 31u) == 0) warp_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQ8Threads / 32; ++w) amax = max(amax, warp_max[w]);
  const Quant8Scale c = quant8_scale<kPow2>(amax);
  if (threadIdx.x == 0) p.scales[blockIdx.x] = c.s;
#pragma unroll
  for (int u = 0; u < kQ8TileRuns; ++u) {
    const uint32_t row = row0 + static_cast<uint32_t>(u) * (kQ8Threads / kQ8Lanes);
    if (row < static_cast<uint32_t>(p.rows) && col < static_cast<uint32_t>(p.width))
      *reinterpret_cast<uint4 *>(p.q + (base + row) * p.width + col) = quant8_codes<T, kPow2>(raw[u], c);
  }
}

// Eight consecutive elements.
template <class T>
struct QuantRaw8 { uint32_t w[sizeof(T) * 2]; };

template <class T, bool kVec>
__device__ __forceinline__ QuantRaw8<T> quant_load8(const uint8_t *p) {
  QuantRaw8<T> r;
  constexpr int kWords = sizeof(r.w) / 4;
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) *reinterpret_cast<uint4 *>(&r.w[4 * i]) = __ldg(reinterpret_cast<const uint4 *>(p) + i);
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

template <class T>
__device__ __forceinline__ float quant_value8(const QuantRaw8<T> &r, int i) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(r.w[i]);
  else if constexpr (std::is_same_v<T, __half>)
    return __half2float(__ushort_as_half(static_cast<unsigned short>(r.w[i / 2] >> (16 * (i & 1)))));
  else return __uint_as_float((i & 1) ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
}

// The element negated, its sign flipped in the word so that -0 keeps it.
template <class T>
__device__ __forceinline__ float quant_negated8(const QuantRaw8<T> &r, int i) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(r.w[i] ^ 0x80000000u);
  const uint32_t w = r.w[i / 2] ^ 0x80008000u;
  if constexpr (std::is_same_v<T, __half>) return __half2float(__ushort_as_half(static_cast<unsigned short>(w >> (16 * (i & 1)))));
  else return __uint_as_float((i & 1) ? w & 0xffff0000u : w << 16);
}

// Magnitudes in the order of fp32's bits: of 16-bit types two to a word, compared as they stand.
template <class T>
struct QuantMax8 { uint32_t w[sizeof(T) * 2]; };

template <class T>
__device__ __forceinline__ uint32_t quant_mag(uint32_t a, uint32_t b) {   // max(a, |b|)
  if constexpr (sizeof(T) == 4) return max(a, b & 0x7fffffffu);
  else return __vmaxu2(a, b & 0x7fff7fffu);
}
template <class T>
__device__ __forceinline__ uint32_t quant_max2(uint32_t a, uint32_t b) {
  if constexpr (sizeof(T) == 4) return max(a, b);
  else return __vmaxu2(a, b);
}
// One magnitude of the type as fp32 bits.
template <class T>
__device__ __forceinline__ uint32_t quant_bits(uint32_t m) {
  if constexpr (sizeof(T) == 4) return m;
  else if constexpr (std::is_same_v<T, __half>) return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
  else return m << 16;
}

// Cols: a CTA takes 128 rows of a group and 128 columns (four CTAs an SM for 16-bit rows: 99 us, 114 with
// three); thread (cv, rg) holds 8 columns from 8 cv
// of 8 rows from 8 rg, so that a warp's load is two whole row pieces, a column's codes of 8 rows are
// 8 bytes of the transposed tile in shared memory, and a row's codes of 8 columns 8 bytes of q.
template <class T, bool kVec, bool kBoth>
__global__ void __launch_bounds__(kQ8Threads, sizeof(T) == 2 ? 4 : 2) gmm_quantize_fp8_cols_kernel(const __grid_constant__ Quant8Params p) {
  constexpr int kWords = sizeof(T) * 2, kWarps = kQ8Threads / 32;
  __shared__ __align__(16) uint8_t tile[kQ8Block * kQ8Block];
  __shared__ uint32_t part[kWarps][kWords * 16];
  __shared__ __align__(16) float inv[kQ8Block];
  __shared__ float2 row_scale[kQ8Block];
  __shared__ uint32_t s_first, s_rows;
  const int tid = threadIdx.x, cv = tid & 15, rg = tid >> 4, lane = tid & 31, warp = tid >> 5;
  const uint32_t block = blockIdx.x / static_cast<uint32_t>(p.blocks), cb = blockIdx.x - block * p.blocks;

  // The group whose blocks hold this one; offsets that decrease or lead past the buffers: nothing.  Up to 32
  // groups every warp looks for itself, which saves two barriers.
  bool bad = false;
  uint32_t first = 0, n = 0;
  auto look = [&](int g) {
    const uint32_t r0 = __ldg(p.a_offsets + g), r1 = __ldg(p.a_offsets + g + 1);
    bad |= r1 < r0 || r1 > static_cast<uint32_t>(p.rows);
    const uint32_t at = block - (r0 / kQ8Block + static_cast<uint32_t>(g));   // of the group's blocks
    if (!bad && at < 0x80000000u && at * kQ8Block < r1 - r0) {
      first = r0 + at * kQ8Block;
      n = min(static_cast<uint32_t>(kQ8Block), r1 - r0 - at * kQ8Block);
    }
  };
  if (p.groups <= 32) {
    if (lane < p.groups) look(lane);
    bad = __any_sync(0xffffffffu, bad);
    n = __reduce_max_sync(0xffffffffu, n);
    first = __reduce_max_sync(0xffffffffu, first);
  } else {
    if (tid == 0) s_rows = 0;
    __syncthreads();
    for (int g = tid; g < p.groups; g += kQ8Threads) look(g);
    if (n != 0) {
      s_first = first;
      s_rows = n;
    }
    bad = __syncthreads_or(bad);
    n = s_rows;
    first = s_first;
  }
  if (bad) {
    if (tid == 0 && blockIdx.x == 0) atomicOr(p.status, kStatusBadOffsets);
    return;
  }
  if (n == 0) return;   // no group's block

  // Source rows: the lane of column piece i < 8 finds the one of row rg 8 + i.
  int src = -1;
  if (cv < 8 && static_cast<uint32_t>(rg * 8 + cv) < n) src = quant8_source(p, static_cast<int>(first) + rg * 8 + cv);
  const uint32_t live = (__ballot_sync(0xffffffffu, src >= 0) >> (lane & 16)) & 0xffu;   // bit i: row rg 8 + i has one

  const int c0 = static_cast<int>(cb) * kQ8Block, col = c0 + cv * 8;
  const bool in = col < p.width;
  QuantRaw8<T> raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    raw[i] = QuantRaw8<T>{};
    const int from = __shfl_sync(0xffffffffu, src, (lane & 16) + i);
    if (from >= 0 && in) raw[i] = quant_load8<T, kVec>(p.x + from * p.x_pitch + static_cast<long long>(col) * sizeof(T));
  }

  // Largest magnitudes of the columns: over the thread's rows, the warp's, the CTA's.
  uint32_t m[kWords];
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    m[k] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m[k] = quant_mag<T>(m[k], raw[i].w[k]);
    m[k] = quant_max2<T>(m[k], __shfl_xor_sync(0xffffffffu, m[k], 16));
  }
  if (lane < 16)
#pragma unroll
    for (int k = 0; k < kWords; ++k) part[warp][cv * kWords + k] = m[k];

  if constexpr (kBoth) {
    // Largest magnitudes of the rows, over 16 lanes: every step halves the rows that a lane has left,
    // so that two lanes end with each row, and its division is made once instead of in every lane.
    uint32_t a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = 0;
#pragma unroll
      for (int k = 0; k < kWords; ++k) a[i] = quant_mag<T>(a[i], raw[i].w[k]);
      if constexpr (sizeof(T) == 2) a[i] = max(a[i] & 0xffffu, a[i] >> 16);
    }
    int mine = 0;   // this lane's row of the eight
#pragma unroll
    for (int half = 4; half > 0; half >>= 1) {
      const bool up = (lane & (2 * half)) != 0;
      mine += up ? half : 0;
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const uint32_t sent = up ? a[i] : a[i + half], kept = up ? a[i + half] : a[i];
        a[i] = max(kept, __shfl_xor_sync(0xffffffffu, sent, 2 * half));
      }
    }
    a[0] = max(a[0], __shfl_xor_sync(0xffffffffu, a[0], 1));
    const Quant8Scale c = quant8_scale<false>(quant_bits<T>(a[0]));
    const int r = rg * 8 + mine;
    if ((lane & 1) == 0) {
      row_scale[r] = make_float2(c.s, c.how == 3 ? -1.0f : c.r);   // -1: divide; 0: all codes are zero
      if ((live >> mine) & 1u)
        p.scales[static_cast<size_t>(first + static_cast<uint32_t>(r)) * p.blocks + cb] = c.s;
    }
    __syncwarp();
    uint8_t *out = p.q + static_cast<size_t>(first + static_cast<uint32_t>(rg * 8)) * p.width + col;
#pragma unroll
    for (int i = 0; i < 8; ++i, out += p.width) {
      if (!((live >> i) & 1u) || !in) continue;
      const float2 f = row_scale[rg * 8 + i];
      float v[8], y[8];   // -x, and x / s
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = quant_negated8<T>(raw[i], j);
      if (f.y > 0.0f) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          mul_f32x2(y[j], y[j + 1], -f.y, v[j], v[j + 1]);
          fma_f32x2(v[j], v[j + 1], f.x, y[j], y[j + 1]);
          fma_f32x2(y[j], y[j + 1], -f.y, v[j], v[j + 1]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = f.y < 0.0f ? __fdiv_rn(-v[j], f.x) : 0.0f;
      }
      *reinterpret_cast<uint2 *>(out) = make_uint2(pack_e4m3x4(y[0], y[1], y[2], y[3]), pack_e4m3x4(y[4], y[5], y[6], y[7]));
    }
  }
  __syncthreads();
  if (tid < kQ8Block) {
    uint32_t a = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t x = part[w][sizeof(T) == 4 ? tid : tid / 2];
      a = max(a, sizeof(T) == 4 ? x : (x >> (16 * (tid & 1))) & 0xffffu);
    }
    a = quant_bits<T>(a);
    const uint32_t code = a >= 0x7f800000u ? 0xffu : pow2_code(a);
    // A block that is not finite, or zeros of any sign: zero codes, by a mark that no inverse has.
    inv[tid] = code == 0xffu || a == 0u ? -1.0f : pow2_inverse(code);
    if (c0 + tid < p.width) p.t_scales[static_cast<size_t>(block) * p.width + c0 + tid] = static_cast<uint8_t>(code);
  }
  __syncthreads();

  // The columns' codes, eight rows of a column at a time: chunk rg / 2 of the column's 128 bytes, its
  // place turned by cv so that the warp's stores spread over the banks.
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float f = inv[cv * 8 + j];
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      mul_f32x2(y[i], y[i + 1], f, quant_value8<T>(raw[i], j), quant_value8<T>(raw[i + 1], j));
    uint2 w = make_uint2(pack_e4m3x4(y[0], y[1], y[2], y[3]), pack_e4m3x4(y[4], y[5], y[6], y[7]));
    if (f < 0.0f) w = make_uint2(0u, 0u);
    *reinterpret_cast<uint2 *>(tile + (cv * 8 + j) * kQ8Block + ((((rg >> 1) ^ cv) & 7) << 4) + ((rg & 1) << 3)) = w;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kQ8Block * 8 / kQ8Threads; ++u) {
    const int at = u * kQ8Threads + tid, c = at >> 3, chunk = at & 7;
    if (c0 + c < p.width)
      *reinterpret_cast<uint4 *>(p.q_t + static_cast<size_t>(c0 + c) * p.pitch + static_cast<size_t>(block) * kQ8Block + chunk * 16) =
          *reinterpret_cast<const uint4 *>(tile + c * kQ8Block + (((chunk ^ (c >> 3)) & 7) << 4));
  }
}

}  // namespace gmm
