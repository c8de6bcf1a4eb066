// A router's choice of experts and its gradient, for sm_103a.
//
// For token t with logits x_e (E experts) and a score function
//   softmax   s_e = exp(x_e) / sum_i exp(x_i)
//   sigmoid   s_e = 1 / (1 + exp(-x_e))
// the experts are chosen by the key y_e = s_e + b_e (b: an optional bias that only the choice
// sees):
//   groups    the experts are `groups` equal runs; a group's key is the sum of its group_top (1
//             or 2) largest y_e, and only the top_groups groups with the largest keys are kept;
//   choice    the top_k largest y_e of the kept groups, in descending order;
//   weights   w_j = scale * s_j, or scale * s_j / sum_i s_i over the chosen (renormalise).
// Equal keys go to the lowest index.  An expert whose key is -infinity or NaN (a masked logit or
// bias) is never chosen; slots that find no expert get id -1 and weight 0.  A token with a NaN
// logit (or, with softmax, one of +infinity) gets none at all and is reported.
//
// Gradient, with g_j = scale * d w_j and the chosen ids given:
//   renormalised, u_j = s_j / sum_i s_i:
//     softmax   d x_j = u_j (g_j - sum_i u_i g_i)
//     sigmoid   d x_j = u_j (g_j - sum_i u_i g_i) (1 - s_j)
//   not renormalised:
//     softmax   d x_e = s_e (sum_{j: id_j = e} g_j - sum_j s_j g_j)        (every expert)
//     sigmoid   d x_j = g_j s_j (1 - s_j)
// and zero elsewhere; slots that name an expert twice add up.
//
// The choice is that of the keys to 64-bit accuracy.  Without a bias the scores stand in the order of
// the logits, which are compared themselves; a group's sum of two is a score pair.  Where fp32 keys
// (with a bias) or sums are nearer than their error bounds and of different logit or bias, those
// near enough to matter are computed again in 64 bits (about one token in a hundred at 256 experts),
// because fp32 sums of near keys would otherwise choose by their rounding.
//
// Bound by latency and, with many tokens, by instruction issue (integer minimum and maximum run at
// half rate).  L lanes hold a token's logits in registers, V each, as unsigned keys in the order of the
// values.  16-bit logits carry the expert's number in their key's low half, and sorted lists of eight are
// merged across the lanes.  Of 32-bit keys those that reach a bound are gathered, a lane each, and
// ranked against one another, which also settles ties.
// Measured: 32768 tokens of 128 bf16 logits, top-8, 6.0 us (their bytes
// take 1.5); 256 tokens of 256 fp32 logits with a bias and groups 4.4 us, 5.6 with a token in 64 bits; one token
// 1.8 us, about an empty launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

#include "gmm_common.cuh"

namespace gmm {

constexpr int kScoreSoftmax = 0;
constexpr int kScoreSigmoid = 1;
constexpr int kChooseWarps = 4;
constexpr int kChooseMaxGroups = 32;    // one lane at least holds a group
constexpr int kChooseMaxPerLane = 128;  // logits a lane holds, at most

struct ChooseParams {
  const uint8_t *logits;        // [tokens, E], row pitch logits_pitch
  long long logits_pitch;       // bytes
  const float *bias;            // [E] or null
  int32_t *ids;                 // [tokens, top_k]; the gradient's input
  float *weights;               // [tokens, top_k]; gradient: d_weights
  uint8_t *d_logits;            // gradient: [tokens, E], row pitch d_pitch
  long long d_pitch;            // bytes
  int num_tokens;
  int num_experts;
  int top_k;
  int scoring;
  int groups;
  int group_size;               // experts per group
  int group_lanes;              // lanes per group: a token's lanes / (groups rounded up to a power of two)
  int top_groups;
  int group_top;
  int renormalise;
  int bias_vec;                 // bias is 16-byte aligned
  float scale;
  uint32_t *status;
};

__device__ __forceinline__ uint32_t redux_max(uint32_t x) {
  uint32_t r;
  asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(r) : "r"(x));
  return r;
}

// Maximum over the L lanes of a token.
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
  if constexpr (L == 32) {
    return redux_max(x);
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
  }
}

template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Words in the order of the values, 0 for -infinity and NaN (never chosen); -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t k = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return x > -INFINITY ? k : 0u;
}
__device__ __forceinline__ float key_value(uint32_t k) {   // its inverse; -infinity for 0
  return k == 0u ? -INFINITY : __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long order_key(double x) {
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(x + 0.0));
  const unsigned long long k = (b >> 63) ? ~b : b | (1ull << 63);
  return x > -static_cast<double>(INFINITY) ? k : 0ull;
}

template <class T>
__device__ __forceinline__ float choose_float(T x) {
  if constexpr (std::is_same_v<T, float>) return x;
  else if constexpr (std::is_same_v<T, __half>) return __half2float(x);
  else return __bfloat162float(x);
}

// Where a lane's V logits lie.  kRun (every lane's run is whole, its rows aligned to 16 bytes or the run's
// size): consecutive, one vector load.  Else a lane's logits are `step` apart, so that the lanes of a
// token (of a group) read consecutive ones.
template <bool kRun>
struct ChoosePlace {
  int first, step, end;   // experts first + v (* step), below `end`
  __device__ __forceinline__ ChoosePlace(int base, int size, int lane, int lanes, int V)
      : first(base + (kRun ? lane * V : lane)), step(lanes), end(base + size) {}
  __device__ __forceinline__ int expert(int v) const { return kRun ? first + v : first + v * step; }
  __device__ __forceinline__ bool there(int v) const { return kRun ? first < end : first + v * step < end; }
};

// A lane's logits as fp32, -infinity where there is none.
template <class T, int V, bool kVec>
__device__ __forceinline__ void choose_load(const T *row, const ChoosePlace<kVec> &at, float (&x)[V]) {
  constexpr int kBytes = V * static_cast<int>(sizeof(T));
  if constexpr (kVec) {
    alignas(16) T raw[V];
    const bool there = at.there(0);
    if (there) {
      if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
          reinterpret_cast<uint4 *>(raw)[i] = __ldg(reinterpret_cast<const uint4 *>(row + at.first) + i);
      } else if constexpr (kBytes == 8) {
        *reinterpret_cast<uint2 *>(raw) = __ldg(reinterpret_cast<const uint2 *>(row + at.first));
      } else {
        *reinterpret_cast<uint32_t *>(raw) = __ldg(reinterpret_cast<const uint32_t *>(row + at.first));
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = there ? choose_float<T>(raw[v]) : -INFINITY;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = at.there(v) ? choose_float<T>(row[at.expert(v)]) : -INFINITY;
  }
}

// 16-bit logits compared as they stand.  A key holds the logit's 16 bits in the order of the values above
// 65535 less the expert's number, so that the largest key is the largest logit's lowest expert.
template <class T>
struct Packed16 {
  static constexpr uint32_t kMinusInf = std::is_same_v<T, __half> ? 0x03ffu : 0x007fu;   // of -infinity
  static constexpr uint32_t kPlusInf = std::is_same_v<T, __half> ? 0xfc00u : 0xff80u;    // of +infinity; NaN is above
  static constexpr uint32_t kPad = std::is_same_v<T, __half> ? 0xfc00fc00u : 0xff80ff80u;   // two logits of -infinity
  static constexpr uint32_t kNone = kMinusInf << 16 | 0xffffu;   // keys up to here are never chosen
  __device__ __forceinline__ static uint32_t canonical(uint32_t w) {   // -0 becomes +0, a NaN a positive one
    if constexpr (std::is_same_v<T, __half>) {
      const __half2 h = __hadd2(*reinterpret_cast<const __half2 *>(&w), __half2half2(__ushort_as_half(0)));
      return *reinterpret_cast<const uint32_t *>(&h);
    } else {
      const __nv_bfloat162 h = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&w), __bfloat162bfloat162(__ushort_as_bfloat16(0)));
      return *reinterpret_cast<const uint32_t *>(&h);
    }
  }
  __device__ __forceinline__ static float value(uint32_t bits) {   // of 16 bits
    if constexpr (std::is_same_v<T, __half>) return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
    else return __uint_as_float(bits << 16);
  }
  __device__ __forceinline__ static float key_value(uint32_t key) {
    const uint32_t k = key >> 16;
    return value((k & 0x8000u) ? k & 0x7fffu : ~k & 0xffffu);
  }
  // Two keys of a word of two logits, experts e0 and e1.
  __device__ __forceinline__ static void keys(uint32_t w, uint32_t e0, uint32_t e1, uint32_t &k0, uint32_t &k1) {
    uint32_t sign;   // each half all ones where it is negative
    asm("prmt.b32 %0, %1, 0, 0xbb99;" : "=r"(sign) : "r"(w));
    const uint32_t k = w ^ (sign | 0x80008000u);
    k0 = (k << 16) | (0xffffu - e0);
    k1 = (k & 0xffff0000u) | (0xffffu - e1);
  }
};

// A lane's 16-bit logits as words of two, -infinity where there is none.
template <class T, int V, bool kVec>
__device__ __forceinline__ void choose_load16(const T *row, const ChoosePlace<kVec> &at, uint32_t (&w)[V / 2]) {
  constexpr uint32_t kPad = Packed16<T>::kPad;
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = kPad;
    if (at.there(0)) {
      if constexpr (V >= 8) {
#pragma unroll
        for (int i = 0; i < V / 8; ++i)
          *reinterpret_cast<uint4 *>(&w[4 * i]) = __ldg(reinterpret_cast<const uint4 *>(row + at.first) + i);
      } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t *>(row + at.first) + i);
      }
    }
  } else {
    const unsigned short *p = reinterpret_cast<const unsigned short *>(row);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const uint32_t a = at.there(2 * i) ? __ldg(p + at.expert(2 * i)) : kPad & 0xffffu;
      const uint32_t b = at.there(2 * i + 1) ? __ldg(p + at.expert(2 * i + 1)) : kPad & 0xffffu;
      w[i] = a | (b << 16);
    }
  }
}

// Off by about 4 units in the last place (the quotient by 2).  Below -20 the exponential itself (1 + exp(x) is 1 to
// 2.1e-9), which keeps the scores under 2^-126 that the quotient makes 0.
__device__ __forceinline__ float sigmoid32(float x) {
  const float e = expf(x < -20.0f ? x : -x);
  return x < -20.0f ? e : __fdividef(1.0f, 1.0f + e);
}
// A chosen expert's score over a factor that the token's others share, m the largest chosen logit: relative to m's score
// (softmax, and sigmoids that are exponentials all), else times 2^64, so that small ones keep their bits next to m's.
__device__ __forceinline__ float relative_score(bool softmax, float x, float m) {
  if (softmax || m < -20.0f) return expf(x - m);
  const float e = expf(0.5f * x);
  return x < -20.0f ? e * (e * 0x1p64f) : sigmoid32(x) * 0x1p64f;
}
// For keys, which allow for its error: 2.7e-7 at most (the exponential of 2^-22 relative and 2^-24 a unit of x,
// times s (1 - s); the sum half a step, the quotient one unit in the last place).
__device__ __forceinline__ float sigmoid_key(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-x)));
  return r;
}
__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

// The largest two of a run of lanes, each lane with its own two.
__device__ __forceinline__ void merge_top2(float &a1, float &a2, float b1, float b2) {
  a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
  a1 = fmaxf(a1, b1);
}

// Sorted lists of the eight largest keys, in registers.
__device__ __forceinline__ void order2(uint32_t &hi, uint32_t &lo) {
  const uint32_t a = max(hi, lo), b = min(hi, lo);
  hi = a;
  lo = b;
}
__device__ __forceinline__ void sort8(uint32_t (&a)[8]) {   // descending, the 19-comparator network
  order2(a[0], a[2]), order2(a[1], a[3]), order2(a[4], a[6]), order2(a[5], a[7]);
  order2(a[0], a[4]), order2(a[1], a[5]), order2(a[2], a[6]), order2(a[3], a[7]);
  order2(a[0], a[1]), order2(a[2], a[3]), order2(a[4], a[5]), order2(a[6], a[7]);
  order2(a[2], a[4]), order2(a[3], a[5]);
  order2(a[1], a[4]), order2(a[3], a[6]);
  order2(a[1], a[2]), order2(a[3], a[4]), order2(a[5], a[6]);
}
// a: the eight largest of two sorted lists, sorted.  The larger of a[i] and b[7 - i] are these eight, rising
// and falling once, which three rounds of comparators at distances 4, 2, 1 sort (Batcher's merge).
__device__ __forceinline__ void merge8(uint32_t (&a)[8], const uint32_t (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = max(a[i], b[7 - i]);
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & d) == 0) order2(a[i], a[i + d]);
}
// The eight largest keys of a token's L lanes, in every one of them.
template <int L, int V>
__device__ __forceinline__ void largest8(const uint32_t (&key)[V], uint32_t (&a)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = i < V ? key[i] : 0u;
  sort8(a);
#pragma unroll
  for (int c = 8; c < V; c += 8) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = key[c + i];
    sort8(b);
    merge8(a, b);
  }
#pragma unroll
  for (int o = 1; o < L; o <<= 1) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __shfl_xor_sync(0xffffffffu, a[i], o);
    merge8(a, b);
  }
}
__device__ __forceinline__ uint32_t pick8(const uint32_t (&a)[8], int j) {   // a[j & 7]
  const uint32_t w = (j & 1) ? a[1] : a[0], x = (j & 1) ? a[3] : a[2], y = (j & 1) ? a[5] : a[4], z = (j & 1) ? a[7] : a[6];
  const uint32_t u = (j & 2) ? x : w, v = (j & 2) ? z : y;
  return (j & 4) ? v : u;
}

// Score of logit x in 64 bits; zd: softmax's sum relative to `top`.
__device__ __forceinline__ double score64(int scoring, float x, float top, double zd) {
  return scoring == kScoreSoftmax ? exp(static_cast<double>(x) - static_cast<double>(top)) / zd : sigmoid64(static_cast<double>(x));
}

// Whether the key of (xi, bi) is surely above that of (xj, bj), by their difference: s_i - s_j is s of the larger
// logit times 1 - exp(-d) (sigmoid: times sigmoid of the smaller one's negative too), d the logits' distance, whose
// error is relative to the difference and not to the scores.  Softmax: z is off by 3e-7 and V + 5 half steps
// relative, an exponential by 2.4e-7 and a half step of its argument, the rest by six half steps.  `y`: the keys'
// magnitude; what 64 bits do not tell apart is not told apart here.  (1685 tokens of
// 98 fp16, softmax, with a bias: 10.1 -> 3.7 us; near keys went to 64 bits, at a few operations a clock.)
template <int V>
__device__ __forceinline__ bool surely_above(int scoring, float xi, float bi, float xj, float bj, float top, float z, float y) {
  const float hi = fmaxf(xi, xj), lo = fminf(xi, xj), e = -expm1f(lo - hi);
  const float s = scoring == kScoreSoftmax ? expf(hi - top) / z * e : sigmoid32(hi) * sigmoid32(-lo) * e;
  const float rel = scoring == kScoreSoftmax ? 1.2e-7f * (V + 30 + (top - hi)) : 2e-6f;
  const float bd = bi - bj, d = (xi >= xj ? s : -s) + bd;
  return d > rel * s + 1.2e-7f * fabsf(bd) + 1e-15f * y + 1e-37f;
}

// Softmax's sum in 64 bits, by the L lanes of a token (every lane of the warp takes part).
template <class T, int L>
__device__ __noinline__ double choose_sum64(const T *row, int E, float top) {
  double zd = 0.0;
#pragma unroll 4
  for (int e = static_cast<int>(threadIdx.x & (L - 1)); e < E; e += L)   // several at a time: an exponential is one long chain
    zd += exp(static_cast<double>(choose_float<T>(row[e])) - static_cast<double>(top));
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) zd += __shfl_xor_sync(0xffffffffu, zd, o);
  return zd;
}

// The key of this lane's group in 64 bits (every lane of the warp takes part): the sum of its two largest
// keys (or the one).  Only experts whose fp32 key reaches `least` of their group are computed.
template <class T, int L>
__device__ __noinline__ double choose_group64(const ChooseParams &p, const T *row, int base, int size, int lane, float top, float z,
                                              float least) {
  const double zd = p.scoring == kScoreSoftmax ? choose_sum64<T, L>(row, p.num_experts, top) : 0.0;
  double m1 = -INFINITY, m2 = -INFINITY;
  for (int i = lane; i < size; i += p.group_lanes) {
    const float x = choose_float<T>(row[base + i]), b = __ldg(p.bias + base + i);
    const float s = p.scoring == kScoreSoftmax ? expf(x - top) / z : sigmoid32(x);
    if (x > -INFINITY && s + b >= least) {
      const double k = score64(p.scoring, x, top, zd) + static_cast<double>(b);
      m2 = fmax(fmin(k, m1), m2);
      m1 = fmax(k, m1);
    }
  }
  for (int o = p.group_lanes / 2; o > 0; o >>= 1) {
    const double k1 = __shfl_xor_sync(0xffffffffu, m1, o), k2 = __shfl_xor_sync(0xffffffffu, m2, o);
    m2 = fmax(fmin(m1, k1), fmax(m2, k2));
    m1 = fmax(m1, k1);
  }
  return p.group_top == 2 && m2 > -static_cast<double>(INFINITY) ? m1 + m2 : m1;
}

// The choice of a token by 64-bit keys in shared memory, by its L lanes (every lane of the warp takes part):
// ids[j] for lane j < top_k.  Only the experts whose fp32 key reaches `least` are looked at; `kept`: bit g,
// group g is kept.
template <class T, int L>
__device__ __noinline__ int choose_exact(const ChooseParams &p, const T *row, float top, float z, float least, uint32_t kept,
                                         unsigned long long *keys) {
  const int sub = static_cast<int>(threadIdx.x & (L - 1)), E = p.num_experts;
  const double zd = p.scoring == kScoreSoftmax ? choose_sum64<T, L>(row, E, top) : 0.0;
#pragma unroll 4
  for (int e = sub; e < E; e += L) {
    const float x = choose_float<T>(row[e]), b = __ldg(p.bias + e);
    const float s = p.scoring == kScoreSoftmax ? expf(x - top) / z : sigmoid32(x);
    keys[e] = x > -INFINITY && s + b >= least && ((kept >> (e / p.group_size)) & 1u)
                  ? order_key(score64(p.scoring, x, top, zd) + static_cast<double>(b))
                  : 0ull;
  }
  __syncwarp();
  int id = -1;
  for (int j = 0; j < p.top_k; ++j) {
    unsigned long long m = 0ull;
    int at = E;
    for (int e = sub; e < E; e += L)
      if (keys[e] > m) {
        m = keys[e];
        at = e;
      }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
      const unsigned long long mo = __shfl_xor_sync(0xffffffffu, m, o);
      const int ao = __shfl_xor_sync(0xffffffffu, at, o);
      if (mo > m || (mo == m && ao < at)) {
        m = mo;
        at = ao;
      }
    }
    if (m != 0ull) {
      if (sub == j) id = at;
      if (sub == (at & (L - 1))) keys[at] = 0ull;
    }
    __syncwarp();
  }
  return id;
}

// Slots of a token's gathered keys (key, expert, logit, bias), and those of a CTA in shared memory.
template <int L, bool kScore>
constexpr int kChooseTokenSlots = kScore && L < 32 ? 2 * L : L;
template <class T, int L, bool kScore>
constexpr int kChooseSlots = !kScore && sizeof(T) == 2 ? 1 : 32 / L * kChooseTokenSlots<L, kScore> * kChooseWarps;

// One token per L lanes, 32 / L tokens a warp.  kScore: a bias, the keys are not the logits themselves.  A whole
// warp has the shortest way through a token, eight lanes leave fewer of them idle; with a bias up to 16 experts
// a lane, as a lane works through them one after the other (32768 tokens with a bias, 32 lanes and 8: of 64
// experts fp32 20.6 and 11.2 us, of 64 in 8 groups 26.6 and 14.8, of 128 bf16 24.3 and 16.2, of 256 fp32 in 8
// groups 43.2 and 59.6; of 256 bf16 in 8 groups without one 27.4 and 14.1).
template <class T, int L, int V, bool kVec, bool kScore>
__global__ void __launch_bounds__(32 * kChooseWarps, V <= 8 ? 8 : (L == 8 && V <= 16 ? 6 : (V <= 32 ? 4 : 1))) gmm_route_kernel(const __grid_constant__ ChooseParams p) {
  constexpr bool kPacked = !kScore && sizeof(T) == 2;
  constexpr bool kLong = V > 32;   // a lane's keys fill its registers (with biases and logits beside them its stack passed 2 KB)
  constexpr bool kKeep = kScore && L == 32 && !kLong;   // logits and biases stay in registers, else they are read again
  extern __shared__ unsigned long long choose_smem[];
  constexpr int kSlots = kChooseTokenSlots<L, kScore>;
  __shared__ uint4 choose_slots[kChooseSlots<T, L, kScore>];
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const int sub = lane & (L - 1), seg = lane & ~(L - 1);
  const uint32_t seg_mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << seg;
  const long long w = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + warp;   // fewer warps where they need much shared memory
  const long long t = w * (32 / L) + lane / L;
  if (w * (32 / L) >= p.num_tokens) return;   // the whole warp
  const bool live = t < p.num_tokens;
  const T *row = reinterpret_cast<const T *>(p.logits + (live ? t : 0) * p.logits_pitch);
  const bool softmax = p.scoring == kScoreSoftmax;

  // This lane's experts: of group `mine`.
  const bool grouped = p.groups > 1;
  const int mine = grouped ? sub / p.group_lanes : 0, part = grouped ? sub - mine * p.group_lanes : sub;
  const int base = mine * p.group_size, size = mine < p.groups ? p.group_size : 0;
  const ChoosePlace<kVec> at(base, size, part, grouped ? p.group_lanes : L, V);
  float x[kPacked ? 1 : V];
  uint32_t raw[kPacked ? V / 2 : 1], key[V];
  if constexpr (kPacked) choose_load16<T, V, kVec>(row, at, raw);
  else choose_load<T, V, kVec>(row, at, x);
  float bias[kScore && !kLong ? V : 1];   // beside the logits' loads, not behind them
  if constexpr (kScore && !kLong) {
    if (kVec && V % 4 == 0 && p.bias_vec) {
#pragma unroll
      for (int v = 0; v < V; v += 4) {
        const float4 b = at.there(0) ? __ldg(reinterpret_cast<const float4 *>(p.bias + at.first + v)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        bias[v] = b.x, bias[v + 1] = b.y, bias[v + 2] = b.z, bias[v + 3] = b.w;
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) bias[v] = at.there(v) ? __ldg(p.bias + at.expert(v)) : 0.0f;
    }
  }
  // NaN (and, for softmax, +infinity) anywhere: no expert at all.  Of packed keys the largest one tells.
  bool bad = false;
  if constexpr (kPacked) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      raw[i] = Packed16<T>::canonical(raw[i]);
      Packed16<T>::keys(raw[i], static_cast<uint32_t>(at.expert(2 * i)), static_cast<uint32_t>(at.expert(2 * i + 1)), key[2 * i],
                        key[2 * i + 1]);
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      bad |= softmax ? !(x[v] < INFINITY) : x[v] != x[v];
      if constexpr (!kScore) key[v] = order_key(x[v]);
    }
    bad = (__ballot_sync(0xffffffffu, bad) & seg_mask) != 0u;
  }

  // Softmax's maximum and sum, where a score itself is needed.
  float top = 0.0f, z = 1.0f;
  if (softmax && (kScore || !p.renormalise)) {
    auto logit = [&](int v) {
      if constexpr (kPacked) return Packed16<T>::value((raw[v / 2] >> (16 * (v & 1))) & 0xffffu);
      else return x[v];
    };
    float m = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) m = fmaxf(m, logit(v));
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    top = m > -INFINITY ? m : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) sum += kScore ? __expf(logit(v) - top) : expf(logit(v) - top);
    z = lanes_sum<L>(sum);
  }

  // How far apart two fp32 keys have to be, beside 2.4e-7 of the larger one (the bias added, twice half a
  // step), for their order to be sure.  sigmoid: each is off by sigmoid_key's error.  softmax: an
  // exponential at distance d below the largest is exp(-d) off by 2.4e-7 + 1.5e-7 d relative, 3e-7 at
  // most, the sum by as much and V + 5 half steps, the quotient by one step: 2 (9 + V + 5) half steps of 1 / z.
  float score_tol = 0.0f;
  if constexpr (kScore) {
    score_tol = softmax ? 1.2e-7f * (V + 20) / z : 6e-7f;
    auto bias_at = [&](int v) {
      if constexpr (kLong) return at.there(v) ? __ldg(p.bias + at.expert(v)) : 0.0f;
      else return bias[v];
    };
    if (softmax) {
      const float rz = 1.0f / z;
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = x[v] > -INFINITY ? order_key(__expf(x[v] - top) * rz + bias_at(v)) : 0u;
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = x[v] > -INFINITY ? order_key(sigmoid_key(x[v]) + bias_at(v)) : 0u;
    }
  }

  uint32_t kept_lanes = 0xffffffffu;   // lanes whose group is kept
  if (grouped) {
    float g1 = -INFINITY, g2 = -INFINITY;   // the group's two largest keys (without a bias: logits)
    if constexpr (kPacked) {
      uint32_t m1 = 0u, m2 = 0u;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        m2 = max(min(m1, key[v]), m2);
        m1 = max(m1, key[v]);
      }
      bad = (lanes_max<L>(m1) >> 16) > Packed16<T>::kPlusInf - (softmax ? 1u : 0u);   // before its group is left out
      if (m1 > Packed16<T>::kNone) g1 = Packed16<T>::key_value(m1);
      if (m2 > Packed16<T>::kNone) g2 = Packed16<T>::key_value(m2);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) merge_top2(g1, g2, key_value(key[v]), -INFINITY);
    }
    for (int o = p.group_lanes / 2; o > 0; o >>= 1)
      merge_top2(g1, g2, __shfl_xor_sync(0xffffffffu, g1, o), __shfl_xor_sync(0xffffffffu, g2, o));
    const bool pair = p.group_top == 2;
    float far = 0.0f, gv = g1;   // far: how far below the largest logit the group's is
    if (pair) {
      if constexpr (kScore) {   // a sum below fp32's lowest value is not that of a group without experts
        gv = g2 > -INFINITY ? fmaxf(g1 + g2, -3.402823466e38f) : g1;
      } else if (softmax) {   // scores relative to the largest logit's
        float m = g1;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        top = p.renormalise ? m : top;
        far = m - g1;
        gv = g1 > -INFINITY ? expf(g1 - m) + expf(g2 - m) : -INFINITY;
      } else {
        gv = g1 > -INFINITY ? sigmoid32(g1) + sigmoid32(g2) : -INFINITY;
      }
    }
    const uint32_t gk = mine < p.groups ? order_key(gv) : 0u;
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const uint32_t o = __shfl_sync(0xffffffffu, gk, seg + g * p.group_lanes);
      rank += o > gk || (o == gk && g < mine) ? 1 : 0;
    }
    bool keep = mine < p.groups && rank < p.top_groups;
    if (kScore || pair) {
      // Is one left out near enough to one kept that they might be the other way round?  `err`: how far a group's sum may
      // be off, with a bias as its terms are (they may cancel), else relative (3.6e-7 and half a step of the exponentials'
      // argument; sigmoids 4.8e-7; half a step more as it is added), and by two scores below 2^-126 (1.2e-38), which
      // fp32 may lose.
      float err;
      if constexpr (kScore) err = score_tol + 2.4e-7f * (fabsf(g1) + (pair && g2 > -INFINITY ? fabsf(g2) : 0.0f));
      else err = gv * (6e-7f + 6.5e-8f * far) + 2.5e-38f;
      const uint32_t high = lanes_max<L>(keep || gk == 0u ? 0u : order_key(gv + err));    // 0: none left out that has an expert
      const uint32_t low = ~lanes_max<L>(keep ? ~order_key(gv - err) : 0u);               // 0 for NaN: an infinite bias
      const bool near = high != 0u && high >= low && !bad;
      if (__any_sync(0xffffffffu, near)) {
        double gd;
        if constexpr (kScore) {
          const float g = pair ? g2 : g1;
          gd = choose_group64<T, L>(p, row, base, size, part, top, z,
                                 fabsf(g) < INFINITY ? g - 2.0f * (score_tol + 2.4e-7f * fabsf(g)) : -INFINITY);
        } else {
          gd = score64(p.scoring, g1, top, 1.0) + score64(p.scoring, g2, top, 1.0);
        }
        const unsigned long long k = mine < p.groups && g1 > -INFINITY ? order_key(gd) : 0ull;
        rank = 0;
        for (int g = 0; g < p.groups; ++g) {
          const unsigned long long o = __shfl_sync(0xffffffffu, k, seg + g * p.group_lanes);
          rank += o > k || (o == k && g < mine) ? 1 : 0;
        }
        if (near) keep = mine < p.groups && rank < p.top_groups;
      }
    }
    kept_lanes = __ballot_sync(0xffffffffu, keep);
    if (!keep)
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = 0u;
  }

  // An expert's logit and bias, once its key is made.
  auto logit_of = [&](int v) {
    if constexpr (kKeep) return x[v];
    else if constexpr (kScore) return choose_float<T>(row[at.expert(v)]);
    else return key_value(key[v]);
  };
  auto bias_of = [&](int v) {
    if constexpr (kKeep) return bias[v];
    else if constexpr (kScore) return __ldg(p.bias + at.expert(v));
    else return 0.0f;
  };

  // The chosen experts: lane j keeps the j-th one's number and logit.
  int id = -1;
  float xj = -INFINITY;
  bool done = false;
  if (p.top_k <= 8) {
    if constexpr (kPacked) {
      // Every lane gets the eight largest keys, sorted.
      uint32_t best[8];
      largest8<L, V>(key, best);
      const uint32_t mine_key = sub < p.top_k ? pick8(best, sub) : 0u;
      done = true;
      bad |= (best[0] >> 16) > Packed16<T>::kPlusInf - (softmax ? 1u : 0u);
      if (mine_key > Packed16<T>::kNone) {
        id = static_cast<int>(0xffffu - (mine_key & 0xffffu));
        xj = Packed16<T>::key_value(mine_key);
      }
    } else {
      // A key that top_k others reach: with a whole warp the top_k-th largest of the lanes' largest (about
      // nine keys reach the eighth), else the top_k-th largest itself, from sorted lists.
      uint32_t least;
      if constexpr (L == 32) {
        uint32_t m = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = max(m, key[v]);
#pragma unroll
        for (int k = 2; k <= 32; k <<= 1)   // a bitonic sort across the lanes, descending
#pragma unroll
          for (int j = k >> 1; j > 0; j >>= 1) {
            const uint32_t o = __shfl_xor_sync(0xffffffffu, m, j);
            m = ((lane & j) == 0) == ((lane & k) == 0) ? max(m, o) : min(m, o);
          }
        least = __shfl_sync(0xffffffffu, m, p.top_k - 1);
      } else {
        uint32_t best[8];
        largest8<L, V>(key, best);
        least = pick8(best, p.top_k - 1);
      }
      if constexpr (kScore) {   // and those that are so near that they might belong to them
        const float l = key_value(least);
        if (least != 0u && l < INFINITY) least = order_key(l - 2.0f * (score_tol + 2.4e-7f * fabsf(l)));
      }
      least = max(least, 1u);
      // They are gathered, a lane each (or two), and ranked against one another.
      uint4 *slots = choose_slots + (warp * 32 + seg) * (kSlots / L);
      int count = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const bool hit = key[v] >= least;
        const uint32_t hits = __ballot_sync(0xffffffffu, hit) & seg_mask;
        if (hit) {
          const int to = count + __popc(hits & ((1u << lane) - 1u));
          if (to < kSlots)
            slots[to] = make_uint4(key[v], static_cast<uint32_t>(at.expert(v)),
                                   kScore && !kKeep ? 0u : __float_as_uint(logit_of(v)), kKeep ? __float_as_uint(bias_of(v)) : 0u);
        }
        count += __popc(hits);
      }
      __syncwarp();
      const int most = L == 32 ? count : static_cast<int>(redux_max(static_cast<uint32_t>(count)));
      done = most <= kSlots;
      if (most <= L) {
        const bool have = sub < count;
        uint4 f = have ? slots[sub] : make_uint4(0u, 0xffffffffu, 0u, 0u);
        if (kScore && !kKeep && have) {
          f.z = __float_as_uint(choose_float<T>(row[f.y]));
          f.w = __float_as_uint(__ldg(p.bias + f.y));
        }
        int rank = 0;
        for (int i = 0; i < most; ++i) {
          const uint32_t ko = __shfl_sync(0xffffffffu, f.x, seg + i), eo = __shfl_sync(0xffffffffu, f.y, seg + i);
          rank += ko > f.x || (ko == f.x && eo < f.y) ? 1 : 0;
        }
        __syncwarp();   // the slots are read
        if (have) slots[rank] = f;
        __syncwarp();
        if (have) f = slots[sub];   // in descending order now
        if constexpr (kScore) {
          // A key as near to its neighbour that their order is not sure, of another logit or bias?  (Behind
          // the last one too: equal ones may stand between it and one that belongs before them.)
          const float v = key_value(f.x), vo = key_value(__shfl_down_sync(0xffffffffu, f.x, 1));
          const uint32_t xo = __shfl_down_sync(0xffffffffu, f.z, 1), bo = __shfl_down_sync(0xffffffffu, f.w, 1);
          const bool near = sub + 1 < count && !(v - vo > score_tol + 2.4e-7f * fmaxf(fabsf(v), fabsf(vo))) &&
                            !(__uint_as_float(xo) == __uint_as_float(f.z) && __uint_as_float(bo) == __uint_as_float(f.w)) &&
                            !surely_above<V>(p.scoring, __uint_as_float(f.z), __uint_as_float(f.w), __uint_as_float(xo),
                                             __uint_as_float(bo), top, z, fabsf(v));
          if (__any_sync(0xffffffffu, near && !bad)) {
            const double zd = softmax ? choose_sum64<T, L>(row, p.num_experts, top) : 0.0;
            const unsigned long long k =
                have ? order_key(score64(p.scoring, __uint_as_float(f.z), top, zd) + static_cast<double>(__uint_as_float(f.w))) : 0ull;
            rank = 0;
            for (int i = 0; i < most; ++i) {
              const unsigned long long o = __shfl_sync(0xffffffffu, k, seg + i);
              const uint32_t eo = __shfl_sync(0xffffffffu, f.y, seg + i);
              rank += o > k || (o == k && eo < f.y) ? 1 : 0;
            }
            __syncwarp();
            if (have) slots[rank] = f;
            __syncwarp();
            if (have) f = slots[sub];
          }
        }
        if (have && sub < p.top_k) {
          id = static_cast<int>(f.y);
          xj = __uint_as_float(f.z);
        }
      } else if constexpr (kSlots > L) {
        if (done) {   // two keys a lane, as above
          uint4 f[2];
          unsigned long long k[2];
          int rank[2];
          auto have = [&](int h) { return sub + h * L < count; };
          auto sort = [&]() {   // by (k, expert)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              rank[h] = 0;
              for (int i = 0; i < most; ++i) {
                const unsigned long long ko = __shfl_sync(0xffffffffu, i < L ? k[0] : k[1], seg + (i & (L - 1)));
                const uint32_t eo = __shfl_sync(0xffffffffu, i < L ? f[0].y : f[1].y, seg + (i & (L - 1)));
                rank[h] += ko > k[h] || (ko == k[h] && eo < f[h].y) ? 1 : 0;
              }
            }
            __syncwarp();   // the slots are read
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (have(h)) slots[rank[h]] = f[h];
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (have(h)) f[h] = slots[sub + h * L];
          };
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f[h] = have(h) ? slots[sub + h * L] : make_uint4(0u, 0xffffffffu, 0u, 0u);
            if (have(h)) {
              f[h].z = __float_as_uint(choose_float<T>(row[f[h].y]));
              f[h].w = __float_as_uint(__ldg(p.bias + f[h].y));
            }
            k[h] = f[h].x;
          }
          sort();
          bool near = false;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (sub + h * L + 1 < count) {
              const uint4 o = slots[sub + h * L + 1];
              const float v = key_value(f[h].x), vo = key_value(o.x);
              near |= !(v - vo > score_tol + 2.4e-7f * fmaxf(fabsf(v), fabsf(vo))) &&
                      !(__uint_as_float(o.z) == __uint_as_float(f[h].z) && __uint_as_float(o.w) == __uint_as_float(f[h].w)) &&
                      !surely_above<V>(p.scoring, __uint_as_float(f[h].z), __uint_as_float(f[h].w), __uint_as_float(o.z),
                                       __uint_as_float(o.w), top, z, fabsf(v));
            }
          if (__any_sync(0xffffffffu, near && !bad)) {
            const double zd = softmax ? choose_sum64<T, L>(row, p.num_experts, top) : 0.0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              k[h] = have(h) ? order_key(score64(p.scoring, __uint_as_float(f[h].z), top, zd) + static_cast<double>(__uint_as_float(f[h].w)))
                             : 0ull;
            sort();
          }
          if (have(0) && sub < p.top_k) {
            id = static_cast<int>(f[0].y);
            xj = __uint_as_float(f[0].z);
          }
        }
      }
    }
  }
  if (!done) {
    // One maximum after the other.
    bool unsure = false;
    float kth = 0.0f, prev_key = 0.0f, prev_x = 0.0f, prev_b = 0.0f;
    auto take = [&](int &e) -> uint32_t {   // the largest key left, and its lowest expert
      uint32_t m = key[0];
#pragma unroll
      for (int v = 1; v < V; ++v) m = max(m, key[v]);
      const uint32_t M = lanes_max<L>(m);
      if constexpr (kPacked) {
        e = static_cast<int>(0xffffu - (M & 0xffffu));
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = key[v] == M ? 0u : key[v];
      } else {
        uint32_t lowest = 0u;   // its complement
#pragma unroll
        for (int v = 0; v < V; ++v) lowest = max(lowest, key[v] == M ? ~static_cast<uint32_t>(at.expert(v)) : 0u);
        e = static_cast<int>(~lanes_max<L>(lowest));
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = key[v] == M && at.expert(v) == e ? 0u : key[v];
      }
      return M;
    };
    if constexpr (kPacked)
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = key[v] > Packed16<T>::kNone ? key[v] : 0u;
    int taken = 0;
    for (; taken < p.top_k; ++taken) {
      int e;
      const uint32_t M = take(e);
      if (kPacked && taken == 0) bad |= (M >> 16) > Packed16<T>::kPlusInf - (softmax ? 1u : 0u);
      if (sub == taken && M != 0u) id = e;
      if (__all_sync(0xffffffffu, M == 0u)) break;
      if (kScore && M != 0u) {
        const float k = key_value(M), xe = choose_float<T>(row[e]), be = __ldg(p.bias + e);
        if (taken > 0 && !(prev_key - k > score_tol + 2.4e-7f * fabsf(prev_key)) && !(prev_x == xe && prev_b == be)) unsure = true;
        prev_key = k;
        prev_x = xe;
        prev_b = be;
        kth = k;
      }
    }
    if constexpr (kScore) {
      const bool full = (__ballot_sync(0xffffffffu, sub == p.top_k - 1 && id >= 0) & seg_mask) != 0u;   // every slot is filled
      const float tol = score_tol + 2.4e-7f * fabsf(kth);
      bool near = false;   // is one of those left as near to the last one?
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (full && key[v] != 0u && !(kth - key_value(key[v]) > tol)) near |= !(logit_of(v) == prev_x && bias_of(v) == prev_b);
      const uint32_t nears = __ballot_sync(0xffffffffu, near) & seg_mask;   // by every lane, sure or not
      unsure = (unsure || nears != 0u) && !bad;
      if (__any_sync(0xffffffffu, unsure)) {
        uint32_t kept = 0u;
        for (int g = 0; g < p.groups; ++g) kept |= (kept_lanes >> (seg + g * p.group_lanes) & 1u) << g;
        const int exact = choose_exact<T, L>(p, row, top, z, full && kth < INFINITY ? kth - 2.0f * tol : -INFINITY, kept,
                                             choose_smem + static_cast<size_t>(warp * (32 / L) + lane / L) * p.num_experts);
        if (unsure) id = exact;
      }
    }
    if (id >= 0) xj = choose_float<T>(row[id]);
  }
  if (bad) {
    id = -1;
    if (live && sub == 0) atomicOr(p.status, kStatusBadLogit);
  }

  // Weights.
  if (id < 0) xj = -INFINITY;
  float wj;
  if (p.renormalise) {
    float m = xj;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    wj = id < 0 ? 0.0f : relative_score(softmax, xj, m);
    const float sum = lanes_sum<L>(wj);
    if (id >= 0) wj = wj / sum;
  } else {
    wj = id < 0 ? 0.0f : (softmax ? expf(xj - top) / z : sigmoid32(xj));
  }
  if (live && sub < p.top_k) {
    const long long s = t * p.top_k + sub;
    p.ids[s] = id;
    p.weights[s] = id < 0 ? 0.0f : wj * p.scale;
  }
}

// The gradient (16384 tokens of 64 bf16 logits, all of them in it, 4.2 us; 5003 of 161 fp32 4.2 us: latency of
// one pass).  L lanes a token; a token's row of d_logits is put together in shared memory (zeros,
// then the chosen experts') and written V consecutive experts a lane; kDense (softmax, not
// renormalised): every logit is read, and every expert's value is its score times a difference.
template <class T, int L, int V, bool kVec, bool kDense>
__global__ void __launch_bounds__(32 * kChooseWarps) gmm_route_grad_kernel(const __grid_constant__ ChooseParams p) {
  extern __shared__ __align__(16) float choose_row[];
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const int sub = lane & (L - 1), seg = lane & ~(L - 1);
  const long long w = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + warp;   // fewer warps where they need much shared memory
  const long long t = w * (32 / L) + lane / L;
  if (w * (32 / L) >= p.num_tokens) return;
  const bool live = t < p.num_tokens;
  const T *row = reinterpret_cast<const T *>(p.logits + (live ? t : 0) * p.logits_pitch);
  float *buf = choose_row + (static_cast<size_t>(warp) * (32 / L) + lane / L) * (L * V);
  const ChoosePlace<kVec> at(0, p.num_experts, sub, L, V);

  int id = -1;
  float g = 0.0f, xj = -INFINITY;
  if (live && sub < p.top_k) {
    id = __ldg(p.ids + t * p.top_k + sub);
    if (id >= p.num_experts) {
      atomicOr(p.status, kStatusBadExpert);
      id = -1;
    }
    if (id >= 0) {
      g = __ldg(p.weights + t * p.top_k + sub) * p.scale;
      xj = choose_float<T>(row[id]);
      if (xj == -INFINITY) id = -1;   // a score of zero: no gradient, and none through the others' sum
    }
  }
  float x[V];
  float top = 0.0f, z = 1.0f;
  bool bad = id >= 0 && (!(xj < INFINITY) && (p.scoring == kScoreSoftmax || xj != xj));
  if constexpr (kDense) {
    choose_load<T, V, kVec>(row, at, x);
    float m = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      bad |= !(x[v] < INFINITY);
      m = fmaxf(m, x[v]);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    top = m > -INFINITY ? m : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = expf(x[v] - top);
      sum += x[v];
    }
    z = lanes_sum<L>(sum);
  }
  const uint32_t bads = __ballot_sync(0xffffffffu, bad);
  bad = ((L == 32 ? bads : (bads >> seg) & ((1u << (L & 31)) - 1u))) != 0u;
  if (bad) {   // such a token has no experts: no gradient
    id = -1;
    if (live && sub == 0) atomicOr(p.status, kStatusBadLogit);
  }
  float dj = 0.0f, common = 0.0f;
  if constexpr (kDense) {
    dj = id >= 0 ? g : 0.0f;
    common = lanes_sum<L>(id >= 0 ? g * (expf(xj - top) / z) : 0.0f);
  } else if (p.renormalise) {
    float m = id >= 0 ? xj : -INFINITY;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float s = id >= 0 ? relative_score(p.scoring == kScoreSoftmax, xj, m) : 0.0f;
    const float sum = lanes_sum<L>(s);
    const float u = id >= 0 ? s / sum : 0.0f;
    const float mean = lanes_sum<L>(id >= 0 ? u * g : 0.0f);
    dj = id >= 0 ? u * (g - mean) : 0.0f;
    if (p.scoring == kScoreSigmoid) dj *= sigmoid32(-xj);
  } else if (id >= 0) {
    dj = g * sigmoid32(xj) * sigmoid32(-xj);
  }
  if (id < 0) dj = 0.0f;

#pragma unroll
  for (int v = 0; v < V; ++v) buf[sub + v * L] = 0.0f;
  __syncwarp();
  // A lane whose expert an earlier slot names too adds after it, in the slots' order.
  for (int j = 0; j < p.top_k; ++j) {
    if (sub == j && id >= 0) buf[id] += dj;
    __syncwarp();
  }
  if (!live) return;
  T *out = reinterpret_cast<T *>(p.d_logits + t * p.d_pitch);
  alignas(16) T y[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float d = buf[kVec ? at.first + v : sub + v * L];
    if constexpr (kDense) d = bad || z == 0.0f ? 0.0f : x[v] / z * (d - common);   // z = 0: every logit is masked
    y[v] = route_from_float<T>(d);
  }
  constexpr int kBytes = V * static_cast<int>(sizeof(T));
  if constexpr (kVec) {
    if (!at.there(0)) return;
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4 *>(out + at.first)[i] = reinterpret_cast<const uint4 *>(y)[i];
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2 *>(out + at.first) = *reinterpret_cast<const uint2 *>(y);
    } else {
      *reinterpret_cast<uint32_t *>(out + at.first) = *reinterpret_cast<const uint32_t *>(y);
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (at.there(v)) out[at.expert(v)] = y[v];
  }
}

}  // namespace gmm
