// Tokens sorted by expert and back, for sm_103a.
//
// A router gives every token t its top_k experts: slot s = t * top_k + j holds expert
// id e_s.  With E experts and S = tokens * top_k slots:
//   dispatch      a stable counting sort of the slots by expert:
//                   a_offsets[e] = #{ s : 0 <= e_s < e },  a_offsets[E] = the rows in use,
//                   row(s) = a_offsets[e_s] + #{ s' < s : e_s' = e_s },
//                 slot_rows[s] = row(s) (-1 for a dropped slot), row_slots its inverse (-1
//                 past the rows in use), and rows[row(s), :] = tokens[s / top_k, :].
//   combine       out[t, :] = sum_j w[t, j] * rows[slot_rows[t, j], :]
//                 (w = 1: the gradient of dispatch's copy).
//   combine_grad  d_rows[slot_rows[t, j], :] = w[t, j] * d_out[t, :],
//                 d_w[t, j] = < d_out[t, :], rows[slot_rows[t, j], :] >;
//                 the caller's named rows are distinct (dispatch's are), so each has one writer.
// Every sum has a fixed order (j ascending; a dot product per lane, then a fixed tree),
// no result depends on the order of atomics.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

#include "gmm_common.cuh"

namespace gmm {

constexpr int kRouteThreads = 512;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteMaxWidth = 0x7fffffff - 4095;   // columns are counted in 32 bits, by steps of up to 2048 past the last one
constexpr int kRouteSmallSlots = 4096;     // up to here (and kRouteSmallExperts) one launch sorts and copies
constexpr int kRouteSmallExperts = 1024;
constexpr int kRouteMaxCounts = 32768;     // chunk counts (chunks x experts) in the workspace
constexpr int kRouteMaxChunks = 152;
constexpr long long kRoutePrefetch = 64 * 1024;   // bytes of its tokens that a CTA prefetches while the count runs
constexpr int kRouteBatch = 64;            // tokens whose rows a CTA holds in shared memory at a time

struct DispatchParams {
  const int32_t *slot_experts;   // [tokens, top_k]
  uint32_t *a_offsets;           // [E + 1]
  int32_t *slot_rows;            // [tokens, top_k]
  int32_t *row_slots;            // [tokens * top_k]
  const uint8_t *tokens;         // [tokens, width] with a row pitch, or null (no copy)
  uint8_t *rows;                 // [tokens * top_k, width] contiguous
  long long token_pitch;         // bytes
  long long row_bytes;
  int num_tokens;
  int top_k;
  int num_experts;
  int chunks;                    // two-launch form: chunks of chunk_tokens tokens
  int chunk_tokens;
  int subs;                      // two-launch form: CTAs of the copy per chunk
  uint32_t *counts;              // workspace [chunks, E]
  uint32_t *status;
};

// Stable ranks of the slots [begin, end) (one warp's contiguous share) among the slots of
// the same expert in that share; cnt[e] ends as the share's count of expert e.  Thirty-two
// slots a step: lanes with the same expert find one another by a ballot on every bit of the
// expert's number (a warp match takes a turn for every different one: 256 tokens, top-8 of 64
// experts, 0.8 us more than the 5.8 in all), the lowest of them advances the count.  `emit(s, e, rank)`
// is called for every slot (rank -1 when its expert id is out of range).
template <class Emit>
__device__ __forceinline__ uint32_t route_rank_share(const int32_t *ids, int begin, int end, int E, uint32_t *cnt,
                                                     Emit emit) {
  const uint32_t lane = threadIdx.x & 31u;
  uint32_t flags = 0;
  const int bits = 32 - __clz(E - 1);
  int e_next = begin + static_cast<int>(lane) < end ? __ldg(ids + begin + lane) : -1;   // one step ahead
  for (int s0 = begin; s0 < end; s0 += 32) {
    const int s = s0 + static_cast<int>(lane);
    const int e = e_next;
    e_next = s + 32 < end ? __ldg(ids + s + 32) : -1;
    const bool ok = e >= 0 && e < E;
    if (e >= E) flags = kStatusBadExpert;
    uint32_t peers = __ballot_sync(0xffffffffu, ok);
    for (int b = 0; b < bits; ++b) {
      const uint32_t set = __ballot_sync(0xffffffffu, (e >> b) & 1);
      peers &= ((e >> b) & 1) ? set : ~set;
    }
    const uint32_t below = __popc(peers & ((1u << lane) - 1u));
    uint32_t first = 0;
    if (ok) first = cnt[e];
    __syncwarp();
    if (ok && below == 0) cnt[e] = first + __popc(peers);
    __syncwarp();
    if (s < end) emit(s, e, ok ? static_cast<int>(first + below) : -1);
  }
  return flags;
}

// Exclusive scan of v[0 .. n) in shared memory by the whole CTA; v[n] receives the total.
// `warp_sums` holds kRouteWarps words.
__device__ __forceinline__ void route_scan(uint32_t *v, int n, uint32_t *warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + kRouteThreads - 1) / kRouteThreads;
  const int b = min(n, tid * per), e = min(n, b + per);
  uint32_t mine = 0;
  for (int i = b; i < e; ++i) mine += v[i];
  uint32_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  uint32_t run = incl - mine;
  for (int w = 0; w < warp; ++w) run += warp_sums[w];
  for (int i = b; i < e; ++i) {
    const uint32_t x = v[i];
    v[i] = run;
    run += x;
  }
  if (tid == kRouteThreads - 1) v[n] = run;
  __syncthreads();
}

// Vectors a lane and copy unit: 2 KB of a token with 16-byte vectors; with narrow ones more of
// them, to keep as many bytes in flight.  Few bytes (kFew) are spread over many SMs instead:
// 512 bytes a unit.
template <int VB, bool kFew>
constexpr int kRouteUnit = VB == 16 ? (kFew ? 1 : 4) : (kFew ? 4 : 16);

template <int VB>
struct RouteVec;
template <>
struct RouteVec<16> { using type = uint4; };
template <>
struct RouteVec<4> { using type = uint32_t; };
template <>
struct RouteVec<2> { using type = unsigned short; };

// Copies of tokens [t0, t0 + n) to their rows; rows_s[i * top_k + j] is the row of slot j
// of token t0 + i (-1: dropped).  A unit is up to kU vectors a lane of one token: read once,
// written to each of its rows.  Units go to the CTA's warps in turn, `part` of `parts` CTAs.
template <int VB, int kU>
__device__ __forceinline__ void route_copy(const DispatchParams &p, const int *rows_s, int t0, int n, int part,
                                           int parts) {
  using V = typename RouteVec<VB>::type;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nvec = static_cast<int>(p.row_bytes / VB);
  const int pieces = (nvec + 32 * kU - 1) / (32 * kU);
  const int units = n * pieces;
  for (int u = part * kRouteWarps + warp; u < units; u += parts * kRouteWarps) {
    const int i = u / pieces, v0 = (u - i * pieces) * 32 * kU + lane;
    const V *src = reinterpret_cast<const V *>(p.tokens + (t0 + i) * p.token_pitch);
    V x[kU];
#pragma unroll
    for (int q = 0; q < kU; ++q)
      if (v0 + 32 * q < nvec) x[q] = __ldg(src + v0 + 32 * q);
    for (int j = 0; j < p.top_k; ++j) {
      const int r = rows_s[i * p.top_k + j];
      if (r < 0) continue;
      V *dst = reinterpret_cast<V *>(p.rows + r * p.row_bytes);
#pragma unroll
      for (int q = 0; q < kU; ++q)
        if (v0 + 32 * q < nvec) dst[v0 + 32 * q] = x[q];
    }
  }
}

// One launch for few slots: every CTA sorts all of them (a read of at most 16 KB that sits
// in L2, about a microsecond) and copies its share, which saves the second launch that a
// count before the copy would need.  CTA 0 writes the maps.  Bound by its latency: 256
// tokens of 2048 bf16 to 8 of 64 experts take 5.8 us (3 more with 2 KB copy units, which only
// 32 CTAs shared).
template <int VB, bool kFew>
__global__ void __launch_bounds__(kRouteThreads) gmm_dispatch_small_kernel(const __grid_constant__ DispatchParams p) {
  extern __shared__ uint32_t route_smem[];
  __shared__ uint32_t warp_sums[kRouteWarps];
  const int tid = threadIdx.x, warp = tid >> 5;
  const int E = p.num_experts, S = p.num_tokens * p.top_k;
  uint32_t *cnt = route_smem;                                       // [kRouteWarps][E]
  uint32_t *off = cnt + kRouteWarps * E;                            // [E + 1]
  int *row_s = reinterpret_cast<int *>(off + E + 1);                // [S]
  for (int i = tid; i < kRouteWarps * E; i += kRouteThreads) cnt[i] = 0;
  __syncthreads();
  const int share = ((S + kRouteWarps - 1) / kRouteWarps + 31) & ~31;
  const int begin = min(S, warp * share), end = min(S, begin + share);
  const uint32_t flags = route_rank_share(p.slot_experts, begin, end, E, cnt + warp * E,
                                          [&](int s, int, int rank) { row_s[s] = rank; });
  __syncthreads();
  for (int e = tid; e < E; e += kRouteThreads) {
    uint32_t run = 0;
#pragma unroll
    for (int w = 0; w < kRouteWarps; ++w) {
      const uint32_t c = cnt[w * E + e];
      cnt[w * E + e] = run;
      run += c;
    }
    off[e] = run;
  }
  __syncthreads();
  route_scan(off, E, warp_sums);
  for (int s = begin + (tid & 31); s < end; s += 32) {
    const int rank = row_s[s];
    int row = -1;
    if (rank >= 0) {
      const int e = __ldg(p.slot_experts + s);
      row = static_cast<int>(off[e] + cnt[warp * E + e]) + rank;
    }
    row_s[s] = row;
    if (blockIdx.x == 0) {
      p.slot_rows[s] = row;
      if (row >= 0) p.row_slots[row] = s;
    }
  }
  if (blockIdx.x == 0) {
    for (int e = tid; e <= E; e += kRouteThreads) p.a_offsets[e] = off[e];
    for (int r = static_cast<int>(off[E]) + tid; r < S; r += kRouteThreads) p.row_slots[r] = -1;
    if (flags) atomicOr(p.status, flags);
  }
  if (p.tokens == nullptr) return;
  __syncthreads();
  route_copy<VB, kRouteUnit<VB, kFew>>(p, row_s, 0, p.num_tokens, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
}

// Many slots, first launch: CTA c counts the experts of its chunk of tokens and leaves every
// slot's rank among the chunk's slots of the same expert in slot_rows.
__global__ void __launch_bounds__(kRouteThreads) gmm_dispatch_count_kernel(const __grid_constant__ DispatchParams p,
                                                                           int warps) {
  extern __shared__ uint32_t route_smem[];
  grid_launch_dependents();   // the copy's CTAs start, and wait where they need these results
  const int tid = threadIdx.x, warp = tid >> 5;
  const int E = p.num_experts;
  const long long t0 = static_cast<long long>(blockIdx.x) * p.chunk_tokens;
  const int first = static_cast<int>(min(t0, static_cast<long long>(p.num_tokens))) * p.top_k;
  const int last = static_cast<int>(min(t0 + p.chunk_tokens, static_cast<long long>(p.num_tokens))) * p.top_k;
  uint32_t *cnt = route_smem;   // [warps][E]
  for (int i = tid; i < warps * E; i += kRouteThreads) cnt[i] = 0;
  __syncthreads();
  const int share = ((last - first + warps - 1) / warps + 31) & ~31;
  const int begin = min(last, first + warp * share), end = warp < warps ? min(last, begin + share) : begin;
  if (warp < warps) {
    const uint32_t flags = route_rank_share(p.slot_experts, begin, end, E, cnt + warp * E,
                                            [&](int s, int, int rank) { p.slot_rows[s] = rank; });
    if (flags) atomicOr(p.status, flags);
  }
  __syncthreads();
  for (int e = tid; e < E; e += kRouteThreads) {
    uint32_t run = 0;
    for (int w = 0; w < warps; ++w) {
      const uint32_t c = cnt[w * E + e];
      cnt[w * E + e] = run;
      run += c;
    }
    p.counts[static_cast<size_t>(blockIdx.x) * E + e] = run;
  }
  __syncthreads();
  for (int s = begin + (tid & 31); s < end; s += 32) {   // the same thread wrote slot_rows[s] above
    const int e = __ldg(p.slot_experts + s);
    if (e >= 0 && e < E) p.slot_rows[s] += static_cast<int>(cnt[warp * E + e]);
  }
}

// Second launch, started while the first one runs: a CTA sums the chunk counts (at most 128 KB, from L2) into the first row of
// every expert's slots in its chunk, then places and copies its tokens, kRouteBatch at a time.
// Bound by the copy's bytes: 16384 tokens of 8 KB to two rows each take 69 us with the
// count, 5.8 TB/s.
template <int VB>
__global__ void __launch_bounds__(kRouteThreads) gmm_dispatch_place_kernel(const __grid_constant__ DispatchParams p) {
  extern __shared__ uint32_t route_smem[];
  __shared__ uint32_t warp_sums[kRouteWarps];
  const int tid = threadIdx.x;
  const int E = p.num_experts, S = p.num_tokens * p.top_k;
  uint32_t *off = route_smem;                                // [E + 1]: totals, then their exclusive scan
  uint32_t *bef = off + E + 1;                               // [E]: counts of the chunks before this one
  int *row_s = reinterpret_cast<int *>(bef + E);             // [kRouteBatch * top_k]
  const int chunk = static_cast<int>(blockIdx.x) / p.subs, sub = static_cast<int>(blockIdx.x) % p.subs;
  const long long c0 = static_cast<long long>(chunk) * p.chunk_tokens;
  const int per = (p.chunk_tokens + p.subs - 1) / p.subs;
  const int lim = static_cast<int>(min(c0 + p.chunk_tokens, static_cast<long long>(p.num_tokens)));
  const int t_begin = static_cast<int>(min(c0 + static_cast<long long>(sub) * per, static_cast<long long>(lim)));
  const int t_end = min(lim, t_begin + per);
  // Ahead of the count's results: the first of this CTA's tokens into L2.
  if (p.tokens != nullptr && t_begin < t_end) {
    const long long bytes = min((t_end - t_begin - 1) * p.token_pitch + p.row_bytes, kRoutePrefetch);
    const uint8_t *at = p.tokens + t_begin * p.token_pitch;
    for (long long i = tid * 128ll; i < bytes; i += kRouteThreads * 128ll) prefetch_l2(at + i);
  }
  for (int e = tid; e < E; e += kRouteThreads) {
    off[e] = 0;
    bef[e] = 0;
  }
  __syncthreads();
  grid_wait_dependency();
  // Threads in groups of E (one expert a thread) take the chunks in turn.
  const int groups = max(1, kRouteThreads / E);
  const int g = E <= kRouteThreads ? tid / E : 0;
  if (g < groups) {
    for (int e = E <= kRouteThreads ? tid - g * E : tid; e < E; e += kRouteThreads) {
      uint32_t total = 0, before = 0;
#pragma unroll 4
      for (int c = g; c < p.chunks; c += groups) {
        const uint32_t n = p.counts[static_cast<size_t>(c) * E + e];
        total += n;
        before += c < chunk ? n : 0u;
      }
      atomicAdd(&off[e], total);
      atomicAdd(&bef[e], before);
    }
  }
  __syncthreads();
  route_scan(off, E, warp_sums);
  if (blockIdx.x == 0)
    for (int e = tid; e <= E; e += kRouteThreads) p.a_offsets[e] = off[e];
  for (int r = static_cast<int>(off[E]) + static_cast<int>(blockIdx.x) * kRouteThreads + tid; r < S;
       r += static_cast<int>(gridDim.x) * kRouteThreads)
    p.row_slots[r] = -1;
  for (int t = t_begin; t < t_end; t += kRouteBatch) {
    const int n = min(kRouteBatch, t_end - t);
    __syncthreads();   // the previous batch's copies have read row_s
    for (int i = tid; i < n * p.top_k; i += kRouteThreads) {
      const int s = t * p.top_k + i;
      const int e = __ldg(p.slot_experts + s);
      int row = -1;
      if (e >= 0 && e < E) {
        row = static_cast<int>(off[e] + bef[e]) + p.slot_rows[s];
        p.row_slots[row] = s;
        p.slot_rows[s] = row;
      }
      row_s[i] = row;
    }
    __syncthreads();
    if (p.tokens != nullptr) route_copy<VB, kRouteUnit<VB, false>>(p, row_s, t, n, 0, 1);
  }
}

// ---------------------------------------------------------------- combine and its gradient

struct CombineParams {
  uint8_t *out;                // combine: [tokens, width], row pitch out_pitch
  const uint8_t *rows;         // [num_rows, width] contiguous
  const int32_t *slot_rows;    // [tokens, top_k]
  const float *weights;        // [tokens, top_k] or null (ones)
  const uint8_t *d_out;        // gradient: [tokens, width], row pitch out_pitch
  uint8_t *d_rows;             // gradient: [num_rows, width]
  float *d_weights;            // gradient: [tokens, top_k] or null
  long long out_pitch;         // bytes
  long long row_bytes;
  int num_tokens;
  int top_k;
  int num_rows;
  int warps_per_token;         // gradient
  uint32_t *status;
};

// VN consecutive elements of type T as loaded: 16 bytes, or one element.
template <class T, int VN>
struct RoutePack {
  static constexpr int kWords = sizeof(T) * VN / 4;
  uint32_t w[kWords];
};
template <class T>
struct RoutePack<T, 1> {
  T x;
};

template <class T, int VN>
__device__ __forceinline__ RoutePack<T, VN> route_load(const uint8_t *row, int i) {
  RoutePack<T, VN> r;
  if constexpr (VN > 1) {
    const uint4 x = __ldg(reinterpret_cast<const uint4 *>(row) + i);
    r.w[0] = x.x;
    r.w[1] = x.y;
    r.w[2] = x.z;
    r.w[3] = x.w;
  } else {
    r.x = reinterpret_cast<const T *>(row)[i];
  }
  return r;
}

// The pack's values in fp32.
template <class T, int VN>
__device__ __forceinline__ void route_unpack(const RoutePack<T, VN> &p, float (&v)[VN]) {
  if constexpr (VN == 1) {
    if constexpr (std::is_same_v<T, float>) v[0] = p.x;
    else if constexpr (std::is_same_v<T, __half>) v[0] = __half2float(p.x);
    else v[0] = __bfloat162float(p.x);
  } else if constexpr (std::is_same_v<T, float>) {
#pragma unroll
    for (int i = 0; i < VN; ++i) v[i] = __uint_as_float(p.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VN / 2; ++i) {
      if constexpr (std::is_same_v<T, __half>) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&p.w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      } else {
        v[2 * i] = __uint_as_float(p.w[i] << 16);
        v[2 * i + 1] = __uint_as_float(p.w[i] & 0xffff0000u);
      }
    }
  }
}

// VN fp32 values rounded to T and stored.
template <class T, int VN>
__device__ __forceinline__ void route_store(uint8_t *row, int i, const float (&v)[VN]) {
  if constexpr (VN == 1) {
    reinterpret_cast<T *>(row)[i] = route_from_float<T>(v[0]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (std::is_same_v<T, float>) {
        w[j] = __float_as_uint(v[j]);
      } else if constexpr (std::is_same_v<T, __half>) {
        const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t *>(&h);
      } else {
        w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
      }
    }
    reinterpret_cast<uint4 *>(row)[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// acc += a * x, paired where there are pairs (each value rounded as by fmaf).
template <int VN>
__device__ __forceinline__ void route_fma(float (&acc)[VN], float a, const float (&x)[VN]) {
  if constexpr (VN == 1) {
    acc[0] = fmaf(a, x[0], acc[0]);
  } else {
#pragma unroll
    for (int i = 0; i < VN; i += 2) fma_f32x2(acc[i], acc[i + 1], a, x[i], x[i + 1]);
  }
}

// This lane's slot of token t: its row (-1: none) and weight.
__device__ __forceinline__ int route_slot(const CombineParams &p, int t, int lane, float *w) {
  int r = -1;
  *w = 0.0f;
  if (lane < p.top_k) {
    const size_t s = static_cast<size_t>(t) * p.top_k + lane;
    r = __ldg(p.slot_rows + s);
    if (r >= p.num_rows) {
      atomicOr(p.status, kStatusBadSlot);
      r = -1;
    }
    if (r >= 0) *w = p.weights != nullptr ? __ldg(p.weights + s) : 1.0f;
  }
  return r;
}

constexpr int kCombineWarps = 8;

// Bound by the rows' bytes.  A warp per (token, 32 kSeq kUnits vectors): its slots are read
// once, a lane each, and the loads of kBatch rows of kUnits vectors are in flight together
// (kBatch by top_k, so that few of the unrolled rows are idle: top-2 with batches of 8 took twice
// as long; single elements, for rows that are not 16-byte aligned, in larger units).  At 64
// registers a thread half of an SM's warps are resident, which keeps enough loads in flight
// (with 100 registers and a quarter, 32768 rows of 8 KB to 4096 tokens took 73 us, now 47: 6.4 TB/s).
template <class T, int VN, int kBatch, int kSeq, int kUnits>
__global__ void __launch_bounds__(32 * kCombineWarps, 4) gmm_combine_kernel(const __grid_constant__ CombineParams p) {
  const int lane = threadIdx.x & 31;
  const int nvec = static_cast<int>(p.row_bytes / (sizeof(T) * VN));
  constexpr int kPiece = 32 * kSeq * kUnits;
  const uint32_t pieces = static_cast<uint32_t>((nvec + kPiece - 1) / kPiece);
  const uint32_t u = blockIdx.x * kCombineWarps + (threadIdx.x >> 5);
  const uint32_t t = u / pieces;
  if (t >= static_cast<uint32_t>(p.num_tokens)) return;
  const int first = static_cast<int>(u - t * pieces) * kPiece + lane;
  float w;
  const int r = route_slot(p, static_cast<int>(t), lane, &w);
#pragma unroll
  for (int s = 0; s < kSeq; ++s) {
    const int v0 = first + 32 * kUnits * s;
    float acc[kUnits][VN];
#pragma unroll
    for (int q = 0; q < kUnits; ++q)
#pragma unroll
      for (int i = 0; i < VN; ++i) acc[q][i] = 0.0f;
    for (int j0 = 0; j0 < p.top_k; j0 += kBatch) {
      RoutePack<T, VN> x[kBatch][kUnits];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int rj = __shfl_sync(0xffffffffu, r, (j0 + j) & 31);   // (a lane past top_k holds -1)
#pragma unroll
        for (int q = 0; q < kUnits; ++q)
          if (rj >= 0 && j0 + j < p.top_k && v0 + 32 * q < nvec)
            x[j][q] = route_load<T, VN>(p.rows + rj * p.row_bytes, v0 + 32 * q);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int rj = __shfl_sync(0xffffffffu, r, (j0 + j) & 31);
        const float wj = __shfl_sync(0xffffffffu, w, (j0 + j) & 31);
        if (rj >= 0 && j0 + j < p.top_k) {
#pragma unroll
          for (int q = 0; q < kUnits; ++q)
            if (v0 + 32 * q < nvec) {
              float y[VN];
              route_unpack<T, VN>(x[j][q], y);
              route_fma<VN>(acc[q], wj, y);
            }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kUnits; ++q)
      if (v0 + 32 * q < nvec) route_store<T, VN>(p.out + t * p.out_pitch, v0 + 32 * q, acc[q]);
  }
}

// Bound by the bytes of d_out, rows and d_rows.  warps_per_token warps per token (a power of two
// up to kCombineWarps, more than one where there are few tokens): they take the token's
// 32 kUnits-vector pieces in turn, kRows rows at a time, and join their dot products through
// shared memory in warp order.  The loads of a piece's kUnits (kRows + 1) vectors are in flight
// together.  16384 tokens of 8 KB, top-2: 101 us, 6.6 TB/s (118 with a third of the warps
// resident and four rows' code for two); 1003 tokens of 1411 fp32, top-6: 15.2 us with six
// rows' code, 1.5 more with four's.
template <class T, int VN, int kRows, int kUnits>
__global__ void __launch_bounds__(32 * kCombineWarps, kRows == 8 ? 3 : 4)
    gmm_combine_grad_kernel(const __grid_constant__ CombineParams p) {
  __shared__ float part[kCombineWarps][kRouteMaxTopK];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nvec = static_cast<int>(p.row_bytes / (sizeof(T) * VN));
  const int wpt = p.warps_per_token, tpc = kCombineWarps / wpt;
  const int t = static_cast<int>(blockIdx.x) * tpc + warp / wpt, sub = warp % wpt;
  const bool live = t < p.num_tokens;
  float w = 0.0f;
  int r = -1;
  if (live) r = route_slot(p, t, lane, &w);
  const uint8_t *g_row = p.d_out + (live ? t : 0) * p.out_pitch;
  for (int j0 = 0; j0 < p.top_k; j0 += kRows) {
    int rj[kRows];
    float wj[kRows], dot[kRows];
    bool any = false;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      rj[j] = __shfl_sync(0xffffffffu, r, (j0 + j) & 31);
      wj[j] = __shfl_sync(0xffffffffu, w, (j0 + j) & 31);
      if (j0 + j >= p.top_k) rj[j] = -1;
      any = any || rj[j] >= 0;
      dot[j] = 0.0f;
    }
    if (any) {
      for (int v0 = sub * 32 * kUnits + lane; v0 < nvec; v0 += wpt * 32 * kUnits) {
        RoutePack<T, VN> g[kUnits], x[kUnits][kRows];
#pragma unroll
        for (int q = 0; q < kUnits; ++q)
          if (v0 + 32 * q < nvec) {
            g[q] = route_load<T, VN>(g_row, v0 + 32 * q);
#pragma unroll
            for (int j = 0; j < kRows; ++j)
              if (rj[j] >= 0 && p.d_weights != nullptr)
                x[q][j] = route_load<T, VN>(p.rows + rj[j] * p.row_bytes, v0 + 32 * q);
          }
#pragma unroll
        for (int q = 0; q < kUnits; ++q)
          if (v0 + 32 * q < nvec) {
            float gv[VN];
            route_unpack<T, VN>(g[q], gv);
#pragma unroll
            for (int j = 0; j < kRows; ++j)
              if (rj[j] >= 0) {
                float y[VN];
                if (p.d_weights != nullptr) {
                  route_unpack<T, VN>(x[q][j], y);
#pragma unroll
                  for (int i = 0; i < VN; ++i) dot[j] = fmaf(gv[i], y[i], dot[j]);
                }
#pragma unroll
                for (int i = 0; i < VN; ++i) y[i] = wj[j] * gv[i];
                route_store<T, VN>(p.d_rows + rj[j] * p.row_bytes, v0 + 32 * q, y);
              }
          }
      }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
      if (lane == 0 && j0 + j < p.top_k) part[warp][j0 + j] = dot[j];
    }
  }
  if (p.d_weights == nullptr) return;
  __syncthreads();
  if (live && sub == 0 && lane < p.top_k) {
    float d = 0.0f;
    for (int i = 0; i < wpt; ++i) d += part[warp + i][lane];
    p.d_weights[static_cast<size_t>(t) * p.top_k + lane] = d;
  }
}

}  // namespace gmm
