// The gradient of the expert weights on 8-bit operands, for sm_103a:
//   d_b[g, n, k] (+)= sum_{r in group g} dc[r, n] * a[r, k],
//   dc[r, n] = 2^(sd - 127) qd[n, at(r)],  a[r, k] = 2^(sa - 127) qa[k, at(r)]
// with e4m3 codes q, stored transposed, and an exponent code s for each 128 rows of a group and
// column (gmm_quantize_fp8_cols).  The contraction runs over the group's rows, 128 (one scale
// block, a 128-byte swizzled row of codes) a stage; the scales enter in the tensor core
// (tcgen05.mma kind::mxf8f6f4, a scale for each 32 of K: the block's, four times).
//
// A tile is 256 n over a CTA pair (the MMA's M) times up to 240 k (its N): K is cut into
// ceil(K / 240) tiles whose widths are multiples of 16 and differ by 16 at most, so that no column
// is computed twice or for nothing.  240 because tensor memory holds two such accumulators, one
// under the MMAs and one under the epilogue, beside 12 columns of scales.
//
// Scales.  A stage needs one byte per operand row; the MMA takes a 32-bit word per row (four scales,
// here the same byte) from tensor memory, row m in lane m % 32 and column m / 32.  Warps load the
// bytes ahead, four stages at a time, and write each 128 rows' words as a 512-byte atom that
// tcgen05.cp spreads over the lane quadrants, in order with the MMAs.  Both CTAs hold the scales of
// all of the tile's k and of their own 128 n.  They have a ring of their own, of entries of four
// stages: the way of a scale (a freed entry, the peer's warps, its forwarder, the leader) takes
// longer than the values' ring is deep.
//
// Roles (416 threads per CTA):
//   warp 0       TMA producer of both operands' codes;
//   warp 1       TMEM allocation; in the pair's leader the scale copies and MMAs, in the peer the news
//                that its scales of a stage are written;
//   warps 2..9   epilogue, one or two per TMEM lane quadrant (the host's choice): 32 columns at a time
//                through shared memory to a TMA store (or reduction, when the call accumulates);
//   warps 10..12 scales: the n rows' block, and the k rows' two.
// Measured: 32768 rows over 8 groups, N = 14336, K = 4096, bf16: 1083 us, 3.55 PFLOP/s; 1245 back to back,
// at the power cap.  Power bounds it: the tensor pipe is 83% active at 1.64 GHz (ncu, half the groups of half
// the rows), and the launch without operand loads and epilogue takes 12% fewer cycles.  Many short groups in
// fp32 (64 groups, 16384 rows, N = 2816, K = 2048): 278 us, the gradient's 1.5 GB at 5.3 TB/s.
//
// Every group has the same tiles, so a tile's group is a division, and the offsets are in shared
// memory: each role finds its tiles itself.  Every wait is bounded as in the grouped kernel.
#pragma once

#include <type_traits>

#include "gmm_common.cuh"
#include "gmm_kernel.cuh"

namespace gmm {

constexpr uint32_t kWgEpiWarps = 8;
constexpr uint32_t kWgScaleWarps = 3;
constexpr uint32_t kWgFirstScaleWarp = 2 + kWgEpiWarps;
constexpr int kWgThreads = 32 * static_cast<int>(2 + kWgEpiWarps + kWgScaleWarps);
constexpr uint32_t kWgBlock = 128;                           // rows of a stage, and of a scale
constexpr uint32_t kWgTileN = 2 * kBlockN;                   // n of a pair's tile
constexpr uint32_t kWgMaxK = 240;                            // k of a tile, at most
constexpr uint32_t kWgUnit = 16;                             // widths are multiples of it
constexpr uint32_t kWgABytes = kBlockN * kWgBlock;           // a CTA's 128 n
constexpr uint32_t kWgBBytes = kWgMaxK / 2 * kWgBlock;       // a CTA's half of the k
constexpr uint32_t kWgAtom = 512;                            // scale words of 128 rows
constexpr uint32_t kWgScaleBytes = 3 * kWgAtom;              // a stage's
constexpr int kWgAhead = 4;                                  // stages of an entry of the scales' ring
constexpr uint32_t kWgEntryBytes = kWgAhead * kWgScaleBytes;
constexpr uint32_t kWgEntries = 3;
constexpr uint32_t kWgStageBytes = kWgABytes + kWgBBytes;
constexpr uint32_t kWgAccCols = kWgMaxK;
constexpr uint32_t kWgScaleCol = 2 * kWgAccCols;
template <bool kBf16>
constexpr uint32_t kWgStgBytes = 32 * 32 * (kBf16 ? 2 : 4);  // one staging buffer: 32 n x 32 k
constexpr int kWgMaxStages = 8;
constexpr uint64_t kWgStageNs = 4000;   // allowed for one stage of a tile (0.3 us measured, of one tile alone)
constexpr size_t kWgFixedBytes = 1024 + kWgEntries * kWgEntryBytes;   // and the staging buffers
static_assert(kWgScaleCol + 12 <= kTmemCols, "scales beside the accumulators");
static_assert(kWgABytes % 1024 == 0 && kWgBBytes % 1024 == 0 && kWgStgBytes<true> % 1024 == 0, "swizzled tiles start at 1024 bytes");

struct alignas(128) WeightGradParams {
  CUtensorMap d_map;        // codes of dc {pitch, N}, box {128, 128}, 128-byte swizzle
  CUtensorMap a_map[2];     // codes of a {pitch, K}, box {128, half of a narrow / wide tile}
  CUtensorMap out_map[2];   // d_b {K, N, G}, box {16, 32, 1} / {32, 32, 1}, the staging buffer's swizzle
  const uint8_t *d_scales;  // [pitch / 128, N]
  const uint8_t *a_scales;  // [pitch / 128, K]
  const uint32_t *a_offsets;   // [G + 1], or null: no group has rows
  uint32_t *status;
  int num_groups;
  int rows;
  int N;
  int K;
  int num_stages;
  int epi_warps;            // epilogue warps at work: 4 or 8
  int stg_bufs;             // staging buffers of each: 1 or 2
  int accumulate;
  uint32_t k_tiles;         // tiles along K, of which the first `wide` are 16 wider than `width`
  uint32_t wide;
  uint32_t width;
  uint32_t n_tiles;
  Divisor band;           // n tiles per band of the tile order (the last band has n_tiles % band, `rest`)
  Divisor rest;
  Divisor whole;          // tiles of a whole band: band * k_tiles
  Divisor per_group;      // n_tiles * k_tiles
  uint32_t total;           // tiles
  unsigned long long wait_limit_ns;
};

struct WgTile {
  uint32_t g, n0, k0, width, stages, block0;   // block0: the group's first block
  bool wide;
};

// Within a group the n tiles are cut into bands; a band is walked k tile by k tile with its n tiles
// fastest, so that tiles that run side by side share both operands' panels in L2.
__device__ __forceinline__ WgTile wg_tile(const WeightGradParams &p, const uint32_t *off, uint32_t t) {
  WgTile x;
  x.g = p.per_group.quotient(t);
  const uint32_t in = t - x.g * p.per_group.d, b = p.whole.quotient(in), in_band = in - b * p.whole.d;
  const bool last = (b + 1u) * p.band.d > p.n_tiles;
  const uint32_t kt = last ? p.rest.quotient(in_band) : p.band.quotient(in_band);
  const uint32_t nt = b * p.band.d + in_band - kt * (last ? p.rest.d : p.band.d);
  x.n0 = nt * kWgTileN;
  x.wide = kt < p.wide;
  x.k0 = kt * p.width + min(kt, p.wide) * kWgUnit;
  x.width = p.width + (x.wide ? kWgUnit : 0u);
  const uint32_t r0 = off[x.g];
  x.stages = (off[x.g + 1] - r0 + kWgBlock - 1) / kWgBlock;
  x.block0 = r0 / kWgBlock + x.g;
  return x;
}

struct __align__(16) WgCtrl {
  uint64_t full[kWgMaxStages];       // leader: both CTAs' bytes
  uint64_t empty[kWgMaxStages];      // the MMAs that read the stage completed (both CTAs)
  uint64_t scales_full[kWgEntries];  // leader: its scale warps, the peer's forwarder
  uint64_t scales_empty[kWgEntries]; // the copies that read the entry completed (both CTAs)
  uint64_t scales_in[kWgEntries];    // peer: its scale warps have written an entry
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ void wg_store_3d(const CUtensorMap *map, uint32_t src, int32_t x, int32_t y, int32_t z, bool add) {
  if (add)
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group.L2::cache_hint [%0, {%2, %3, %4}], [%1], %5;" ::"l"(map),
                 "r"(src), "r"(x), "r"(y), "r"(z), "l"(l2_policy_evict_first())
                 : "memory");
}

// 16-byte chunk j of row r in a staging buffer, as the store's tensor map has it swizzled over its
// rows of 32, 64 or 128 bytes.
template <uint32_t kRowBytes>
__device__ __forceinline__ uint32_t wg_chunk(uint32_t r, uint32_t j) {
  return r * kRowBytes + ((j ^ (r / (128 / kRowBytes) & (kRowBytes / 16 - 1))) << 4);
}

// kCols fp32 columns of the thread's row to a staging buffer.
template <bool kBf16, int kCols>
__device__ __forceinline__ void wg_stage_row(uint32_t stg, uint32_t r, const uint32_t (&v)[kCols]) {
  constexpr uint32_t kRow = kCols * (kBf16 ? 2 : 4);
#pragma unroll
  for (uint32_t j = 0; j < kRow / 16; ++j) {
    const uint32_t at = stg + wg_chunk<kRow>(r, j);
    if constexpr (kBf16) {
      uint32_t w[4];
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i)
        w[i] = pack_bf16x2(__uint_as_float(v[8 * j + 2 * i]), __uint_as_float(v[8 * j + 2 * i + 1]));
      st_shared_v4(at, w[0], w[1], w[2], w[3]);
    } else {
      st_shared_v4(at, v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
  }
}

template <bool kBf16>
__global__ void __launch_bounds__(kWgThreads, 1) gmm_weight_grad_fp8_kernel(const __grid_constant__ WeightGradParams p) {
  __shared__ WgCtrl ctl;
  extern __shared__ uint8_t dyn_smem[];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = static_cast<int>(__shfl_sync(0xffffffffu, static_cast<uint32_t>(tid) >> 5, 0));
  const uint32_t ST = static_cast<uint32_t>(p.num_stages);
  const uint32_t rank = __shfl_sync(0xffffffffu, cluster_ctarank(), 0);

  const uint32_t dyn_base = smem_addr(dyn_smem);
  const uint32_t a_ring = (dyn_base + 1023u) & ~1023u;
  const uint32_t b_ring = a_ring + ST * kWgABytes;
  const uint32_t stg_ring = b_ring + ST * kWgBBytes;
  const uint32_t stg_bufs = static_cast<uint32_t>(p.stg_bufs);
  const uint32_t epi_warps = static_cast<uint32_t>(p.epi_warps);
  const uint32_t s_ring = stg_ring + epi_warps * stg_bufs * kWgStgBytes<kBf16>;
  uint32_t *off = reinterpret_cast<uint32_t *>(dyn_smem + (s_ring + kWgEntries * kWgEntryBytes - dyn_base));

  if (tid == 0) {
    set_wait_limit(p.wait_limit_ns);
    for (uint32_t s = 0; s < ST; ++s) {
      mbar_init(smem_addr(&ctl.full[s]), 1);
      mbar_init(smem_addr(&ctl.empty[s]), 1);
    }
    for (uint32_t s = 0; s < kWgEntries; ++s) {
      mbar_init(smem_addr(&ctl.scales_full[s]), kWgScaleWarps + 1);
      mbar_init(smem_addr(&ctl.scales_empty[s]), 1);
      mbar_init(smem_addr(&ctl.scales_in[s]), kWgScaleWarps);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_addr(&ctl.acc_full[a]), 1);
      mbar_init(smem_addr(&ctl.acc_empty[a]), 2 * epi_warps);
    }
    ctl.abort = 0;
    fence_barrier_init();
    if (p.a_offsets != nullptr) {   // else there are no operands
      prefetch_tensormap(&p.d_map);
      prefetch_tensormap(&p.a_map[0]);
      prefetch_tensormap(&p.a_map[1]);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_addr(&ctl.tmem_base), kTmemCols);
    tmem_relinquish_pair();
    tc_fence_before_sync();
  }
  bool bad = false;
  for (int g = tid; g <= p.num_groups; g += kWgThreads) {
    const uint32_t r = p.a_offsets != nullptr ? __ldg(p.a_offsets + g) : 0u;
    off[g] = r;
    bad |= r > static_cast<uint32_t>(p.rows);
    if (p.a_offsets != nullptr && g < p.num_groups) bad |= __ldg(p.a_offsets + g + 1) < r;
  }
  bad = __syncthreads_or(bad);
  cluster_sync();   // the peer's barriers are initialised before anyone signals them
  if (bad && blockIdx.x == 0 && tid == 0) atomicOr(p.status, kStatusBadOffsets);
  tc_fence_after_sync();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, ctl.tmem_base, 0);
  const uint32_t total = bad ? 0u : p.total;
  volatile int *abort = &ctl.abort;
  const uint32_t unit0 = cluster_id_x(), units = cluster_count_x();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      // The operands' panels are read by many tiles, the gradient is written once: they are to stay in
      // L2 (prefill shapes 1100 -> 1088 us, 64 experts in fp32 276 -> 272).
      const uint64_t pol = l2_policy_evict_last();
      Ring rt;
      uint32_t pending = 0, pend_phase = 0;
      bool ok = true;
      for (uint32_t t = unit0; t < total && ok; t += units) {
        const WgTile x = wg_tile(p, off, t);
        const uint32_t half = x.width / 2, tx = 2u * (kWgABytes + half * kWgBlock);
        const int32_t d_row = static_cast<int32_t>(x.n0 + rank * kBlockN), a_row = static_cast<int32_t>(x.k0 + rank * half);
        const CUtensorMap *a_map = &p.a_map[x.wide];
        for (uint32_t kb = 0; kb < x.stages; ++kb) {
          if (!wait_phase(smem_addr(&ctl.empty[rt.slot]), rt.phase ^ 1u, abort)) { ok = false; break; }
          const uint32_t full_local = smem_addr(&ctl.full[rt.slot]);
          if (rank == 0) mbar_arrive_expect_tx(full_local, tx);
          const uint32_t full_leader = map_to_rank(full_local, 0);
          const int32_t col = static_cast<int32_t>((x.block0 + kb) * kWgBlock);
          tma_load_2d_pair(a_ring + rt.slot * kWgABytes, &p.d_map, full_leader, col, d_row, pol);
          tma_load_2d_pair(b_ring + rt.slot * kWgBBytes, a_map, full_leader, col, a_row, pol);
          pending |= 1u << rt.slot;
          pend_phase = (pend_phase & ~(1u << rt.slot)) | (rt.phase << rt.slot);
          rt.next(ST);
        }
      }
      if (!ok) {
        // As in the grouped kernel: the leader lets the copies already issued land (its
        // barriers count both CTAs' bytes), the peer is held at the final cluster barrier.
        for (uint32_t s = 0; s < ST; ++s)
          if ((pending & (1u << s)) && rank == 0)
            wait_phase_for(smem_addr(&ctl.full[s]), (pend_phase >> s) & 1u, kDrainLimitNs);
        atomicOr(p.status, kStatusTimeout);
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ---------------------------------------------------------- scale copies and MMAs (leader)
      Ring rt, rs;
      uint32_t acc = 0, acc_phase = 0;
      bool ok = true;
      const uint64_t a_desc = smem_desc_k_sw128(a_ring), b_desc = smem_desc_k_sw128(b_ring);
      const uint64_t s_desc = smem_desc_scales(s_ring);
      const uint32_t a_lo = static_cast<uint32_t>(a_desc), b_lo = static_cast<uint32_t>(b_desc);
      const uint32_t v_hi = static_cast<uint32_t>(a_desc >> 32);
      const uint32_t s_lo = static_cast<uint32_t>(s_desc), s_hi = static_cast<uint32_t>(s_desc >> 32);
      const uint32_t full0 = smem_addr(&ctl.full[0]), empty0 = smem_addr(&ctl.empty[0]);
      const uint32_t s_full0 = smem_addr(&ctl.scales_full[0]), s_empty0 = smem_addr(&ctl.scales_empty[0]);
      const uint32_t sfa = tmem_base + kWgScaleCol, sfb = sfa + 4u;
      for (uint32_t t = unit0; t < total && ok; t += units) {
        const WgTile x = wg_tile(p, off, t);   // ahead of its use, behind a tile's first MMAs, it measured slower (1.92 M cycles for 1.77)
        if (x.stages == 0) continue;
        if (!__all_sync(0xffffffffu, wait_phase_cluster<true>(smem_addr(&ctl.acc_empty[acc]), acc_phase ^ 1u, abort))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + acc * kWgAccCols;
        const uint32_t idesc = idesc_e4m3_mx_f32(kWgTileN, x.width), two = x.width > 128u;
        for (uint32_t kb = 0; kb < x.stages; ++kb) {
          const uint32_t in = kb % kWgAhead;
          bool there = true;
          if (in == 0) there = wait_phase_cluster(s_full0 + rs.slot * 8u, rs.phase, abort);
          there = there && wait_phase_cluster<true>(full0 + rt.slot * 8u, rt.phase, abort);
          if (!__all_sync(0xffffffffu, there)) { ok = false; break; }
          tc_fence_after_sync();
          mma_stage_e4m3_mx_pair(d_tmem, a_lo + rt.slot * (kWgABytes >> 4), b_lo + rt.slot * (kWgBBytes >> 4), v_hi, idesc,
                                 s_lo + ((rs.slot * kWgEntryBytes + in * kWgScaleBytes) >> 4), s_hi, sfa, sfb, kb != 0, two,
                                 empty0 + rt.slot * 8u);
          rt.next(ST);
          if (in == kWgAhead - 1 || kb + 1 == x.stages) {
            mma_commit_pair(s_empty0 + rs.slot * 8u, 0x3);
            rs.next(kWgEntries);
          }
        }
        if (!ok) break;
        mma_commit_pair(smem_addr(&ctl.acc_full[acc]), 0x3);
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!ok && lane == 0) atomicOr(p.status, kStatusTimeout);
    } else if (lane == 0) {
      // The peer's scales to the leader, whose MMA warp issues the copies that read them: acquired
      // in this CTA, released at cluster scope.
      const uint32_t full0 = map_to_rank(smem_addr(&ctl.scales_full[0]), 0);
      Ring rs;
      bool ok = true;
      for (uint32_t t = unit0; t < total && ok; t += units) {
        const uint32_t stages = wg_tile(p, off, t).stages;
        for (uint32_t kb = 0; kb < stages; kb += kWgAhead) {
          if (!wait_phase(smem_addr(&ctl.scales_in[rs.slot]), rs.phase, abort)) { ok = false; break; }
          mbar_arrive_cluster_shared(full0 + rs.slot * 8u);
          rs.next(kWgEntries);
        }
      }
      if (!ok) atomicOr(p.status, kStatusTimeout);
    }
    __syncwarp();
  } else if (warp < static_cast<int>(kWgFirstScaleWarp)) {
    // ------------------------------------------------------------ epilogue
    const uint32_t quad = static_cast<uint32_t>(warp & 3), r = static_cast<uint32_t>(lane);
    const uint32_t ew = static_cast<uint32_t>(warp - 2), stg0 = stg_ring + ew * stg_bufs * kWgStgBytes<kBf16>;
    const uint32_t acc_empty0 = map_to_rank(smem_addr(&ctl.acc_empty[0]), 0);
    const bool add = p.accumulate != 0;
    uint32_t acc = 0, acc_phase = 0, buf = 0;
    for (uint32_t t = ew < epi_warps ? unit0 : total; t < total; t += units) {
      const WgTile x = wg_tile(p, off, t);
      const bool zero = x.stages == 0;
      if (zero && add) continue;
      const uint32_t n = x.n0 + rank * kBlockN + quad * 32u;   // this warp's first row of d_b
      const bool in = n < static_cast<uint32_t>(p.N);
      const uint32_t taddr = tmem_base + ((quad * 32u) << 16) + acc * kWgAccCols;
      if (!zero) {
        int ok = 1;
        // A whole tile's wait, as long as its group.  What stops a stage ends that role's own wait, and this one by `abort`.
        if (lane == 0) ok = wait_phase(smem_addr(&ctl.acc_full[acc]), acc_phase, abort, x.stages * kWgStageNs);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) {
          if (lane == 0) atomicOr(p.status, kStatusTimeout);
          break;
        }
        tc_fence_after_sync();
      }
      if (in) {
        // 32 columns at a time, or 16 at the end of a tile that is no multiple of 32 wide.
        auto store = [&](uint32_t c, auto cols) {
          constexpr int kCols = decltype(cols)::value;
          uint32_t v[kCols];
          if (zero) {
#pragma unroll
            for (int i = 0; i < kCols; ++i) v[i] = 0u;
          } else if constexpr (kCols == 32) {
            tmem_ld_x32(taddr + c, v);
          } else {
            tmem_ld_x16(taddr + c, v);
          }
          const uint32_t stg = stg0 + buf * kWgStgBytes<kBf16>;
          if (lane == 0) {   // the buffer's last store has read it
            if (stg_bufs == 2u) bulk_wait_read<1>(); else bulk_wait_read<0>();
          }
          if (!zero) tmem_ld_wait();
          __syncwarp();
          wg_stage_row<kBf16, kCols>(stg, r, v);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            wg_store_3d(&p.out_map[kCols == 32], stg, static_cast<int32_t>(x.k0 + c), static_cast<int32_t>(n),
                        static_cast<int32_t>(x.g), add);
            bulk_commit();
          }
          buf = buf + 1 == stg_bufs ? 0u : buf + 1;
        };
        for (uint32_t c = 32u * (ew >> 2); c < x.width; c += 8u * epi_warps) {
          if (c + 32u <= x.width) store(c, std::integral_constant<int, 32>());
          else store(c, std::integral_constant<int, 16>());
        }
      }
      if (!zero) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty0 + acc * 8u);
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
    }
    if (lane == 0) bulk_wait_read<0>();   // the staging buffers; the stores complete with the grid
  } else {
    // ------------------------------------------------------------ scales
    // Rows past the matrix repeat its last one (their results are not stored).
    const uint32_t role = static_cast<uint32_t>(warp) - kWgFirstScaleWarp;
    const uint32_t written0 = smem_addr(rank == 0 ? &ctl.scales_full[0] : &ctl.scales_in[0]);
    const uint8_t *base = role == 0 ? p.d_scales : p.a_scales;
    const uint32_t width = static_cast<uint32_t>(role == 0 ? p.N : p.K);
    const uint32_t dst0 = s_ring + role * kWgAtom + static_cast<uint32_t>(lane) * 16u;
    Ring rs;
    bool ok = true;
    uint32_t t = unit0, kb = 0;   // the next chunk of kWgAhead stages
    WgTile x{};
    uint32_t pos[4] = {0, 0, 0, 0};
    auto enter = [&]() {   // to the first tile from t on that has stages
      for (; t < total; t += units) {
        x = wg_tile(p, off, t);
        if (x.stages != 0) break;
      }
      kb = 0;
#pragma unroll
      for (uint32_t c = 0; c < 4; ++c) {
        const uint32_t m = 32u * c + static_cast<uint32_t>(lane);
        pos[c] = min(role == 0 ? x.n0 + rank * kBlockN + m : x.k0 + (role - 1u) * 128u + m, width - 1u);
      }
    };
    // A chunk's scales, and how many stages it has (0: there is none).
    auto load = [&](uint32_t (&v)[kWgAhead][4]) -> uint32_t {
      if (t >= total) return 0u;
      const uint32_t n = min(static_cast<uint32_t>(kWgAhead), x.stages - kb);
#pragma unroll
      for (uint32_t i = 0; i < kWgAhead; ++i)
        if (i < n) {
          const uint8_t *row = base + static_cast<size_t>(x.block0 + kb + i) * width;
#pragma unroll
          for (int c = 0; c < 4; ++c) v[i][c] = __ldg(row + pos[c]);
        }
      kb += n;
      if (kb == x.stages) {
        t += units;
        enter();
      }
      return n;
    };
    auto put = [&](const uint32_t (&v)[kWgAhead][4], uint32_t n) {
      if (!ok) return;
      if (!__all_sync(0xffffffffu, wait_phase(smem_addr(&ctl.scales_empty[rs.slot]), rs.phase ^ 1u, abort))) {
        ok = false;
        return;
      }
      const uint32_t dst = dst0 + rs.slot * kWgEntryBytes;
#pragma unroll
      for (uint32_t i = 0; i < kWgAhead; ++i)
        if (i < n)
          st_shared_v4(dst + i * kWgScaleBytes, v[i][0] * 0x01010101u, v[i][1] * 0x01010101u, v[i][2] * 0x01010101u,
                       v[i][3] * 0x01010101u);
      fence_async_smem();   // these writes, before the tensor-memory copies read them
      __syncwarp();
      if (lane == 0) mbar_arrive(written0 + rs.slot * 8u);
      rs.next(kWgEntries);
    };
    uint32_t v0[kWgAhead][4], v1[kWgAhead][4];
    enter();
    uint32_t n0 = load(v0);
    while (n0 != 0u && ok) {
      const uint32_t n1 = load(v1);
      put(v0, n0);
      n0 = load(v0);
      if (n1 != 0u) put(v1, n1);
    }
    if (!ok && lane == 0) atomicOr(p.status, kStatusTimeout);
  }

  __syncthreads();
  cluster_sync();   // no CTA leaves while its peer may still signal it
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

}  // namespace gmm
