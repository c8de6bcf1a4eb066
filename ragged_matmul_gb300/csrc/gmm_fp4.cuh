// 4-bit block-scaled grouped GEMM (e2m1 operands, e4m3 or e8m0 block scales), for sm_103a.
//
// Operation, for each active group g with expert e and rows r of the group (b = 16 for
// nvfp4, 32 for mxfp4):
//   C[r, n] = bf16( epi( ga * gb[e] * sum_k sa[r, k / b] qa[r, k] sb[e, n, k / b] qb[e, n, k] ) )
// The scales enter in the tensor core (tcgen05.mma kind::mxf4nvf4), fp32 accumulation.
//
// Orientation and pairs are the grouped kernel's: weights are the MMA's M (256 rows over a
// CTA pair), tokens its N (a multiple of 16 up to 240).  A stage is 256 of K: 128-byte rows
// of packed values, so the value operands go through the bf16 kernel's tensor maps, swizzle
// and descriptors unchanged.
//
// Scales.  The MMA takes them from tensor memory, 4 scales (one 32-bit word) per operand
// row, row m in lane m % 32 and column m / 32, the same in all four lane quadrants.  In
// global memory a row's scales follow one another (16 bytes per stage for nvfp4, 8 for
// mxfp4), rows may start anywhere, and a tensor copy cannot transpose 4-byte words.  So
// warps load them: lane l takes rows l, l + 32, l + 64, l + 96 of a 128-row block, and the
// four rows' word j are 16 bytes of a 512-byte atom (one per block and word) in the stage's
// shared memory, from where tcgen05.cp spreads it over the quadrants.  The copies run in
// order with the MMAs of the issuing thread and beside them (12 copies and 4 MMAs of 192
// columns measured 385 cycles, the MMAs alone 385), so one set of scale columns serves all
// stages.
// Both CTAs of a pair hold the scales of all the tile's tokens (each computes its own 128
// weight rows against all of them), and of their own 128 weight rows.
//
// Tensor memory: two accumulators of 240 columns and 24 columns of scales (half a stage's).
//
// Roles (448 threads per CTA):
//   warp 0        TMA producer of the stage's weight and token values.
//   warp 1        TMEM allocation; in the pair's leader the scale copies and MMAs, in the peer the
//                 news that the peer's scales of a stage are written (see the scales' role).
//   warps 2..9    epilogue, two per TMEM lane quadrant taking every second 32-row chunk.
//   warps 10..12  scales: the weight rows' block, and the tokens' two.
//   warp 13       scheduler: decodes the CTA's tiles into a queue that every role reads.
//
// Measured: 32768 rows over 8 experts, K = 4096, N = 14336, nvfp4: 0.63 ms, 6.1 PFLOP/s (0.70 to
// 0.73 back to back, at the power cap).  Measured by parts, of 0.64 ms: the MMAs alone 0.42; without
// them 0.574, without the epilogue too 0.518, which is 37 KB a stage and CTA (31 KB of values, 6 KB
// of scales) entering the SMs at 18.4 TB/s, 64 bytes a clock and SM.  So a tile holds as many tokens
// as tensor memory allows beside a second accumulator (224 instead of 240: 0.693 ms).  Whether
// multicast would shorten that part is open: a program of copies alone gained nothing from it, but it
// brought only 45 to 48 bytes a clock into an SM with it or without.  2048 rows over 64 experts,
// K = 2048, N = 2816: 46 us with cold weights, 4.8 TB/s.
//
// Tiles are claimed by the pair as the grouped kernel's are (a static share where there are
// few).  Every wait is bounded as in the grouped kernel.
#pragma once

#include <type_traits>

#include "gmm_kernel.cuh"

namespace gmm {

constexpr uint32_t kF4EpiWarps = 8;
constexpr uint32_t kF4ScaleWarps = 3;
constexpr uint32_t kF4FirstScaleWarp = 2 + kF4EpiWarps;
constexpr int kF4Threads = 32 * static_cast<int>(2 + kF4EpiWarps + kF4ScaleWarps + 1);
constexpr uint32_t kF4MaxTok = 240;
constexpr uint32_t kF4TokAlign = 16;
constexpr uint32_t kF4TokMaps = kF4MaxTok / 16;             // a CTA loads half of a tile's tokens: 8, 16, ... 120 rows
static_assert(kF4TokMaps <= static_cast<uint32_t>(kTokMaps), "a map slot per copy height");
constexpr uint32_t kF4StageK = 256;
constexpr uint32_t kF4WBytes = kBlockN * 128;               // 128 weight rows x 128 bytes
constexpr uint32_t kF4TBytes = kF4MaxTok / 2 * 128;         // a CTA's half of the tokens
constexpr uint32_t kF4Atom = 512;                           // one scale word of 128 rows
constexpr uint32_t kF4AccCols = kF4MaxTok;
constexpr uint32_t kF4ScaleCol = 2 * kF4AccCols;            // scale columns follow the accumulators
constexpr uint32_t kF4Queue = 3;                            // tile queue entries
constexpr uint32_t kF4DynamicTiles = 8;                     // claimed tiles from this many tiles a pair
constexpr uint32_t kF4StgBytes = kEpiRows * kEpiRowBytes;   // one epilogue staging buffer
constexpr uint32_t kF4StgBufs = 2;                          // per epilogue warp

// Scale words per row and stage, and the instructions of K = 64 that share one.
template <bool kMx>
struct F4Scale {
  static constexpr uint32_t kWords = kMx ? 2 : 4;
  static constexpr uint32_t kStepsPerWord = kMx ? 2 : 1;
  static constexpr uint32_t kBlock = kMx ? 32 : 16;
  static constexpr uint32_t kBytes = 3 * kWords * kF4Atom;   // a stage's atoms: weights, then tokens
  static constexpr uint32_t kHalfWords = kWords / 2;         // words of half a stage, in tensor memory at a time
  static_assert(kF4ScaleCol + 12 * kHalfWords <= kTmemCols, "scales beside the accumulators");
};

template <bool kMx>
struct F4Geom {
  static constexpr uint32_t kRows = 2 * kBlockN;
  static constexpr uint32_t kMaxTok = kF4MaxTok;
  static constexpr uint32_t kTokAlign = kF4TokAlign;
  static constexpr uint32_t kStageBytes = kF4WBytes + kF4TBytes + F4Scale<kMx>::kBytes;
};
constexpr size_t kF4FixedBytes = 1024 + kF4EpiWarps * kF4StgBufs * kF4StgBytes;

struct alignas(128) F4Params : GmmParams {   // K counts two-byte units: 4 elements each
  const uint8_t *sf_a;     // [rows, sf_pitch]
  const uint8_t *sf_w;     // [E, N, sf_pitch]
  int sf_pitch;            // bytes, a multiple of 16
  const float *g_a;        // one value or null
  const float *g_w;        // [E] or null
};

__device__ __forceinline__ uint32_t warp_uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// Reader of the CTA's tile queue, which its scheduler warp fills in the order of the CTA's
// tiles: 1 with the tile, 0 after the last one, -1 when a wait gave up.  By a whole warp or by
// one thread of it (kWarp = false).
struct F4Feed {
  uint32_t pos = 0;
  template <bool kWarp = true>
  __device__ __forceinline__ int next(Ctrl &ctl, volatile int *abort, Tile *x) {
    const uint32_t slot = pos % kF4Queue, parity = (pos / kF4Queue) & 1u;
    bool ok = wait_phase_cluster(smem_addr(&ctl.tq_full[slot]), parity, abort);   // the leader fills both CTAs' queues
    if (kWarp) ok = __all_sync(0xffffffffu, ok);
    if (!ok) return -1;
    uint4 w0 = ld_shared_v4(smem_addr(&ctl.tq_info[slot])), w1 = ld_shared_v4(smem_addr(&ctl.tq_info[slot]) + 16u);
    if (kWarp) {
      w0.x = warp_uniform(w0.x);
      w0.y = warp_uniform(w0.y);
      w0.z = warp_uniform(w0.z);
      w0.w = warp_uniform(w0.w);
      w1.x = warp_uniform(w1.x);
      w1.y = warp_uniform(w1.y);
    }
    if (!kWarp || (threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&ctl.tq_empty[slot]));
    ++pos;
    x->e = static_cast<int32_t>(w0.x);
    x->single_block = w0.y;
    x->row0 = w0.z;
    x->nrows = w0.w;
    x->ntok = w1.x;
    x->n0 = w1.y;
    return w0.w != 0u;   // no rows: the end
  }
};

template <bool kMx>
__global__ void __launch_bounds__(kF4Threads, 1) gmm_fp4_kernel(const __grid_constant__ F4Params p) {
  using G = F4Geom<kMx>;
  using S = F4Scale<kMx>;
  constexpr uint32_t kFullArrivals = 1 + kF4ScaleWarps + 1;   // the values, the leader's scale warps, the peer's forwarder
  constexpr uint32_t kEpiArrivals = 2 * kF4EpiWarps;
  __shared__ Ctrl ctl;
  __shared__ uint64_t peer_free[kF4Queue];   // leader: the peer's readers have taken a queue entry
  __shared__ uint64_t scales_in[kMaxStages];   // peer: its scale warps have written a stage's atoms
  extern __shared__ uint8_t dyn_smem[];

  // Warp-uniform values that steer the roles are broadcast from lane 0: the compiler then knows
  // them to be uniform and keeps what the MMA warp computes from them in uniform registers,
  // which the tcgen05 instructions read.
  const int tid = threadIdx.x, warp = static_cast<int>(warp_uniform(static_cast<uint32_t>(tid) >> 5)), lane = tid & 31;
  const uint32_t ST = static_cast<uint32_t>(p.num_stages);
  const int KB = (p.K + kBK - 1) / kBK;   // stages per tile: 64 two-byte units = 256 of K
  const uint32_t rank = warp_uniform(cluster_ctarank());

  const uint32_t dyn_base = smem_addr(dyn_smem);
  const uint32_t w_ring = (dyn_base + 1023u) & ~1023u;
  const uint32_t t_ring = w_ring + ST * kF4WBytes;
  const uint32_t s_ring = t_ring + ST * kF4TBytes;
  const uint32_t epi_ring = s_ring + ST * S::kBytes;
  uint32_t *prefix = reinterpret_cast<uint32_t *>(dyn_smem + (epi_ring + kF4EpiWarps * kF4StgBufs * kF4StgBytes - dyn_base));

  if (tid == 0) {
    set_wait_limit(p.wait_limit_ns);
    for (uint32_t s = 0; s < ST; ++s) {
      mbar_init(smem_addr(&ctl.full[s]), kFullArrivals);
      mbar_init(smem_addr(&ctl.empty[s]), 1);
      mbar_init(smem_addr(&scales_in[s]), kF4ScaleWarps);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_addr(&ctl.acc_full[a]), 1);
      mbar_init(smem_addr(&ctl.acc_empty[a]), kEpiArrivals);
    }
    mbar_init(smem_addr(&ctl.maps_ready), 1);
    for (uint32_t q = 0; q < kF4Queue; ++q) {
      mbar_init(smem_addr(&peer_free[q]), 1);
      mbar_init(smem_addr(&ctl.tq_full[q]), 1);
      mbar_init(smem_addr(&ctl.tq_empty[q]), 2 + kF4EpiWarps + kF4ScaleWarps);   // warps 0 and 1 too
    }
    ctl.abort = 0;
    ctl.active = 0;
    ctl.flags = 0;
    ctl.max_group_tiles = 0;
    ctl.min_group_tiles = 0xffffffffu;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_addr(&ctl.tmem_base), kTmemCols);
    tmem_relinquish_pair();
    tc_fence_before_sync();
  }
  if (tid == 0) prefetch_tensormap(&p.w_map);
  __syncthreads();
  cluster_arrive();   // the peer's barriers are initialised before anyone signals them
  build_schedule<G>(p, ctl, prefix, kF4Threads);
  cluster_wait();

  if (blockIdx.x == 0 && tid == 0) {
    p.stats[1] = ctl.active;
    const uint32_t f = ctl.flags & (kStatusBadOffsets | kStatusBadExpert | kStatusTooLarge);
    if (f) atomicOr(p.status, f);
  }
  tc_fence_after_sync();
  const uint32_t tmem_base = warp_uniform(ctl.tmem_base);
  const uint32_t total = ctl.total_tiles;
  volatile int *abort = &ctl.abort;
  const uint32_t unit0 = cluster_id_x(), units = cluster_count_x();

  if (warp == 0) {
    // ------------------------------------------------------------ value producer
    uint8_t *slot = p.map_slots + static_cast<size_t>(blockIdx.x) * kMapSlotBytes;
    if (lane == 0) {
      const CUtensorMap *tok_maps = reinterpret_cast<const CUtensorMap *>(slot);
      const uint64_t pol_first = l2_policy_evict_first();
      const uint64_t pol_last = l2_policy_evict_last();
      const uint64_t pol_normal = l2_policy_evict_normal();
      Ring rt;
      uint32_t pending = 0, pend_phase = 0;
      bool ok = true, maps_acquired = false;
      F4Feed feed;
      for (Tile ti; ok;) {
        const int got = feed.next<false>(ctl, abort, &ti);
        if (got <= 0) {
          ok = got == 0;
          break;
        }
        const uint32_t my_tok = ti.ntok / 2;
        const uint32_t tx = 2u * (kF4WBytes + my_tok * 128u);
        const int32_t w_row = static_cast<int32_t>(ti.n0 + rank * kBlockN);
        const int32_t t_row = static_cast<int32_t>(ti.row0 + rank * my_tok);
        const uint64_t w_pol = (p.cache_hints && ti.single_block) ? pol_first : pol_normal;
        const uint64_t t_pol = p.cache_hints ? pol_last : pol_normal;
        if (!maps_acquired) {
          if (!wait_phase(smem_addr(&ctl.maps_ready), 0, abort)) { ok = false; break; }
          for (uint32_t i = 0; i < kF4TokMaps; ++i) tensormap_acquire(slot + i * 128);
          maps_acquired = true;
        }
        const CUtensorMap *tok = tok_maps + (my_tok / 8u - 1u);
        for (int kb = 0; kb < KB; ++kb) {
          const uint32_t full_local = smem_addr(&ctl.full[rt.slot]);
          if (!wait_phase(smem_addr(&ctl.empty[rt.slot]), rt.phase ^ 1u, abort)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(full_local, tx);
          const uint32_t full_leader = map_to_rank(full_local, 0);
          tma_load_3d_pair(w_ring + rt.slot * kF4WBytes, &p.w_map, full_leader, kb * kBK, w_row, ti.e, w_pol);
          tma_load_2d_pair(t_ring + rt.slot * kF4TBytes, tok, full_leader, kb * kBK, t_row, t_pol);
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
    // ------------------------------------------------------------ scale copies and MMAs (leader)
    if (rank == 0) {
      Ring rt;
      uint32_t acc = 0, acc_phase = 0;
      bool ok = true;
      const uint64_t w_desc = smem_desc_k_sw128(w_ring), t_desc = smem_desc_k_sw128(t_ring);
      const uint64_t s_desc = smem_desc_scales(s_ring);
      const uint32_t w_lo = static_cast<uint32_t>(w_desc), t_lo = static_cast<uint32_t>(t_desc);
      const uint32_t v_hi = static_cast<uint32_t>(w_desc >> 32);   // the same for both value operands
      const uint32_t s_lo = static_cast<uint32_t>(s_desc), s_hi = static_cast<uint32_t>(s_desc >> 32);
      const uint32_t full0 = smem_addr(&ctl.full[0]), empty0 = smem_addr(&ctl.empty[0]);
      const uint32_t sfa = tmem_base + kF4ScaleCol, sfb = sfa + 4u * S::kHalfWords;
      F4Feed feed;
      Tile ti, tn;
      int got = feed.next(ctl, abort, &ti);
      for (; got > 0; ti = tn) {
        const bool acc_free = __all_sync(
            0xffffffffu, wait_phase_cluster<true>(smem_addr(&ctl.acc_empty[acc]), acc_phase ^ 1u, abort));
        if (!acc_free) { ok = false; break; }
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + acc * kF4AccCols;
        const uint32_t idesc = idesc_e2m1_f32(G::kRows, ti.ntok, kMx, 0);
        const uint32_t idesc2 = idesc_e2m1_f32(G::kRows, ti.ntok, kMx, 2);
        const uint32_t two = ti.ntok > 128u;
        bool staged = false;
        for (int kb = 0; kb < KB; ++kb) {
          if (!staged) {
            if (!__all_sync(0xffffffffu, wait_phase_cluster(full0 + rt.slot * 8u, rt.phase, abort))) { ok = false; break; }
            tc_fence_after_sync();
          }
          const uint32_t a = w_lo + rt.slot * (kF4WBytes >> 4), b = t_lo + rt.slot * (kF4TBytes >> 4);
          const uint32_t s = s_lo + rt.slot * (S::kBytes >> 4), empty = empty0 + rt.slot * 8u;
          mma_half_stage_e2m1_pair<!kMx, 0>(d_tmem, a, b, v_hi, idesc, idesc2, s, s_hi, sfa, sfb, kb != 0, two, empty);
          // The next stage's barrier, tested while these MMAs run: when it has completed, as it
          // has unless the operands are late, the next stage follows without a gap.
          rt.next(ST);
          staged = kb + 1 < KB && __all_sync(0xffffffffu, mbar_test_wait_cluster(full0 + rt.slot * 8u, rt.phase));
          if (staged) tc_fence_after_sync();
          mma_half_stage_e2m1_pair<!kMx, 1>(d_tmem, a, b, v_hi, idesc, idesc2, s, s_hi, sfa, sfb, 1u, two, empty);
          if (kb == 0) got = feed.next(ctl, abort, &tn);   // behind the MMAs in the pipe
        }
        if (!ok) break;
        mma_commit_pair(smem_addr(&ctl.acc_full[acc]), 0x3);
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
      if ((!ok || got < 0) && lane == 0) atomicOr(p.status, kStatusTimeout);
    } else if (lane == 0) {
      // The peer's scales to the leader, whose MMA warp issues the copies that read them: acquired
      // in this CTA, released at cluster scope.
      const uint32_t full0 = map_to_rank(smem_addr(&ctl.full[0]), 0);
      Ring rt;
      bool ok = true;
      F4Feed feed;
      for (Tile ti; ok;) {
        const int got = feed.next<false>(ctl, abort, &ti);
        if (got <= 0) {
          ok = got == 0;
          break;
        }
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait_phase(smem_addr(&scales_in[rt.slot]), rt.phase, abort)) { ok = false; break; }
          mbar_arrive_cluster_shared(full0 + rt.slot * 8u);
          rt.next(ST);
        }
      }
      if (!ok) atomicOr(p.status, kStatusTimeout);
    }
    __syncwarp();
  } else if (warp < static_cast<int>(kF4FirstScaleWarp)) {
    // ------------------------------------------------------------ epilogue
    if (warp == 2) {
      // The producer's token maps, as in the grouped kernel, of 8, 16, ... rows.
      uint8_t *slot = p.map_slots + static_cast<size_t>(blockIdx.x) * kMapSlotBytes;
      if (total > 0 && lane < static_cast<int>(kF4TokMaps)) {
        const uint4 *src = reinterpret_cast<const uint4 *>(&p.tok_map);
        uint4 *dst = reinterpret_cast<uint4 *>(slot + lane * 128);
#pragma unroll
        for (int i = 0; i < 8; ++i) dst[i] = src[i];
        tensormap_set_dim1(dst, __ldg(p.a_offsets + p.num_groups));
        tensormap_set_box1(dst, 8u * static_cast<uint32_t>(lane + 1));
        tensormap_release();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&ctl.maps_ready));
    }
    const uint32_t quad = static_cast<uint32_t>(warp & 3);
    const uint32_t ew = static_cast<uint32_t>(warp - 2), esub = ew >> 2;
    constexpr uint32_t kSub = kF4EpiWarps / 4;   // warps per quadrant
    const uint32_t stg0 = epi_ring + ew * kF4StgBufs * kF4StgBytes;
    const uint32_t acc_empty0 = map_to_rank(smem_addr(&ctl.acc_empty[0]), 0);
    const uint32_t acc_empty1 = map_to_rank(smem_addr(&ctl.acc_empty[1]), 0);
    const float ga = p.g_a != nullptr ? __ldg(p.g_a) : 1.0f;
    const bool fused = p.epi_bias != nullptr || p.epi_row_scale != nullptr || p.epi_act != kActNone;
    uint32_t acc = 0, acc_phase = 0, buf = 0, outstanding = 0;
    F4Feed feed;
    for (Tile ti;;) {
      const int got = feed.next(ctl, abort, &ti);
      if (got < 0 && lane == 0) atomicOr(p.status, kStatusTimeout);
      if (got <= 0) break;
      const uint32_t seg = static_cast<uint32_t>(lane) & 3u, rsub = static_cast<uint32_t>(lane) >> 2;
      const uint32_t ncta = ti.n0 + rank * kBlockN + quad * 32u;   // this warp's first C column
      const uint32_t n8 = ncta + seg * 8u;
      const bool cols_ok = n8 < static_cast<uint32_t>(p.N);
      __nv_bfloat16 *crow = p.c + static_cast<size_t>(ti.row0) * p.N + n8;
      const uint32_t taddr = tmem_base + ((quad * 32u) << 16) + acc * kF4AccCols;
      const float gs = ga * (p.g_w != nullptr ? __ldg(p.g_w + ti.e) : 1.0f);
      // Operands of the fused epilogue, loaded before the accumulator wait: the bias of the
      // thread's 4 fragment columns, the row scales of this warp's chunks (lane l: row l).
      constexpr int kRowRegs = static_cast<int>(((kF4MaxTok + 31) / 32 + kSub - 1) / kSub);
      float rs[kRowRegs], bias4[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t n = ncta + 8u * i + rsub;
        bias4[i] = p.epi_bias != nullptr && n < static_cast<uint32_t>(p.N)
                       ? __bfloat162float(p.epi_bias[static_cast<size_t>(ti.e) * p.N + n])
                       : 0.0f;
      }
#pragma unroll
      for (int q = 0; q < kRowRegs; ++q) {
        const uint32_t r = (static_cast<uint32_t>(q) * kSub + esub) * 32u + static_cast<uint32_t>(lane);
        rs[q] = p.epi_row_scale != nullptr && r < ti.nrows ? __ldg(p.epi_row_scale + ti.row0 + r) : 1.0f;
      }
      int ok = 1;
      if (lane == 0) ok = wait_phase(smem_addr(&ctl.acc_full[acc]), acc_phase, abort);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) {
        if (lane == 0) atomicOr(p.status, kStatusTimeout);
        break;
      }
      tc_fence_after_sync();
      const uint32_t st_row = static_cast<uint32_t>(lane) & 7u, st_blk = static_cast<uint32_t>(lane) >> 3;
      for (uint32_t c0 = esub * 32u; c0 < ti.ntok; c0 += 32u * kSub) {
        uint32_t va[16], vb[16];
        tmem_ld_16x256b_x4(taddr + c0, va);
        tmem_ld_16x256b_x4(taddr + (16u << 16) + c0, vb);
        // The two staging buffers in turn: of the stores in flight, all but the newest must
        // have read theirs.
        const uint32_t stg = stg0 + buf * kF4StgBytes;
        if (lane == 0 && ((outstanding >> buf) & 1u)) {
          if (outstanding == 3u) bulk_wait_read<1>(); else bulk_wait_read<0>();
        }
        outstanding &= ~(1u << buf);
        tmem_ld_wait();
        __syncwarp();
#pragma unroll
        for (uint32_t g = 0; g < 4; ++g) {
          float s0 = 1.0f, s1 = 1.0f;
          if (fused) {
            s0 = __shfl_sync(0xffffffffu, rs[0], static_cast<int>(8 * g + 2 * seg));
            s1 = __shfl_sync(0xffffffffu, rs[0], static_cast<int>(8 * g + 2 * seg + 1));
          }
          uint32_t w[4];
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i) {
            const uint32_t *v = (i >> 1) ? vb : va;
            float y0 = __uint_as_float(v[4 * g + 2 * (i & 1)]) * gs;
            float y1 = __uint_as_float(v[4 * g + 2 * (i & 1) + 1]) * gs;
            if (fused) {
              y0 = epilogue_op(y0, bias4[i], p.epi_act, s0);
              y1 = epilogue_op(y1, bias4[i], p.epi_act, s1);
            }
            w[i] = pack_bf16x2(y0, y1);
          }
          const uint32_t row = 8 * g + st_row;
          stmatrix_x4_trans(stg + row * kEpiRowBytes + ((st_blk ^ ((row >> 1) & 3u)) << 4), w[0], w[1], w[2], w[3]);
        }
        if (p.c_tma && c0 + 32u <= ti.nrows && ncta < static_cast<uint32_t>(p.N)) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&p.c_map, stg, static_cast<int32_t>(ncta), static_cast<int32_t>(ti.row0 + c0));
            bulk_commit();
          }
          outstanding |= 1u << buf;
        } else {   // 16-byte stores masked to the group's rows
          __syncwarp();
          const uint8_t *stg_ptr = dyn_smem + (stg - dyn_base);
#pragma unroll
          for (uint32_t pass = 0; pass < 4; ++pass) {
            const uint32_t rl = pass * 8u + rsub, row = c0 + rl;
            const uint4 out =
                *reinterpret_cast<const uint4 *>(stg_ptr + rl * kEpiRowBytes + ((seg ^ ((rl >> 1) & 3u)) << 4));
            if (cols_ok && row < ti.nrows) *reinterpret_cast<uint4 *>(crow + static_cast<size_t>(row) * p.N) = out;
          }
        }
        buf ^= 1u;
#pragma unroll
        for (int q = 0; q + 1 < kRowRegs; ++q) rs[q] = rs[q + 1];
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(acc ? acc_empty1 : acc_empty0);
      acc ^= 1u;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (lane == 0) bulk_wait_read<0>();   // the staging buffers; the stores complete with the grid
  } else if (warp < static_cast<int>(kF4FirstScaleWarp + kF4ScaleWarps)) {
    // ------------------------------------------------------------ scales
    // Warp role 0: the CTA's 128 weight rows; 1 and 2: token rows 0 .. 127 and 128 .. 239.
    // Rows past the matrix or the group repeat the last one (their results are not stored);
    // scale bytes past K are zeroed, as the values there are.  A row is read 32 bytes (a whole
    // L2 sector, kStages stages) at a time, one chunk ahead of its use in registers, by one
    // load: two loads of 16 bytes fetch a sector twice when the line has left L1 in between
    // (prefill shapes: 0.93 ms instead of 0.71; rows an odd number of 16 bytes apart, which have
    // no other way, pay it: K = 5888 57 us, K = 5632 44 for 6231 rows, N = 1280).
    // The copies that read a stage's atoms are issued in the leader.  Its own scale warps arrive
    // on the stage's barrier; the peer's arrive on a barrier of their CTA, and its warp 1 passes
    // the news on, for a release at CTA scope does not order the atoms for a thread of the other
    // CTA.  That release is restricted to shared memory: an unrestricted one takes 0.95 us a stage
    // (prefill shapes 1.5 ms).  The same fence in the scale warps themselves holds them up
    // (0.648 ms; with the forwarder 0.627, one token's product 13.1 us for 13.0).
    constexpr uint32_t kRowStage = kF4StageK / S::kBlock;   // scale bytes per row and stage
    constexpr int kStages = static_cast<int>(32 / kRowStage);
    const int chunks = (KB + kStages - 1) / kStages;
    const uint32_t role = static_cast<uint32_t>(warp) - kF4FirstScaleWarp;
    const uint32_t written0 = smem_addr(rank == 0 ? &ctl.full[0] : &scales_in[0]);
    const int row_bytes = 4 * p.K / static_cast<int>(S::kBlock);
    const uint32_t atom0 = s_ring + static_cast<uint32_t>(lane) * 16u + (role == 0 ? 0u : (S::kWords + role - 1u) * kF4Atom);
    const uint32_t atom_step = role == 0 ? kF4Atom : 2u * kF4Atom;
    // Every chunk is one 32-byte load when the rows are that far apart and aligned.
    const bool whole = ((static_cast<uint32_t>(p.sf_pitch) | static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p.sf_a)) |
                         static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p.sf_w))) & 31u) == 0;
    bool ok = true;
    // Two copies of the loop: a choice inside it would make every load wait for its result.
    auto run = [&](auto whole_rows) {
      Ring rt;
      F4Feed feed;
      const uint8_t *src[4];   // this lane's four rows of the tile whose chunks are being loaded
      bool src_work = false;   // and whether this warp has rows of it
      int got = 1;
      uint32_t v[2][4][8];
      auto next_tile = [&]() {
        Tile x;
        got = feed.next(ctl, abort, &x);
        if (got <= 0) return;
        src_work = role < 2 || x.ntok > 128u;
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) {
          const uint32_t m = 32u * c + static_cast<uint32_t>(lane);
          if (role == 0) {
            const uint32_t n = min(x.n0 + rank * kBlockN + m, static_cast<uint32_t>(p.N) - 1u);
            src[c] = p.sf_w + (static_cast<size_t>(x.e) * p.N + n) * p.sf_pitch;
          } else {
            const uint32_t r = min((role - 1u) * 128u + m, x.nrows - 1u);
            src[c] = p.sf_a + (static_cast<size_t>(x.row0) + r) * p.sf_pitch;
          }
        }
      };
      auto load = [&](uint32_t (&x)[4][8], int chunk) {
        const int at = chunk * 32;
        if constexpr (decltype(whole_rows)::value) {
#pragma unroll
          for (int c = 0; c < 4; ++c) ld_global_nc_v8(src[c] + at, x[c]);
        } else {   // the row pitch is an odd number of 16 bytes: two loads, the second may lie past the row
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 y = __ldg(reinterpret_cast<const uint4 *>(src[c] + at));
            const uint4 z = at + 16 < p.sf_pitch ? __ldg(reinterpret_cast<const uint4 *>(src[c] + at) + 1)
                                                 : make_uint4(0u, 0u, 0u, 0u);
            x[c][0] = y.x;
            x[c][1] = y.y;
            x[c][2] = y.z;
            x[c][3] = y.w;
            x[c][4] = z.x;
            x[c][5] = z.y;
            x[c][6] = z.z;
            x[c][7] = z.w;
          }
        }
      };
      next_tile();
      if (got > 0 && src_work) load(v[0], 0);
      while (got > 0 && ok) {
        const bool work = src_work;
        bool ahead = false;   // the next tile's first chunk is on its way
        for (int c0 = 0; c0 < chunks && ok; c0 += 2) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int c = c0 + b;
            if (c + 1 < chunks) {
              if (work) load(v[b ^ 1], c + 1);
            } else if (b == 1 && c < chunks) {   // v[0] is free
              next_tile();
              if (got > 0 && src_work) load(v[0], 0);
              ahead = true;
            }
#pragma unroll
            for (int i = 0; i < kStages; ++i) {
              const int kb = c * kStages + i;
              if (kb < KB && ok) {
                if (!__all_sync(0xffffffffu, wait_phase(smem_addr(&ctl.empty[rt.slot]), rt.phase ^ 1u, abort))) {
                  ok = false;
                } else {
                  if (work) {
                    const uint32_t dst = atom0 + rt.slot * S::kBytes;
                    const int left = row_bytes - kb * static_cast<int>(kRowStage);   // scale bytes before K's end
#pragma unroll
                    for (uint32_t j = 0; j < S::kWords; ++j) {
                      const int nb = left - 4 * static_cast<int>(j);
                      const uint32_t mask = nb >= 4 ? 0xffffffffu : (nb <= 0 ? 0u : (1u << (8 * nb)) - 1u);
                      const uint32_t w = static_cast<uint32_t>(i) * S::kWords + j;
                      st_shared_v4(dst + j * atom_step, v[b][0][w] & mask, v[b][1][w] & mask, v[b][2][w] & mask,
                                   v[b][3][w] & mask);
                    }
                  }
                  fence_async_smem();   // these writes, before the tensor-memory copies read them
                  __syncwarp();
                  if (lane == 0) mbar_arrive(written0 + rt.slot * 8u);
                  rt.next(ST);
                }
              }
            }
          }
        }
        if (ok && !ahead) {
          next_tile();
          if (got > 0 && src_work) load(v[0], 0);
        }
      }
      if (got < 0) ok = false;
    };
    if (whole) run(std::true_type()); else run(std::false_type());
    if (!ok && lane == 0) atomicOr(p.status, kStatusTimeout);
  } else if (lane == 0) {
    // ------------------------------------------------------------ scheduler
    // The leader decodes the pair's tiles ahead of the roles (a search and loads of about a
    // microsecond, which in the MMA warp left the tensor cores idle at every tile) into both
    // CTAs' queues and closes them with a tile of no rows; the peer decodes the first one itself,
    // which saves it a remote write's microsecond, and tells the leader which entries its readers
    // have taken.  With many tiles a pair claims them (after its first) from a counter, so that
    // pairs which draw cheaper tiles take more; where group sizes are very uneven every second
    // pair claims from the back of the tile order, so that the small groups' weights stream while
    // the others run the large groups' arithmetic (as in the grouped kernel).
    bool ok = true;
    const bool dynamic = total >= kF4DynamicTiles * units;
    const bool two_ended = dynamic && ctl.max_group_tiles >= kUnevenRatio * ctl.min_group_tiles;
    const bool back = two_ended && (unit0 & 1u);
    uint32_t t = two_ended ? (back ? total - 1u - unit0 / 2u : unit0 / 2u) : unit0;
    Tile first{};
    if (t < total) first = decode_tile<G>(t, prefix, p);
    ctl.tq_info[0] = first;
    mbar_arrive(smem_addr(&ctl.tq_full[0]));
    if (rank == 0) {
      const uint32_t backs = two_ended ? units / 2u : 0u, fronts = units - backs;   // first tiles, not claimed
      const uint32_t info1 = map_to_rank(smem_addr(&ctl.tq_info[0]), 1), full1 = map_to_rank(smem_addr(&ctl.tq_full[0]), 1);
      for (uint32_t pos = 1; t < total; ++pos) {
        t += units;   // the static share's next
        const uint32_t slot = pos % kF4Queue, parity = (pos / kF4Queue) & 1u;
        ok = wait_phase(smem_addr(&ctl.tq_empty[slot]), parity ^ 1u, abort) &&
             (pos < kF4Queue || wait_phase_cluster(smem_addr(&peer_free[slot]), parity ^ 1u, abort));
        if (!ok) break;
        if (dynamic) {   // claimed only now: no further ahead of its use than the queue is long
          const unsigned long long old =
              atomicAdd(reinterpret_cast<unsigned long long *>(p.tile_counter), back ? (1ull << 32) : 1ull);
          const unsigned long long f = fronts + (old & 0xffffffffull), b = backs + (old >> 32);
          t = f + b >= total ? total : static_cast<uint32_t>(back ? total - 1u - b : f);
        }
        Tile x{};
        if (t < total) x = decode_tile<G>(t, prefix, p);
        ctl.tq_info[slot] = x;
        const uint32_t *xw = reinterpret_cast<const uint32_t *>(&x);
#pragma unroll
        for (uint32_t i = 0; i < sizeof(Tile) / 4; ++i)
          st_shared_cluster_u32(info1 + slot * static_cast<uint32_t>(sizeof(Tile)) + 4u * i, xw[i]);
        mbar_arrive(smem_addr(&ctl.tq_full[slot]));
        mbar_arrive_cluster(full1 + slot * 8u);
      }
    } else {
      const uint32_t free0 = map_to_rank(smem_addr(&peer_free[0]), 0);
      for (uint32_t pos = 0;; ++pos) {
        const uint32_t slot = pos % kF4Queue, parity = (pos / kF4Queue) & 1u;
        if (pos >= kF4Queue) {
          ok = wait_phase(smem_addr(&ctl.tq_empty[slot]), parity ^ 1u, abort);
          if (!ok) break;
          mbar_arrive_cluster(free0 + slot * 8u);
        }
        ok = wait_phase_cluster(smem_addr(&ctl.tq_full[slot]), parity, abort);
        if (!ok || *reinterpret_cast<volatile uint32_t *>(&ctl.tq_info[slot].nrows) == 0u) break;
      }
    }
    if (!ok) atomicOr(p.status, kStatusTimeout);
  }

  __syncthreads();
  cluster_sync();   // no CTA leaves while its peer may still signal it
  if (tid == 0) {
    // The last CTA to finish returns the tile counter to zero for the next launch.
    __threadfence();
    if (atomicAdd(p.tile_counter + 2, 1u) == gridDim.x - 1) {
      atomicExch(reinterpret_cast<unsigned long long *>(p.tile_counter), 0ull);
      atomicExch(p.tile_counter + 2, 0u);
    }
  }
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

}  // namespace gmm
