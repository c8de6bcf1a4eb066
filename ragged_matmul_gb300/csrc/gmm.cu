// Host side of the C ABI declared in include/gmm.h: handle management,
// argument validation, tensor-map encoding and the kernel launch.  No call
// here synchronises except gmm_query_status, and gmm_run / gmm_run_int4
// allocate nothing.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <new>

#include "gmm.h"
#include "gmm_host.h"
#include "gmm_kernel.cuh"
#include "gmm_fp8_block.cuh"
#include "gmm_route.cuh"
#include "gmm_fp4_quant.cuh"
#include "gmm_fp4.cuh"

namespace {

using gmm::GmmParams;
using namespace gmm::host;

// Workspace layout: a 256-byte block with the status word at byte 0, the 64-bit
// tile-claim word (front count | back count << 32) at byte 64 and the finished-CTA
// counter at byte 72 (all zero between launches), the dense call's routing at 128 and
// its usage stats at 144; then one slot of tensor maps per CTA, the zero offsets of calls
// without rows and the chunk counts of gmm_dispatch.
constexpr size_t kStatusBytes = 256;
constexpr size_t kTileCounterOffset = 64;
constexpr size_t kDenseRoutingOffset = 128;   // gmm_matmul_int4: a_offsets {0, M} and expert id 0
constexpr size_t kDenseStatsOffset = 144;     // and its usage stats (written, never read)

__global__ void gmm_clear_status_kernel(uint32_t *status, uint32_t bits) { atomicAnd(status, ~bits); }

// Token (A) map, 128-byte swizzle.  The row extent and the box height written here
// are placeholders: each CTA derives one map per box height from it and patches the
// extent to a_offsets[G].
//   2-D {K, rows}, box {64, rows}: one 64-K sub-slab per copy (any K).
//   3-D {64, rows, K / 64} (strides: a row, then 128 bytes to the next 64 of K), box
//   {64, rows, sub}: `sub` sub-slabs of a stage in one copy, landing one after the
//   other in shared memory.  Only when K is a multiple of 64 (the 4-bit path).
int encode_token_maps(gmm_ctx *h, GmmParams &p, const void *a, int K, int sub_per_copy) {
  if (sub_per_copy == 1) {
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), 256};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(K) * 2};
    cuuint32_t box[2] = {gmm::kBK, 128};
    return encode_map(h, &p.tok_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a, dims, strides, box,
                      CU_TENSOR_MAP_SWIZZLE_128B);
  }
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(gmm::kBK), 256, static_cast<cuuint64_t>(K / gmm::kBK)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(K) * 2, static_cast<cuuint64_t>(gmm::kBK) * 2};
  cuuint32_t box[3] = {gmm::kBK, 128, static_cast<cuuint32_t>(sub_per_copy)};
  return encode_map(h, &p.tok_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a, dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_128B);
}

// The optional epilogue: a known activation, and operands aligned for their element type.
int check_epilogue(const gmm_epilogue *e) {
  if (!e) return GMM_OK;
  if (e->activation < GMM_ACT_NONE || e->activation > GMM_ACT_GELU_TANH) return GMM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(e->bias) & 1u) || (reinterpret_cast<uintptr_t>(e->row_scale) & 3u))
    return GMM_ERR_INVALID_ARG;
  return GMM_OK;
}

void set_epilogue(GmmParams &p, const gmm_epilogue *e) {
  static_assert(GMM_ACT_NONE == gmm::kActNone && GMM_ACT_RELU == gmm::kActRelu && GMM_ACT_SILU == gmm::kActSilu &&
                    GMM_ACT_GELU_TANH == gmm::kActGeluTanh,
                "activation codes of the C ABI and the kernel agree");
  p.epi_bias = e ? static_cast<const __nv_bfloat16 *>(e->bias) : nullptr;
  p.epi_row_scale = e ? e->row_scale : nullptr;
  p.epi_act = e ? e->activation : GMM_ACT_NONE;
}

// A call without rows: c and a both NULL, as an empty tensor's pointer is.  Its groups are empty
// whatever a_offsets holds (it gets offsets of zero), so what now stands for c and a is neither
// read nor written.
bool take_no_rows(gmm_ctx *h, void **c, const void **a, const uint32_t **a_offsets) {
  if (!h || *c || *a || !*a_offsets) return false;
  *c = h->ws;
  *a = h->ws;
  *a_offsets = h->zero_offsets;
  return true;
}

int check_common(gmm_ctx *h, void *c, const void *a, const uint32_t *a_offsets, const int32_t *ids,
                 uint32_t *stats, int G, int N, int K) {
  if (!h || !c || !a || !a_offsets || !stats) return GMM_ERR_INVALID_ARG;
  if (!ids && G > 0) return GMM_ERR_INVALID_ARG;   // never read when there are no groups
  if (G < 0 || N < 8 || K < 8 || (N % 8) || (K % 8)) return GMM_ERR_INVALID_ARG;
  if (N > (1 << 24) || K > (1 << 24)) return GMM_ERR_UNSUPPORTED;
  if (G > gmm::kMaxGroups) return GMM_ERR_UNSUPPORTED;
  if (!aligned16(c) || !aligned16(a)) return GMM_ERR_INVALID_ARG;
  return GMM_OK;
}

// Token blocks per band of the tile order: as many 256-row blocks of A as fit in
// about 40 MB, a third of the GB300's L2, so a band's activations stay resident.
constexpr double kBandBytes = 40e6;

void fill_common(gmm_ctx *h, GmmParams &p, void *c, const uint32_t *a_offsets, const int32_t *ids,
                 uint32_t *stats, int G, int N, int K, uint32_t max_tok) {
  p.c = static_cast<__nv_bfloat16 *>(c);
  p.a_offsets = a_offsets;
  p.expert_ids = ids;
  p.stats = stats;
  p.status = reinterpret_cast<uint32_t *>(h->ws);
  p.tile_counter = reinterpret_cast<uint32_t *>(h->ws + kTileCounterOffset);
  p.map_slots = h->ws + kStatusBytes;
  p.num_groups = G;
  p.num_experts = h->num_experts;
  p.N = N;
  p.K = K;
  // C as a TMA store target: {N, 2^31} rows (the real row count is on the device; the
  // kernel only stores whole 32-row chunks inside a group through it), box 32 x 32,
  // 64-byte swizzle (the epilogue staging layout).  Without it every chunk takes the
  // 16-byte store path.
  p.c_tma = 0;
  if (h->encode != nullptr && aligned16(c)) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), 1ull << 31};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(N) * 2u};
    const cuuint32_t box[2] = {32, 32}, estr[2] = {1, 1};
    p.c_tma = with_context(h, [&] {
                return h->encode(&p.c_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c, dims, strides, box, estr,
                                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                                 CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
              }) == CUDA_SUCCESS;
  }
  if (const char *env = getenv("GMM_TMA_STORE")) p.c_tma = p.c_tma && atoi(env) != 0;   // tuning override
  const double block_bytes = static_cast<double>(max_tok) * K * 2.0;
  const double band = kBandBytes / block_bytes;
  p.tok_band = band < 1.0 ? 1 : (band > 1e6 ? 1000000 : static_cast<int>(band));
  if (const char *env = getenv("GMM_TOK_BAND")) {   // tuning override
    const int v = atoi(env);
    if (v > 0) p.tok_band = v;
  }
  p.cache_hints = 1;
  if (const char *env = getenv("GMM_CACHE_HINTS")) p.cache_hints = atoi(env) != 0;   // tuning override
  // Test hooks of the device-timeout path (off unless set): GMM_TEST_WAIT_LIMIT_NS
  // shortens every pipeline wait, GMM_TEST_STALL_STAGE makes the one-CTA bf16 kernel's
  // producer skip that stage, so that the kernel gives up and reports a timeout.
  p.wait_limit_ns = 0;
  p.test_stall_stage = -1;
  if (const char *env = getenv("GMM_TEST_WAIT_LIMIT_NS")) p.wait_limit_ns = strtoull(env, nullptr, 10);
  if (const char *env = getenv("GMM_TEST_STALL_STAGE")) p.test_stall_stage = atoi(env);
}

// Stage-ring depth of a grouped-kernel launch with G groups in a layout: what the budget
// holds after the layout's fixed parts and the prefix, capped at kMaxStages, a multiple
// of stage_mult.
int stages_for(const gmm_variant &v, int G, int layout) {
  const size_t prefix = (static_cast<size_t>(G + 1) * 4 + 15) & ~static_cast<size_t>(15);
  const size_t fixed = v.fixed[layout];
  if (v.budget < fixed + prefix) return 0;
  long st = static_cast<long>((v.budget - fixed - prefix) / v.stage_bytes);
  if (st > gmm::kMaxStages) st = gmm::kMaxStages;
  st -= st % v.stage_mult;
  return static_cast<int>(st);
}

// Ring depths from the shared-memory budget (the pages' launchers likewise derive their
// pipeline depth from the shared memory available, and the quantised GEMM's launcher
// reduces stages or warp partitions when the budget is exceeded): as many stages as fit,
// and for the 4-bit kernel, if even its minimum ring does not fit with the full packed
// ring, a packed ring of half the slots.  The grid: one CTA per SM, or for pairs twice
// the number of clusters of two that fit at once.  `optin` is the budget (the device's
// opt-in shared memory per block, or less when capped for testing), `sm_smem` the SM's
// shared memory: a launch always reserves more than half of it, so one CTA runs per SM.
template <bool kInt4, bool kPair, bool kFp8 = false>
int configure(gmm_variant *v, int optin, int sm_smem, int device_optin, int num_sms) {
  using G = gmm::Geom<kInt4, kPair>;
  auto kernel = gmm::gmm_grouped_kernel<kInt4, kPair, kFp8>;
  cudaFuncAttributes attr;
  if (cudaFuncGetAttributes(&attr, reinterpret_cast<const void *>(kernel)) != cudaSuccess) return GMM_ERR_CUDA;
  const long avail = static_cast<long>(optin) - static_cast<long>(attr.sharedSizeBytes);
  if (avail <= 0) return GMM_ERR_UNSUPPORTED;
  v->budget = static_cast<size_t>(avail);
  v->stage_bytes = G::kStageBytes;
  v->stage_mult = kInt4 ? static_cast<int>(gmm::kAStages) : 1;
  // Candidate layouts.  4-bit, in order of preference: the full packed ring, then half
  // of it.  The variant is usable when at least one layout fits beside a one-group
  // prefix; a launch whose groups' prefix leaves no layout its minimum ring returns
  // GMM_ERR_UNSUPPORTED.
  v->min_stages = kInt4 ? static_cast<int>(gmm::kAStages) : 2;
  v->layouts = kInt4 ? 2 : 1;
  for (int c = 0; c < v->layouts; ++c) {
    v->q_stages[c] = kInt4 ? (c == 0 ? gmm::kQStages : 2) : 0;
    v->fixed[c] = 1024 + gmm::kEpiBytes<kInt4> + static_cast<size_t>(v->q_stages[c]) * gmm::kQSlotBytes;
  }
  v->stages = 0;
  for (int c = 0; c < v->layouts && v->stages < v->min_stages; ++c) v->stages = stages_for(*v, 1, c);
  if (v->stages < v->min_stages) return GMM_ERR_UNSUPPORTED;
  const long reserve = static_cast<long>(sm_smem) / 2 + 1024;   // more than half an SM: one CTA per SM
  const long cap = static_cast<long>(device_optin) - static_cast<long>(attr.sharedSizeBytes);
  v->smem = static_cast<size_t>(std::min(cap, std::max(avail, reserve)));
  if (cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(v->smem)) != cudaSuccess)
    return GMM_ERR_CUDA;
  v->grid = num_sms;
  if (kPair) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute la[1];
    la[0].id = cudaLaunchAttributeClusterDimension;
    la[0].val.clusterDim.x = 2;
    la[0].val.clusterDim.y = 1;
    la[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms & ~1));
    cfg.blockDim = dim3(kInt4 ? gmm::kInt4Threads : gmm::kThreadsWide);   // the larger launch
    cfg.dynamicSmemBytes = v->smem;
    cfg.attrs = la;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess || clusters < 1)
      return GMM_ERR_CUDA;
    v->grid = 2 * clusters < (num_sms & ~1) ? 2 * clusters : (num_sms & ~1);
  }
  return GMM_OK;
}

// The per-K-block e4m3 kernel: as many stages as fit beside the group prefix (sized at
// each launch, as for the grouped kernel), one CTA per SM.
int configure_fp8_block(gmm_variant *v, int optin, int sm_smem, int device_optin, int num_sms) {
  using G = gmm::BwGeom;
  auto kernel = gmm::gmm_fp8_block_kernel;
  cudaFuncAttributes attr;
  if (cudaFuncGetAttributes(&attr, reinterpret_cast<const void *>(kernel)) != cudaSuccess) return GMM_ERR_CUDA;
  // The kernel moves registers from its first warpgroup to the promotion warpgroups
  // (setmaxnreg).  The increase waits until the CTA's pool, the launch's registers a
  // thread times its threads, covers it, so a build whose register count left the pool
  // short would never finish: refuse it here instead.
  if (static_cast<long>(attr.numRegs) * gmm::kBwThreads <
      128L * gmm::kBwRegsLow + 32L * gmm::kBwPromoWarps * gmm::kBwRegsHigh)
    return GMM_ERR_UNSUPPORTED;
  const long avail = static_cast<long>(optin) - static_cast<long>(attr.sharedSizeBytes);
  if (avail <= 0) return GMM_ERR_UNSUPPORTED;
  v->budget = static_cast<size_t>(avail);
  v->stage_bytes = G::kStageBytes;
  v->stage_mult = 1;
  v->min_stages = 2;
  v->layouts = 1;
  v->q_stages[0] = 0;
  v->fixed[0] = static_cast<size_t>(gmm::kBwFixedBytes);
  v->stages = stages_for(*v, 1, 0);
  if (v->stages < v->min_stages) return GMM_ERR_UNSUPPORTED;
  const long reserve = static_cast<long>(sm_smem) / 2 + 1024;   // more than half an SM: one CTA per SM
  const long cap = static_cast<long>(device_optin) - static_cast<long>(attr.sharedSizeBytes);
  v->smem = static_cast<size_t>(std::min(cap, std::max(avail, reserve)));
  if (cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(v->smem)) != cudaSuccess)
    return GMM_ERR_CUDA;
  v->grid = num_sms;
  return GMM_OK;
}

int launch_fp8_block(gmm_ctx *h, GmmParams &p, cudaStream_t stream) {
  DeviceGuard guard(h->device);
  const gmm_variant &v = h->var_fp8_block;
  p.num_stages = stages_for(v, p.num_groups, 0);
  if (p.num_stages < v.min_stages) return GMM_ERR_UNSUPPORTED;   // the prefix leaves no room for the ring
  if (h->debug)
    fprintf(stderr, "gmm: launch e4m3 block, %d groups: stages %d packed slots 0\n", p.num_groups, p.num_stages);
  gmm::gmm_fp8_block_kernel<<<v.grid, gmm::kBwThreads, v.smem, stream>>>(p);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) {
    debug_report("launch of the block-scaled kernel", static_cast<int>(err), cudaGetErrorString(err));
    return GMM_ERR_CUDA;
  }
  return GMM_OK;
}

// The 4-bit floating point kernel: as many stages as fit, two CTAs per tile.  A device or
// budget that cannot run it leaves grid 0 (gmm_run_fp4 then returns GMM_ERR_UNSUPPORTED).
template <bool kMx>
void configure_fp4(gmm_variant *v, int optin, int sm_smem, int device_optin, int num_sms) {
  auto kernel = gmm::gmm_fp4_kernel<kMx>;
  v->grid = 0;
  cudaFuncAttributes attr;
  if (cudaFuncGetAttributes(&attr, reinterpret_cast<const void *>(kernel)) != cudaSuccess) return;
  const long avail = static_cast<long>(optin) - static_cast<long>(attr.sharedSizeBytes);
  if (avail <= 0 || num_sms < 2) return;
  v->budget = static_cast<size_t>(avail);
  v->stage_bytes = gmm::F4Geom<kMx>::kStageBytes;
  v->fixed[0] = gmm::kF4FixedBytes;
  v->stages = stages_for(*v, 1, 0);
  if (v->stages < v->min_stages) return;
  const long reserve = static_cast<long>(sm_smem) / 2 + 1024;   // more than half an SM: one CTA per SM
  const long cap = static_cast<long>(device_optin) - static_cast<long>(attr.sharedSizeBytes);
  v->smem = static_cast<size_t>(std::min(cap, std::max(avail, reserve)));
  if (cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(v->smem)) != cudaSuccess)
    return;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeClusterDimension;
  la[0].val.clusterDim.x = 2;
  la[0].val.clusterDim.y = 1;
  la[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(num_sms & ~1));
  cfg.blockDim = dim3(gmm::kF4Threads);
  cfg.dynamicSmemBytes = v->smem;
  cfg.attrs = la;
  cfg.numAttrs = 1;
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess || clusters < 1) return;
  v->grid = std::min(2 * clusters, num_sms & ~1);
}

template <bool kMx>
int launch_fp4(gmm_ctx *h, gmm::F4Params &p, cudaStream_t stream) {
  DeviceGuard guard(h->device);
  const gmm_variant &v = h->var_fp4[kMx];
  if (v.grid == 0) return GMM_ERR_UNSUPPORTED;
  p.num_stages = stages_for(v, p.num_groups, 0);
  if (p.num_stages < v.min_stages) return GMM_ERR_UNSUPPORTED;   // the prefix leaves no room for the ring
  if (h->debug)
    fprintf(stderr, "gmm: launch %s pair, %d groups: stages %d packed slots 0\n", kMx ? "mxfp4" : "nvfp4", p.num_groups,
            p.num_stages);
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(v.grid));
  cfg.blockDim = dim3(gmm::kF4Threads);
  cfg.dynamicSmemBytes = v.smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, gmm::gmm_fp4_kernel<kMx>, p);
  if (err != cudaSuccess) {
    debug_report("launch of the 4-bit floating point kernel", static_cast<int>(err), cudaGetErrorString(err));
    cudaGetLastError();
    return GMM_ERR_CUDA;
  }
  return GMM_OK;
}

template <bool kInt4, bool kFp8 = false>
int launch(gmm_ctx *h, GmmParams &p, cudaStream_t stream) {
  DeviceGuard guard(h->device);
  const int pairs = kInt4 ? h->use_pairs_int4 : h->use_pairs;
  const gmm_variant &v = kFp8 ? h->var_fp8[pairs] : h->var[kInt4][pairs];
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[1];
  // Short K: 12 epilogue warps (the bf16 / e4m3 kernel reads its warp count from blockDim).
  cfg.blockDim = dim3(kInt4 ? gmm::kInt4Threads : (p.K <= gmm::kWideEpilogueMaxK ? gmm::kThreadsWide : gmm::kThreads));
  cfg.gridDim = dim3(static_cast<unsigned>(v.grid));
  cfg.dynamicSmemBytes = v.smem;
  cfg.stream = stream;
  int layout = 0;
  p.num_stages = 0;
  for (; layout < v.layouts; ++layout)
    if ((p.num_stages = stages_for(v, p.num_groups, layout)) >= v.min_stages) break;
  if (layout == v.layouts) return GMM_ERR_UNSUPPORTED;   // no layout's minimum ring fits beside this prefix
  p.q_stages = v.q_stages[layout];
  if (h->debug)
    fprintf(stderr, "gmm: launch %s%s, %d groups: stages %d packed slots %d\n", kInt4 ? "int4" : (kFp8 ? "e4m3" : "bf16"),
            pairs ? " pair" : "", p.num_groups, p.num_stages, p.q_stages);
  cudaError_t err;
  if (pairs) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, gmm::gmm_grouped_kernel<kInt4, true, kFp8>, p);
  } else {
    err = cudaLaunchKernelEx(&cfg, gmm::gmm_grouped_kernel<kInt4, false, kFp8>, p);
  }
  if (err != cudaSuccess) {
    debug_report("launch of the grouped kernel", static_cast<int>(err), cudaGetErrorString(err));
    cudaGetLastError();
    return GMM_ERR_CUDA;
  }
  return GMM_OK;
}

// Dynamic shared memory of the dispatch kernels.
size_t small_dispatch_smem(int E, int slots) {
  return (static_cast<size_t>(gmm::kRouteWarps) * E + E + 1 + slots) * 4;
}
constexpr size_t kCountSmem = 96 * 1024;   // gmm_dispatch_count_kernel's counters, at most

int configure_route() {
  const int small = static_cast<int>(small_dispatch_smem(gmm::kRouteSmallExperts, gmm::kRouteSmallSlots));
  const void *kernels[6] = {reinterpret_cast<const void *>(gmm::gmm_dispatch_small_kernel<16, true>),
                            reinterpret_cast<const void *>(gmm::gmm_dispatch_small_kernel<4, true>),
                            reinterpret_cast<const void *>(gmm::gmm_dispatch_small_kernel<2, true>),
                            reinterpret_cast<const void *>(gmm::gmm_dispatch_small_kernel<16, false>),
                            reinterpret_cast<const void *>(gmm::gmm_dispatch_small_kernel<4, false>),
                            reinterpret_cast<const void *>(gmm::gmm_dispatch_small_kernel<2, false>)};
  for (const void *k : kernels)
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, small) != cudaSuccess) return GMM_ERR_CUDA;
  if (cudaFuncSetAttribute(reinterpret_cast<const void *>(gmm::gmm_dispatch_count_kernel),
                           cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kCountSmem)) != cudaSuccess)
    return GMM_ERR_CUDA;
  return GMM_OK;
}

// Argument checks shared by the calls that move rows of tokens.
int check_rows(gmm_ctx *h, int num_tokens, int top_k, int width, int dtype, long long stride) {
  if (!h || num_tokens < 0 || top_k < 1 || width < 1 || !dtype_bytes(dtype)) return GMM_ERR_INVALID_ARG;
  if (stride < 0) return GMM_ERR_INVALID_ARG;
  if (top_k > gmm::kRouteMaxTopK || static_cast<long long>(num_tokens) * top_k > (1ll << 30)) return GMM_ERR_UNSUPPORTED;
  if (width > gmm::kRouteMaxWidth) return GMM_ERR_UNSUPPORTED;
  return GMM_OK;
}

template <int VB>
int launch_dispatch(gmm_ctx *h, gmm::DispatchParams &p, cudaStream_t stream) {
  const int E = p.num_experts, S = p.num_tokens * p.top_k;
  if (S <= gmm::kRouteSmallSlots && E <= gmm::kRouteSmallExperts) {
    // Small units while they leave warps without one; else larger ones, and CTAs beside one
    // another on an SM (each sorts again, which costs them no more time than it costs one):
    // 4096 tokens of 8 KB, top-1, 18 us instead of 27.
    const long long nvec = p.tokens ? p.row_bytes / VB : 0;
    constexpr int kFew = 32 * gmm::kRouteUnit<VB, true>, kMany = 32 * gmm::kRouteUnit<VB, false>;
    const long long few = p.num_tokens * ((nvec + kFew - 1) / kFew), many = p.num_tokens * ((nvec + kMany - 1) / kMany);
    const size_t smem = small_dispatch_smem(E, S);
    if (few <= 2ll * gmm::kRouteWarps * h->num_sms) {
      const long long want = (few + gmm::kRouteWarps - 1) / gmm::kRouteWarps;
      const int grid = static_cast<int>(std::max(1ll, std::min<long long>(want, h->num_sms)));
      gmm::gmm_dispatch_small_kernel<VB, true><<<grid, gmm::kRouteThreads, smem, stream>>>(p);
    } else {
      const long long want = (many + gmm::kRouteWarps - 1) / gmm::kRouteWarps;
      const int grid = static_cast<int>(std::min<long long>(want, 3ll * h->num_sms));
      gmm::gmm_dispatch_small_kernel<VB, false><<<grid, gmm::kRouteThreads, smem, stream>>>(p);
    }
    return launch_status("launch of the dispatch kernel");
  }
  // Chunks: the count's time falls with their number (slots / chunks a CTA), the sum of their
  // counts, which every copying CTA makes, rises with it (chunks x E).  32768 slots: 128 experts
  // 58.4 us with 64 chunks, 61.4 with 152; 8 experts 68.2 with 152 chunks, 71.6 with 128.
  int chunks = std::min(gmm::kRouteMaxChunks, std::max(1, gmm::kRouteMaxCounts / E));
  chunks = std::min(chunks, std::max(1, static_cast<int>(4.0 * std::sqrt(static_cast<double>(S) / E))));
  chunks = std::min(chunks, p.num_tokens);
  p.chunk_tokens = (p.num_tokens + chunks - 1) / chunks;
  p.chunks = (p.num_tokens + p.chunk_tokens - 1) / p.chunk_tokens;
  p.subs = std::max(1, std::min(4 * h->num_sms / p.chunks, p.chunk_tokens));
  const int warps = static_cast<int>(std::min<size_t>(gmm::kRouteWarps, kCountSmem / (4u * static_cast<unsigned>(E))));
  gmm::gmm_dispatch_count_kernel<<<p.chunks, gmm::kRouteThreads, static_cast<size_t>(warps) * E * 4, stream>>>(p, warps);
  const int rc = launch_status("launch of the count kernel");
  if (rc) return rc;
  const size_t smem = (2 * static_cast<size_t>(E) + 1 + static_cast<size_t>(gmm::kRouteBatch) * p.top_k) * 4;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.chunks * p.subs));
  cfg.blockDim = dim3(gmm::kRouteThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, gmm::gmm_dispatch_place_kernel<VB>, p);
  return launch_status("launch of the place kernel");
}

template <class T, int VN, int kRows, int kUnits>
void launch_grad(gmm_ctx *h, gmm::CombineParams &p, long long nvec, cudaStream_t stream) {
  // One warp a token when that fills the SMs (32 resident warps each; 24 for single elements,
  // whose pieces are shorter: 1003 tokens of 1411 fp32, top-6, 15.2 us with four warps a token,
  // 0.5 more with eight), else more.
  constexpr long long kFill = VN == 1 ? 24 : 32;
  const long long pieces = (nvec + 32 * kUnits - 1) / (32 * kUnits);
  int wpt = 1;
  while (wpt < gmm::kCombineWarps && wpt < pieces && p.num_tokens * static_cast<long long>(wpt) < kFill * h->num_sms) wpt *= 2;
  p.warps_per_token = wpt;
  const int tpc = gmm::kCombineWarps / wpt;
  gmm::gmm_combine_grad_kernel<T, VN, kRows, kUnits>
      <<<static_cast<unsigned>((p.num_tokens + tpc - 1) / tpc), 32 * gmm::kCombineWarps, 0, stream>>>(p);
}

template <class T, int VN, int kBatch, int kSeq, int kUnits>
int launch_sum(gmm::CombineParams &p, long long nvec, cudaStream_t stream) {
  const long long pieces = (nvec + 32 * kSeq * kUnits - 1) / (32 * kSeq * kUnits);
  const long long ctas = (p.num_tokens * pieces + gmm::kCombineWarps - 1) / gmm::kCombineWarps;
  if (ctas > (1ll << 28)) return GMM_ERR_UNSUPPORTED;   // warps are numbered in 32 bits
  gmm::gmm_combine_kernel<T, VN, kBatch, kSeq, kUnits>
      <<<static_cast<unsigned>(ctas), 32 * gmm::kCombineWarps, 0, stream>>>(p);
  return launch_status("launch of the combine kernel");
}

template <class T, int VN>
int launch_combine(gmm_ctx *h, gmm::CombineParams &p, bool grad, cudaStream_t stream) {
  const long long nvec = p.row_bytes / static_cast<long long>(sizeof(T) * VN);
  if (grad) {
    // Rows at a time by top_k, so that few of the unrolled rows are idle, and as many vectors of each
    // as the registers hold; of single elements more, for as many bytes.  3, 5 and 6 rows (1500,
    // 1000, 1000 tokens of 2047 bf16): 15.5, 14.0 and 16.7 us, with code for four rows 19.3, 19.3
    // and 20.0.  In vectors top-5 and top-6 take three rows twice where there are few tokens (1000 of
    // 2048 bf16, top-6: 11.1 us, 13.3 with eight), else all at once, for d_out is then read once
    // (4096 of 2048 fp32: 69.5 us, 73.4 three by three).
    if constexpr (VN == 1) {
      if (p.top_k == 1) launch_grad<T, VN, 1, 8>(h, p, nvec, stream);
      else if (p.top_k == 2) launch_grad<T, VN, 2, 8>(h, p, nvec, stream);
      else if (p.top_k == 3) launch_grad<T, VN, 3, 4>(h, p, nvec, stream);
      else if (p.top_k == 5 || p.top_k == 6) launch_grad<T, VN, 6, 2>(h, p, nvec, stream);
      else launch_grad<T, VN, 4, 3>(h, p, nvec, stream);
    } else {
      const bool few = p.num_tokens < 16ll * h->num_sms;
      if (p.top_k == 1) launch_grad<T, VN, 1, 4>(h, p, nvec, stream);
      else if (p.top_k == 2) launch_grad<T, VN, 2, 2>(h, p, nvec, stream);
      else if (p.top_k == 3 || (few && (p.top_k == 5 || p.top_k == 6))) launch_grad<T, VN, 3, 2>(h, p, nvec, stream);
      else if (p.top_k == 4) launch_grad<T, VN, 4, 1>(h, p, nvec, stream);
      else launch_grad<T, VN, 8, 1>(h, p, nvec, stream);
    }
    return launch_status("launch of the combine gradient kernel");
  }
  // As for the gradient; single elements in larger units, for as many bytes.  4096 tokens of 2048
  // bf16, top-8: four rows of two vectors 25.7 us, eight of one 26.6; of 2047: 36.0 and 41.0.
  // 1500 tokens, top-3: 4.2 and 6.2 us with code for three rows, 5.8 and 10.5 for eight.
  constexpr int kUnits = VN == 1 ? 8 : 2;
  if (p.top_k <= 2) return launch_sum<T, VN, 2, (VN == 1 ? 1 : 2), (VN == 1 ? 16 : 2)>(p, nvec, stream);
  if (p.top_k == 3 || p.top_k == 5 || p.top_k == 6) return launch_sum<T, VN, 3, 1, kUnits>(p, nvec, stream);
  return launch_sum<T, VN, 4, 1, kUnits>(p, nvec, stream);
}

// 16-byte vectors where every row starts on a 16-byte boundary, else single elements.
int run_combine(gmm_ctx *h, gmm::CombineParams &p, int dtype, bool vec, bool grad, cudaStream_t stream) {
  DeviceGuard guard(h->device);
  switch (dtype) {
    case GMM_DTYPE_BF16:
      return vec ? launch_combine<__nv_bfloat16, 8>(h, p, grad, stream) : launch_combine<__nv_bfloat16, 1>(h, p, grad, stream);
    case GMM_DTYPE_FP16:
      return vec ? launch_combine<__half, 8>(h, p, grad, stream) : launch_combine<__half, 1>(h, p, grad, stream);
    default:
      return vec ? launch_combine<float, 4>(h, p, grad, stream) : launch_combine<float, 1>(h, p, grad, stream);
  }
}

template <class T, bool kMx, int kAlign>
void launch_quant(const gmm::QuantParams &p, bool quantise, unsigned grid, cudaStream_t stream) {
  if (quantise) gmm::gmm_quantize_fp4_kernel<T, kMx, kAlign><<<grid, gmm::kQuantThreads, 0, stream>>>(p);
  else gmm::gmm_dequantize_fp4_kernel<T, kMx, kAlign><<<grid, gmm::kQuantThreads, 0, stream>>>(p);
}

template <class T, bool kMx>
void launch_quant_align(const gmm::QuantParams &p, bool quantise, int align, unsigned grid, cudaStream_t stream) {
  if (align == 32) launch_quant<T, kMx, 32>(p, quantise, grid, stream);
  else if (align == 16) launch_quant<T, kMx, 16>(p, quantise, grid, stream);
  else launch_quant<T, kMx, 1>(p, quantise, grid, stream);
}

template <class T>
void launch_quant_fmt(const gmm::QuantParams &p, int format, bool quantise, int align, unsigned grid, cudaStream_t stream) {
  if (format == GMM_FP4_MX) launch_quant_align<T, true>(p, quantise, align, grid, stream);
  else launch_quant_align<T, false>(p, quantise, align, grid, stream);
}

int fp4_block(int format) { return format == GMM_FP4_MX ? 32 : 16; }
int fp4_scale_pitch(int K, int format) { return (K / fp4_block(format) + 15) / 16 * 16; }

int run_quant(gmm_ctx *h, gmm::QuantParams &p, int dtype, int format, long long stride, bool quantise, cudaStream_t stream) {
  if (!h || !dtype_bytes(dtype) || (format != GMM_FP4_NV && format != GMM_FP4_MX)) return GMM_ERR_INVALID_ARG;
  if (p.rows < 0 || p.K < 32 || p.K % 32 || stride < 0) return GMM_ERR_INVALID_ARG;
  if (p.K > (1 << 24)) return GMM_ERR_UNSUPPORTED;
  if (p.rows == 0) return GMM_OK;
  const int es = dtype_bytes(dtype);
  if (!p.x || !p.packed || !p.scales || !aligned_to(p.x, es) || !aligned16(p.packed) || !aligned16(p.scales) ||
      !aligned_to(p.global_scale, 4) || !aligned_to(p.row_slots, 4) || (format == GMM_FP4_MX && p.global_scale))
    return GMM_ERR_INVALID_ARG;
  if (!quantise && stride < p.K && p.rows > 1) return GMM_ERR_INVALID_ARG;   // rows of the output overlap
  p.x_pitch = stride * es;
  p.scale_pitch = fp4_scale_pitch(p.K, format);
  p.status = reinterpret_cast<uint32_t *>(h->ws);
  const unsigned long long at = reinterpret_cast<uintptr_t>(p.x) | static_cast<unsigned long long>(p.x_pitch);
  const int align = at % 32 == 0 ? 32 : (at % 16 == 0 ? 16 : 1);
  // Blocks of 16 elements are numbered in 31 bits (block / blocks a row is then a multiply and
  // a shift: for block < 2^31 and m = floor(2^(31 + l) / d) + 1 with 2^l >= d, block * m >> (31 + l));
  // longer calls go in slabs of rows.
  const unsigned d = static_cast<unsigned>(p.K / 16);
  unsigned l = 0;
  while ((1ull << l) < d) ++l;
  p.div_mul = static_cast<uint32_t>((1ull << (31 + l)) / d + 1);
  p.div_shift = l - 1;   // K >= 32: d >= 2
  const int per_cta = gmm::kQuantThreads * (quantise ? gmm::kQuantPer : gmm::kDequantPer);
  const int slab = static_cast<int>(((1ll << 31) - per_cta) / d);
  DeviceGuard guard(h->device);
  const int rows = p.rows;
  for (int row0 = 0; row0 < rows; row0 += std::min(slab, rows - row0)) {
    p.row0 = row0;
    p.rows = std::min(slab, rows - row0);
    const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.rows) * d + per_cta - 1) / per_cta);
    switch (dtype) {
      case GMM_DTYPE_BF16: launch_quant_fmt<__nv_bfloat16>(p, format, quantise, align, grid, stream); break;
      case GMM_DTYPE_FP16: launch_quant_fmt<__half>(p, format, quantise, align, grid, stream); break;
      default: launch_quant_fmt<float>(p, format, quantise, align, grid, stream); break;
    }
    const int rc = launch_status(quantise ? "launch of the quantisation kernel" : "launch of the dequantisation kernel");
    if (rc) return rc;
  }
  return GMM_OK;
}

uint32_t max_tok(const gmm_ctx *h, bool int4) {
  if (int4) return h->use_pairs_int4 ? gmm::Geom<true, true>::kMaxTok : gmm::Geom<true, false>::kMaxTok;
  return h->use_pairs ? gmm::Geom<false, true>::kMaxTok : gmm::Geom<false, false>::kMaxTok;
}

}  // namespace

extern "C" {

const char *gmm_error_string(int code) {
  switch (code) {
    case GMM_OK: return "success";
    case GMM_ERR_INVALID_ARG: return "invalid argument";
    case GMM_ERR_UNSUPPORTED: return "unsupported shape or option";
    case GMM_ERR_CUDA: return "CUDA runtime or driver call failed";
    case GMM_ERR_DEVICE_TIMEOUT: return "kernel pipeline wait timed out";
    case GMM_ERR_BAD_INPUT: return "decreasing a_offsets or expert id out of range, or a slot or row index out of range";
    case GMM_ERR_NO_DEVICE: return "no sm_103 device";
    default: return "unknown error code";
  }
}

int gmm_create(gmm_handle_t *out, int num_experts, int device) {
  if (!out) return GMM_ERR_INVALID_ARG;
  *out = nullptr;
  if (num_experts < 1) return GMM_ERR_INVALID_ARG;
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess || device < 0 || device >= ndev) {
    cudaGetLastError();
    return GMM_ERR_NO_DEVICE;
  }
  int major = 0, minor = 0, sms = 0, optin = 0, sm_smem = 0;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, device);
  cudaDeviceGetAttribute(&sm_smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor, device);
  if (major != 10 || minor != 3 || sms < 1) return GMM_ERR_NO_DEVICE;
  const int device_optin = optin;
  // Test override GMM_SMEM_BUDGET (bytes): size the rings as if a block could opt in to
  // no more shared memory than this, which exercises the reduced configurations.
  if (const char *env = getenv("GMM_SMEM_BUDGET")) {
    const int cap = atoi(env);
    if (cap > 0 && cap < optin) optin = cap;
  }

  gmm_ctx *h = new (std::nothrow) gmm_ctx;
  if (!h) return GMM_ERR_CUDA;
  h->device = device;
  h->num_experts = num_experts;
  h->num_sms = sms;

  DeviceGuard guard(device);
  void *fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
          cudaSuccess ||
      q != cudaDriverEntryPointSuccess || !fn) {
    cudaGetLastError();
    delete h;
    return GMM_ERR_CUDA;
  }
  h->encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  fn = nullptr;
  if (cudaGetDriverEntryPointByVersion("cuMemsetD32Async", &fn, 3020, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess || !fn) {
    cudaGetLastError();
    delete h;
    return GMM_ERR_CUDA;
  }
  h->memset32 = reinterpret_cast<PFN_cuMemsetD32Async_v3020>(fn);

  h->smem_per_sm = sm_smem;
  const int single_ok = configure<false, false>(&h->var[0][0], optin, sm_smem, device_optin, sms) == GMM_OK &&
                        configure<true, false>(&h->var[1][0], optin, sm_smem, device_optin, sms) == GMM_OK &&
                        configure<false, false, true>(&h->var_fp8[0], optin, sm_smem, device_optin, sms) == GMM_OK &&
                        configure_fp8_block(&h->var_fp8_block, optin, sm_smem, device_optin, sms) == GMM_OK;
  // Tuning override GMM_VARIANT: "single" forces the one-CTA kernels, "pair" the pairs.
  const char *variant = getenv("GMM_VARIANT");
  const bool pairs_ok = sms >= 2 && configure<false, true>(&h->var[0][1], optin, sm_smem, device_optin, sms) == GMM_OK &&
                        configure<true, true>(&h->var[1][1], optin, sm_smem, device_optin, sms) == GMM_OK &&
                        configure<false, true, true>(&h->var_fp8[1], optin, sm_smem, device_optin, sms) == GMM_OK;
  h->use_pairs = pairs_ok && !(variant && std::strcmp(variant, "single") == 0);
  // The 4-bit path too: each CTA of a pair loads half of a stage's tokens (a 6-deep token
  // ring fits), and one MMA instruction covers both CTAs' 128 weight rows, half the
  // instructions per unit of work for the issuing warp, which shares its SM
  // sub-partition with dequantisation warps.
  h->use_pairs_int4 = h->use_pairs;
  if (!single_ok) {
    cudaGetLastError();
    delete h;
    return GMM_ERR_CUDA;
  }
  configure_fp4<false>(&h->var_fp4[0], optin, sm_smem, device_optin, sms);
  configure_fp4<true>(&h->var_fp4[1], optin, sm_smem, device_optin, sms);
  configure_weight_grad(h->var_weight_grad, optin, sm_smem, device_optin, sms);
  if (configure_route() != GMM_OK) {
    cudaGetLastError();
    delete h;
    return GMM_ERR_CUDA;
  }
  cudaGetLastError();   // a 4-bit or weight gradient configuration that does not fit is not an error of this call

  h->debug = getenv("GMM_DEBUG") != nullptr;
  if (h->debug) {
    const gmm_variant *vs[7] = {&h->var[0][0], &h->var[0][1], &h->var[1][0], &h->var[1][1],
                                &h->var_fp8[0], &h->var_fp8[1], &h->var_fp8_block};
    const char *names[7] = {"bf16", "bf16 pair", "int4", "int4 pair", "e4m3", "e4m3 pair", "e4m3 block"};
    for (int i = 0; i < 7; ++i)
      fprintf(stderr, "gmm: %-16s stages %d smem %zu grid %d\n", names[i], vs[i]->stages, vs[i]->smem, vs[i]->grid);
  }
  const size_t zero_at = kStatusBytes + static_cast<size_t>(sms) * gmm::kMapSlotBytes;
  const size_t counts_at = zero_at + (gmm::kMaxGroups + 4) / 4 * 16;   // kMaxGroups + 1 words, whole 16 bytes
  h->ws_bytes = counts_at + (num_experts <= gmm::kRouteMaxExperts ? gmm::kRouteMaxCounts * sizeof(uint32_t) : 0);
  if (cudaMalloc(&h->ws, h->ws_bytes) != cudaSuccess ||
      cudaMemset(h->ws, 0, h->ws_bytes) != cudaSuccess) {
    cudaGetLastError();
    if (h->ws) cudaFree(h->ws);
    delete h;
    return GMM_ERR_CUDA;
  }
  h->zero_offsets = reinterpret_cast<const uint32_t *>(h->ws + zero_at);
  if (num_experts <= gmm::kRouteMaxExperts) h->route_counts = reinterpret_cast<uint32_t *>(h->ws + counts_at);
  *out = h;
  return GMM_OK;
}

int gmm_destroy(gmm_handle_t h) {
  if (!h) return GMM_OK;
  DeviceGuard guard(h->device);
  int rc = GMM_OK;
  if (h->ws && cudaFree(h->ws) != cudaSuccess) rc = GMM_ERR_CUDA;
  delete h;
  return rc;
}

int gmm_run_ex(gmm_handle_t h, void *c, const void *a, const uint32_t *a_offsets, const void *b,
               const int32_t *expert_ids, uint32_t *expert_usage_stats, int num_groups, int N, int K,
               const gmm_epilogue *epilogue, cudaStream_t stream) {
  take_no_rows(h, &c, &a, &a_offsets);
  int rc = check_common(h, c, a, a_offsets, expert_ids, expert_usage_stats, num_groups, N, K);
  if (rc) return rc;
  rc = check_epilogue(epilogue);
  if (rc) return rc;
  if (!b || !aligned16(b)) return GMM_ERR_INVALID_ARG;

  GmmParams p;
  std::memset(&p, 0, sizeof(p));
  {
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N),
                          static_cast<cuuint64_t>(h->num_experts)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(K) * 2, static_cast<cuuint64_t>(N) * K * 2};
    cuuint32_t box[3] = {gmm::kBK, gmm::kBlockN, 1};
    rc = encode_map(h, &p.w_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, b, dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  rc = encode_token_maps(h, p, a, K, 1);
  if (rc) return rc;
  fill_common(h, p, c, a_offsets, expert_ids, expert_usage_stats, num_groups, N, K, max_tok(h, false));
  set_epilogue(p, epilogue);
  return launch<false>(h, p, stream);
}

int gmm_run(gmm_handle_t h, void *c, const void *a, const uint32_t *a_offsets, const void *b,
            const int32_t *expert_ids, uint32_t *expert_usage_stats, int num_groups, int N, int K,
            cudaStream_t stream) {
  return gmm_run_ex(h, c, a, a_offsets, b, expert_ids, expert_usage_stats, num_groups, N, K, nullptr, stream);
}

// A-plane row offsetting: the bf16 grouped kernel with the tile's token rows read from
// the plane its weight rows belong to (the producer adds plane * a_offsets[G]).
int gmm_run_planes(gmm_handle_t h, void *c, const void *a, const uint32_t *a_offsets, const void *b,
                   const int32_t *expert_ids, uint32_t *expert_usage_stats, int num_groups, int N, int K,
                   const int *a_plane_splits, const gmm_epilogue *epilogue, cudaStream_t stream) {
  if (!a_plane_splits) return GMM_ERR_INVALID_ARG;
  const int s0 = a_plane_splits[0], s1 = a_plane_splits[1];
  if (s0 < 0 || s1 < 0 || s0 > N || s1 > N - s0) return GMM_ERR_INVALID_ARG;
  if (s0 % 256 || s1 % 256) return GMM_ERR_UNSUPPORTED;   // a tile's 256 weight rows in one plane
  take_no_rows(h, &c, &a, &a_offsets);
  int rc = check_common(h, c, a, a_offsets, expert_ids, expert_usage_stats, num_groups, N, K);
  if (rc) return rc;
  rc = check_epilogue(epilogue);
  if (rc) return rc;
  if (!b || !aligned16(b)) return GMM_ERR_INVALID_ARG;
  GmmParams p;
  std::memset(&p, 0, sizeof(p));
  {
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N),
                          static_cast<cuuint64_t>(h->num_experts)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(K) * 2, static_cast<cuuint64_t>(N) * K * 2};
    cuuint32_t box[3] = {gmm::kBK, gmm::kBlockN, 1};
    rc = encode_map(h, &p.w_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, b, dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  rc = encode_token_maps(h, p, a, K, 1);
  if (rc) return rc;
  fill_common(h, p, c, a_offsets, expert_ids, expert_usage_stats, num_groups, N, K, max_tok(h, false));
  set_epilogue(p, epilogue);
  p.plane_s0 = s0;
  p.plane_s1 = s1;
  return launch<false>(h, p, stream);
}

// The e4m3 operands go through the bf16 kernel's tensor maps unchanged, over their
// bytes: a row of K e4m3 values is a row of K / 2 two-byte units, so the maps, the
// stage ring and the swizzled layout are the bf16 ones and only the MMA kind and the
// epilogue's scales differ (see the kernel's kFp8 variant).
int gmm_run_fp8(gmm_handle_t h, void *c, const void *a, const uint32_t *a_offsets, const void *b,
                const int32_t *expert_ids, uint32_t *expert_usage_stats, int num_groups, int N, int K,
                const float *input_scale, const float *weight_scale, const int *scales_granularity_mnk,
                const gmm_epilogue *epilogue, cudaStream_t stream) {
  if (K < 16 || K % 16) return GMM_ERR_INVALID_ARG;
  const int KU = K / 2;   // two-byte units per row
  if (take_no_rows(h, &c, &a, &a_offsets) && !input_scale) input_scale = reinterpret_cast<const float *>(h->ws);
  int rc = check_common(h, c, a, a_offsets, expert_ids, expert_usage_stats, num_groups, N, KU);
  if (rc) return rc;
  rc = check_epilogue(epilogue);
  if (rc) return rc;
  if (!b || !aligned16(b)) return GMM_ERR_INVALID_ARG;
  if (!scales_granularity_mnk || !input_scale || !weight_scale) return GMM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(input_scale) & 3u) || (reinterpret_cast<uintptr_t>(weight_scale) & 3u))
    return GMM_ERR_INVALID_ARG;
  const int gm = scales_granularity_mnk[0], gn = scales_granularity_mnk[1], gk = scales_granularity_mnk[2];
  if (gm < 1 || gn < 1 || gk < 1) return GMM_ERR_INVALID_ARG;
  // Per-K-block scales run the block-scaled kernel: whole 128-K stages per block, and
  // one weight scale per 32-column TMEM load.
  const bool blockwise = gk < K;
  if (blockwise && (gk % 128 || gn % 32)) return GMM_ERR_UNSUPPORTED;

  GmmParams p;
  std::memset(&p, 0, sizeof(p));
  {
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(KU), static_cast<cuuint64_t>(N),
                          static_cast<cuuint64_t>(h->num_experts)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N) * K};
    const cuuint32_t rows = !blockwise ? static_cast<cuuint32_t>(gmm::kBlockN) : gmm::BwGeom::kRows;
    cuuint32_t box[3] = {gmm::kBK, rows, 1};
    rc = encode_map(h, &p.w_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, b, dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  rc = encode_token_maps(h, p, a, KU, 1);
  if (rc) return rc;
  fill_common(h, p, c, a_offsets, expert_ids, expert_usage_stats, num_groups, N, KU,
              !blockwise ? max_tok(h, false) : gmm::BwGeom::kMaxTok);
  set_epilogue(p, epilogue);
  p.in_scale = input_scale;
  p.w_scale = weight_scale;
  p.scale_gm = gm;
  p.scale_gn = gn;
  p.w_scale_cols = (N + gn - 1) / gn;
  p.scale_kb = (K + gk - 1) / gk;
  p.kb_stages = gk / 128;
  return blockwise ? launch_fp8_block(h, p, stream) : launch<false, true>(h, p, stream);
}

}  // extern "C"

namespace {

// The 4-bit path for `num_experts` experts of packed weights (the handle's E for the
// grouped calls, 1 for the dense one).
int run_int4(gmm_handle_t h, int num_experts, void *c, const void *a, const uint32_t *a_offsets,
             const uint32_t *b_packed, const void *b_scales, const int32_t *expert_ids,
             uint32_t *expert_usage_stats, int num_groups, int N, int K, int group_size,
             const gmm_epilogue *epilogue, cudaStream_t stream) {
  int rc = check_common(h, c, a, a_offsets, expert_ids, expert_usage_stats, num_groups, N, K);
  if (rc) return rc;
  rc = check_epilogue(epilogue);
  if (rc) return rc;
  if (!b_packed || !b_scales) return GMM_ERR_INVALID_ARG;
  if (!aligned16(b_packed) || (reinterpret_cast<uintptr_t>(b_scales) & 1u)) return GMM_ERR_INVALID_ARG;
  if (group_size < gmm::kBK || group_size % gmm::kBK || K % group_size) return GMM_ERR_UNSUPPORTED;

  GmmParams p;
  std::memset(&p, 0, sizeof(p));
  {
    // Packed weights as 32-bit words {K/8, N, E}; one box = 128 rows x 32 words (128 B,
    // two 128-K stages), 128-byte swizzle.
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(K / 8), static_cast<cuuint64_t>(N),
                          static_cast<cuuint64_t>(num_experts)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(K / 8) * 4, static_cast<cuuint64_t>(N) * (K / 8) * 4};
    cuuint32_t box[3] = {gmm::kQRowBytes / 4, gmm::kBlockN, 1};
    rc = encode_map(h, &p.w_map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, b_packed, dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  rc = encode_token_maps(h, p, a, K, gmm::kSub4);
  if (rc) return rc;
  fill_common(h, p, c, a_offsets, expert_ids, expert_usage_stats, num_groups, N, K, max_tok(h, true));
  p.scales = static_cast<const __nv_bfloat16 *>(b_scales);
  // Scale index of 64-K sub-slab j is j / (group_size / 64): a shift when that is a power of two.
  p.scale_shift = -1;
  for (int s = 0, g64 = group_size / gmm::kBK; (1 << s) <= g64; ++s)
    if ((1 << s) == g64) p.scale_shift = s;
  p.group_size = group_size;
  p.num_experts = num_experts;
  set_epilogue(p, epilogue);
  return launch<true>(h, p, stream);
}

}  // namespace

extern "C" {

int gmm_run_int4_ex(gmm_handle_t h, void *c, const void *a, const uint32_t *a_offsets,
                    const uint32_t *b_packed, const void *b_scales, const int32_t *expert_ids,
                    uint32_t *expert_usage_stats, int num_groups, int N, int K, int group_size,
                    const gmm_epilogue *epilogue, cudaStream_t stream) {
  if (!h) return GMM_ERR_INVALID_ARG;
  take_no_rows(h, &c, &a, &a_offsets);
  return run_int4(h, h->num_experts, c, a, a_offsets, b_packed, b_scales, expert_ids, expert_usage_stats,
                  num_groups, N, K, group_size, epilogue, stream);
}

int gmm_matmul_int4(gmm_handle_t h, void *c, const void *a, const uint32_t *b_packed, const void *b_scales,
                    int M, int N, int K, int group_size, const gmm_epilogue *epilogue, cudaStream_t stream) {
  if (!h || M < 0) return GMM_ERR_INVALID_ARG;
  if (M == 0) return GMM_OK;
  // One group of M rows with expert 0: its offsets, id and (unread) usage stats live
  // in the handle's status block, written in stream order before the kernel by value
  // writes (memset nodes in a captured CUDA graph, so a replay needs no host memory).
  DeviceGuard guard(h->device);
  const CUdeviceptr routing = reinterpret_cast<CUdeviceptr>(h->ws + kDenseRoutingOffset);   // a_offsets[0..1], expert_ids[0]
  if (with_context(h, [&] { return h->memset32(routing, 0u, 3, reinterpret_cast<CUstream>(stream)); }) != CUDA_SUCCESS ||
      h->memset32(routing + 4, static_cast<unsigned int>(M), 1, reinterpret_cast<CUstream>(stream)) != CUDA_SUCCESS) {
    cudaGetLastError();
    return GMM_ERR_CUDA;
  }
  const uint32_t *off = reinterpret_cast<const uint32_t *>(h->ws + kDenseRoutingOffset);
  const int32_t *ids = reinterpret_cast<const int32_t *>(h->ws + kDenseRoutingOffset + 8);
  uint32_t *stats = reinterpret_cast<uint32_t *>(h->ws + kDenseStatsOffset);
  return run_int4(h, 1, c, a, off, b_packed, b_scales, ids, stats, 1, N, K, group_size, epilogue, stream);
}

int gmm_run_int4(gmm_handle_t h, void *c, const void *a, const uint32_t *a_offsets,
                 const uint32_t *b_packed, const void *b_scales, const int32_t *expert_ids,
                 uint32_t *expert_usage_stats, int num_groups, int N, int K, int group_size,
                 cudaStream_t stream) {
  return gmm_run_int4_ex(h, c, a, a_offsets, b_packed, b_scales, expert_ids, expert_usage_stats, num_groups, N,
                         K, group_size, nullptr, stream);
}

int gmm_dispatch(gmm_handle_t h, uint32_t *a_offsets, int32_t *slot_rows, int32_t *row_slots, void *rows,
                 const int32_t *slot_experts, const void *tokens, long long tokens_stride, int num_tokens, int top_k,
                 int width, int dtype, cudaStream_t stream) {
  if (!rows != !tokens) return GMM_ERR_INVALID_ARG;
  const bool copy = tokens != nullptr;
  int rc = check_rows(h, num_tokens, top_k, copy ? width : 1, copy ? dtype : GMM_DTYPE_BF16, copy ? tokens_stride : 0);
  if (rc) return rc;
  if (!a_offsets || !aligned_to(a_offsets, 4)) return GMM_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!slot_rows || !row_slots || !slot_experts || !aligned_to(slot_rows, 4) ||
                         !aligned_to(row_slots, 4) || !aligned_to(slot_experts, 4)))
    return GMM_ERR_INVALID_ARG;
  if (h->num_experts > gmm::kRouteMaxExperts) return GMM_ERR_UNSUPPORTED;
  if (num_tokens == 0) {   // nothing to sort: every expert has no rows
    DeviceGuard guard(h->device);
    const cudaError_t err = cudaMemsetAsync(a_offsets, 0, (static_cast<size_t>(h->num_experts) + 1) * 4, stream);
    if (err == cudaSuccess) return GMM_OK;
    debug_report("cudaMemsetAsync", static_cast<int>(err), cudaGetErrorString(err));
    cudaGetLastError();
    return GMM_ERR_CUDA;
  }
  gmm::DispatchParams p;
  std::memset(&p, 0, sizeof(p));
  p.slot_experts = slot_experts;
  p.a_offsets = a_offsets;
  p.slot_rows = slot_rows;
  p.row_slots = row_slots;
  p.num_tokens = num_tokens;
  p.top_k = top_k;
  p.num_experts = h->num_experts;
  p.counts = h->route_counts;
  p.status = reinterpret_cast<uint32_t *>(h->ws);
  int vb = 16;
  if (copy) {
    const int es = dtype_bytes(dtype);
    if (!aligned_to(rows, es) || !aligned_to(tokens, es)) return GMM_ERR_INVALID_ARG;
    p.tokens = static_cast<const uint8_t *>(tokens);
    p.rows = static_cast<uint8_t *>(rows);
    p.token_pitch = tokens_stride * es;
    p.row_bytes = static_cast<long long>(width) * es;
    const unsigned long long all = reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(rows) |
                                   static_cast<unsigned long long>(p.token_pitch | p.row_bytes);
    vb = all % 16 == 0 ? 16 : (all % 4 == 0 ? 4 : 2);
  }
  DeviceGuard guard(h->device);
  return vb == 16 ? launch_dispatch<16>(h, p, stream)
                  : (vb == 4 ? launch_dispatch<4>(h, p, stream) : launch_dispatch<2>(h, p, stream));
}

int gmm_combine(gmm_handle_t h, void *out, long long out_stride, const void *rows, int num_rows, const int32_t *slot_rows,
                const float *weights, int num_tokens, int top_k, int width, int dtype, cudaStream_t stream) {
  int rc = check_rows(h, num_tokens, top_k, width, dtype, out_stride);
  if (rc) return rc;
  if (num_rows < 0) return GMM_ERR_INVALID_ARG;
  if (num_tokens == 0) return GMM_OK;
  const int es = dtype_bytes(dtype);
  if (!out || (!rows && num_rows > 0) || !slot_rows || !aligned_to(out, es) || !aligned_to(rows, es) ||
      !aligned_to(slot_rows, 4) || !aligned_to(weights, 4))
    return GMM_ERR_INVALID_ARG;
  if (out_stride < width && num_tokens > 1) return GMM_ERR_INVALID_ARG;   // rows of the output overlap
  gmm::CombineParams p;
  std::memset(&p, 0, sizeof(p));
  p.out = static_cast<uint8_t *>(out);
  p.rows = static_cast<const uint8_t *>(rows);
  p.slot_rows = slot_rows;
  p.weights = weights;
  p.out_pitch = out_stride * es;
  p.row_bytes = static_cast<long long>(width) * es;
  p.num_tokens = num_tokens;
  p.top_k = top_k;
  p.num_rows = num_rows;
  p.status = reinterpret_cast<uint32_t *>(h->ws);
  const bool vec = aligned16(out) && aligned16(rows) && p.out_pitch % 16 == 0 && p.row_bytes % 16 == 0;
  return run_combine(h, p, dtype, vec, false, stream);
}

int gmm_combine_grad(gmm_handle_t h, void *d_rows, float *d_weights, const void *d_out, long long d_out_stride,
                     const void *rows, int num_rows, const int32_t *slot_rows, const float *weights, int num_tokens,
                     int top_k, int width, int dtype, cudaStream_t stream) {
  int rc = check_rows(h, num_tokens, top_k, width, dtype, d_out_stride);
  if (rc) return rc;
  if (num_rows < 0) return GMM_ERR_INVALID_ARG;
  if (num_tokens == 0) return GMM_OK;
  const int es = dtype_bytes(dtype);
  if ((!d_rows && num_rows > 0) || !d_out || (d_weights && !rows && num_rows > 0) || !slot_rows ||
      !aligned_to(d_rows, es) || !aligned_to(d_out, es) || !aligned_to(rows, es) || !aligned_to(slot_rows, 4) ||
      !aligned_to(weights, 4) || !aligned_to(d_weights, 4))
    return GMM_ERR_INVALID_ARG;
  gmm::CombineParams p;
  std::memset(&p, 0, sizeof(p));
  p.rows = static_cast<const uint8_t *>(rows);
  p.slot_rows = slot_rows;
  p.weights = weights;
  p.d_out = static_cast<const uint8_t *>(d_out);
  p.d_rows = static_cast<uint8_t *>(d_rows);
  p.d_weights = d_weights;
  p.out_pitch = d_out_stride * es;
  p.row_bytes = static_cast<long long>(width) * es;
  p.num_tokens = num_tokens;
  p.top_k = top_k;
  p.num_rows = num_rows;
  p.status = reinterpret_cast<uint32_t *>(h->ws);
  const bool vec = aligned16(d_out) && aligned16(d_rows) && (!d_weights || aligned16(rows)) && p.out_pitch % 16 == 0 &&
                   p.row_bytes % 16 == 0;
  return run_combine(h, p, dtype, vec, true, stream);
}

int gmm_quantize_fp4(gmm_handle_t h, void *packed, void *scales, const void *x, long long x_stride, int src_rows,
                     const int32_t *row_slots, int top_k, const float *global_scale, int rows, int K, int dtype,
                     int format, cudaStream_t stream) {
  if (top_k < 1 || src_rows < 0) return GMM_ERR_INVALID_ARG;
  if (!row_slots && src_rows < rows) return GMM_ERR_INVALID_ARG;
  gmm::QuantParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = static_cast<const uint8_t *>(x);
  p.packed = static_cast<uint8_t *>(packed);
  p.scales = static_cast<uint8_t *>(scales);
  p.row_slots = row_slots;
  p.global_scale = global_scale;
  p.rows = rows;
  p.src_rows = src_rows;
  p.K = K;
  p.top_k = top_k;
  return run_quant(h, p, dtype, format, x_stride, true, stream);
}

int gmm_dequantize_fp4(gmm_handle_t h, void *y, long long y_stride, const void *packed, const void *scales,
                       const float *global_scale, int rows, int K, int dtype, int format, cudaStream_t stream) {
  gmm::QuantParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = static_cast<const uint8_t *>(y);
  p.packed = static_cast<uint8_t *>(const_cast<void *>(packed));
  p.scales = static_cast<uint8_t *>(const_cast<void *>(scales));
  p.global_scale = global_scale;
  p.rows = rows;
  p.K = K;
  p.top_k = 1;
  return run_quant(h, p, dtype, format, y_stride, false, stream);
}

// The packed values go through the bf16 kernel's tensor maps over their bytes: a row of K
// e2m1 values is K / 2 bytes, K / 4 two-byte units.
int gmm_run_fp4(gmm_handle_t h, void *c, const void *a, const uint32_t *a_offsets, const void *b,
                const int32_t *expert_ids, uint32_t *expert_usage_stats, int num_groups, int N, int K,
                const void *a_scales, const void *b_scales, int format, const float *a_global, const float *b_global,
                const gmm_epilogue *epilogue, cudaStream_t stream) {
  if (format != GMM_FP4_NV && format != GMM_FP4_MX) return GMM_ERR_INVALID_ARG;
  if (K < 32 || K % 32) return GMM_ERR_INVALID_ARG;
  const int KU = K / 4;
  const bool no_rows = take_no_rows(h, &c, &a, &a_offsets);
  if (h && (no_rows || num_groups == 0)) {   // nothing of them is read or written
    if (!c) c = h->ws;
    if (!a) a = h->ws;
    if (!a_scales) a_scales = h->ws;
  }
  int rc = check_common(h, c, a, a_offsets, expert_ids, expert_usage_stats, num_groups, N, KU);
  if (rc) return rc;
  rc = check_epilogue(epilogue);
  if (rc) return rc;
  if (!b || !aligned16(b) || !a_scales || !b_scales || !aligned16(a_scales) || !aligned16(b_scales) ||
      !aligned_to(a_global, 4) || !aligned_to(b_global, 4))
    return GMM_ERR_INVALID_ARG;
  gmm::F4Params p;
  std::memset(&p, 0, sizeof(p));
  {
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(KU), static_cast<cuuint64_t>(N),
                          static_cast<cuuint64_t>(h->num_experts)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(KU) * 2, static_cast<cuuint64_t>(N) * KU * 2};
    cuuint32_t box[3] = {gmm::kBK, gmm::kBlockN, 1};
    rc = encode_map(h, &p.w_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, b, dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  rc = encode_token_maps(h, p, a, KU, 1);
  if (rc) return rc;
  fill_common(h, p, c, a_offsets, expert_ids, expert_usage_stats, num_groups, N, KU, gmm::kF4MaxTok);
  set_epilogue(p, epilogue);
  p.g_a = a_global;
  p.g_w = b_global;
  p.sf_a = static_cast<const uint8_t *>(a_scales);
  p.sf_w = static_cast<const uint8_t *>(b_scales);
  p.sf_pitch = fp4_scale_pitch(K, format);
  return format == GMM_FP4_MX ? launch_fp4<true>(h, p, stream) : launch_fp4<false>(h, p, stream);
}

int gmm_query_status(gmm_handle_t h, cudaStream_t stream) {
  if (!h) return GMM_ERR_INVALID_ARG;
  DeviceGuard guard(h->device);
  uint32_t status = 0;
  bool ok = cudaMemcpyAsync(&status, h->ws, sizeof(status), cudaMemcpyDeviceToHost, stream) == cudaSuccess &&
            cudaStreamSynchronize(stream) == cudaSuccess;
  if (ok && status) {
    // Only what was read is cleared: a call on another stream may have reported since.  Done when this returns, or
    // the clearing could take back a report of a later call.
    void *args[2] = {&h->ws, &status};
    ok = cudaLaunchKernel(reinterpret_cast<const void *>(gmm_clear_status_kernel), dim3(1), dim3(1), args, 0, stream) == cudaSuccess &&
         cudaStreamSynchronize(stream) == cudaSuccess;
  }
  if (!ok) {
    cudaGetLastError();
    return GMM_ERR_CUDA;
  }
  if (status & gmm::kStatusTimeout) return GMM_ERR_DEVICE_TIMEOUT;
  if (status) return GMM_ERR_BAD_INPUT;
  return GMM_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Allocation-free entry point (gmm_run_noalloc).
//
// Some callers cannot call cudaMalloc at the moment they need a grouped GEMM:
// code running inside a custom allocator or memory-pool callback, a framework
// that has reserved the whole device for its own pool, or an inference runtime
// that forbids allocations after start-up.  gmm_run_noalloc serves them: it
// launches the same bf16 kernel as gmm_run, but takes the kernel's scratch (its
// status word and the per-CTA patched tensor maps) from the fixed array below
// instead of a handle's cudaMalloc'd workspace, and it creates no handle.
//
// g_noalloc_scratch lives in every GPU that loads this library, until the
// process exits.  In host code its name is only a host-side stand-in, so the
// host never passes it to a kernel: it passes the device address obtained from
// cudaGetSymbolAddress once per device.
// ---------------------------------------------------------------------------
namespace {

constexpr int kNoAllocMaxCtas = 256;   // persistent grid = SM count; 152 on GB300
constexpr size_t kNoAllocScratchBytes = kStatusBytes + static_cast<size_t>(kNoAllocMaxCtas) * gmm::kMapSlotBytes;
constexpr int kNoAllocMaxDevices = 64;

static __device__ __align__(256) uint8_t g_noalloc_scratch[kNoAllocScratchBytes];   // 524,544 bytes

struct NoAllocDevice {
  bool ready = false;   // set-up succeeded; a failed set-up is retried by the next call
  gmm_ctx ctx;          // static storage; ctx.ws points into g_noalloc_scratch on this device
};

NoAllocDevice g_noalloc_devices[kNoAllocMaxDevices];
std::mutex g_noalloc_mutex;

// One-time set-up for the current device: resolve the scratch array's device
// address (which loads the library's module on this device, and with it the array,
// if that has not happened yet), the tensor-map encoder and the kernel's
// shared-memory configuration.  Only a successful set-up is kept: one that failed
// (for instance because it was attempted during a stream capture, where some of
// these calls are refused) is attempted again by the next call.
int noalloc_setup(int device, gmm_ctx **out) {
  std::lock_guard<std::mutex> lock(g_noalloc_mutex);
  NoAllocDevice &d = g_noalloc_devices[device];
  if (d.ready) {
    *out = &d.ctx;
    return GMM_OK;
  }
  int major = 0, minor = 0, sms = 0, optin = 0;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, device);
  int rc = GMM_OK;
  if (major != 10 || minor != 3 || sms < 1) rc = GMM_ERR_NO_DEVICE;
  else if (sms > kNoAllocMaxCtas) rc = GMM_ERR_UNSUPPORTED;   // scratch holds 256 CTA slots
  void *scratch = nullptr;
  if (rc == GMM_OK && cudaGetSymbolAddress(&scratch, g_noalloc_scratch) != cudaSuccess) rc = GMM_ERR_CUDA;
  void *fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (rc == GMM_OK &&
      (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
           cudaSuccess ||
       q != cudaDriverEntryPointSuccess || !fn))
    rc = GMM_ERR_CUDA;
  if (rc == GMM_OK) {
    d.ctx.device = device;
    d.ctx.num_sms = sms;
    d.ctx.encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    d.ctx.use_pairs = 0;   // one CTA per tile: the grid is the SM count, one scratch slot per CTA
    int sm_smem = 0;
    cudaDeviceGetAttribute(&sm_smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor, device);
    if (configure<false, false>(&d.ctx.var[0][0], optin, sm_smem, optin, sms) != GMM_OK) rc = GMM_ERR_CUDA;
    d.ctx.ws = static_cast<uint8_t *>(scratch);
    d.ctx.ws_bytes = kNoAllocScratchBytes;
  }
  if (rc != GMM_OK) {
    cudaGetLastError();
    return rc;
  }
  d.ready = true;
  *out = &d.ctx;
  return GMM_OK;
}

}  // namespace

extern "C" int gmm_run_noalloc(void *c, const void *a, const uint32_t *a_offsets, const void *b,
                               const int32_t *expert_ids, uint32_t *expert_usage_stats, int num_experts,
                               int num_groups, int N, int K, cudaStream_t stream) {
  if (num_experts < 1) return GMM_ERR_INVALID_ARG;
  int device = -1;
  if (cudaGetDevice(&device) != cudaSuccess || device < 0) {
    cudaGetLastError();
    return GMM_ERR_NO_DEVICE;
  }
  if (device >= kNoAllocMaxDevices) return GMM_ERR_UNSUPPORTED;
  gmm_ctx *h = nullptr;
  int rc = noalloc_setup(device, &h);
  if (rc) return rc;
  rc = check_common(h, c, a, a_offsets, expert_ids, expert_usage_stats, num_groups, N, K);
  if (rc) return rc;
  if (!b || !aligned16(b)) return GMM_ERR_INVALID_ARG;

  GmmParams p;
  std::memset(&p, 0, sizeof(p));
  {
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N),
                          static_cast<cuuint64_t>(num_experts)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(K) * 2, static_cast<cuuint64_t>(N) * K * 2};
    cuuint32_t box[3] = {gmm::kBK, gmm::kBlockN, 1};
    rc = encode_map(h, &p.w_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, b, dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  rc = encode_token_maps(h, p, a, K, 1);
  if (rc) return rc;
  fill_common(h, p, c, a_offsets, expert_ids, expert_usage_stats, num_groups, N, K, max_tok(h, false));
  p.num_experts = num_experts;
  // The status word keeps the previous call's flags: clear it (stream-ordered, no allocation).
  if (cudaMemsetAsync(h->ws, 0, sizeof(uint32_t), stream) != cudaSuccess) {
    cudaGetLastError();
    return GMM_ERR_CUDA;
  }
  return launch<false>(h, p, stream);
}
