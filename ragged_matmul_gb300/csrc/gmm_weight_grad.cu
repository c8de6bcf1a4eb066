// Host side of the weight gradient on 8-bit operands (gmm_weight_grad_fp8): argument checks,
// tensor maps, the tile grid and the launch.
#include "gmm_host.h"
#include "gmm_weight_grad.cuh"

namespace {

using namespace gmm::host;
using gmm::WeightGradParams;

size_t offsets_bytes(int groups) { return (static_cast<size_t>(groups + 1) * 4 + 15) & ~static_cast<size_t>(15); }

const void *kernel_of(bool bf16) {
  return bf16 ? reinterpret_cast<const void *>(gmm::gmm_weight_grad_fp8_kernel<true>)
              : reinterpret_cast<const void *>(gmm::gmm_weight_grad_fp8_kernel<false>);
}

cudaLaunchConfig_t pair_config(unsigned grid, size_t smem, cudaStream_t stream, cudaLaunchAttribute *attr) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = 2;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(gmm::kWgThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

size_t staging_bytes(bool bf16, int bufs) {   // buffers of all epilogue warps
  return static_cast<size_t>(bufs) * (bf16 ? gmm::kWgStgBytes<true> : gmm::kWgStgBytes<false>);
}

int stages_of(const gmm_variant &v, int groups, bool bf16, int bufs) {
  const size_t fixed = gmm::kWgFixedBytes + staging_bytes(bf16, bufs) + offsets_bytes(groups);
  if (v.budget < fixed) return 0;
  return static_cast<int>(std::min<size_t>(gmm::kWgMaxStages, (v.budget - fixed) / gmm::kWgStageBytes));
}

// A map of e4m3 codes {pitch, rows}: `box` rows of one stage.
int encode_codes(gmm_ctx *h, CUtensorMap *m, const void *codes, long long pitch, int rows, uint32_t box) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(pitch), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
  const cuuint32_t b[2] = {gmm::kWgBlock, box};
  return encode_map(h, m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, strides, b, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

namespace gmm {
namespace host {

// As for the 4-bit floating point kernel: grid 0 where the device or the budget cannot run it.
void configure_weight_grad(gmm_variant (&vars)[2], int optin, int sm_smem, int device_optin, int num_sms) {
  for (int bf16 = 0; bf16 < 2; ++bf16) {
    gmm_variant &v = vars[bf16];
    v.grid = 0;
    const void *kernel = kernel_of(bf16);
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess) return;
    const long avail = static_cast<long>(optin) - static_cast<long>(attr.sharedSizeBytes);
    if (avail <= 0 || num_sms < 2) return;
    v.budget = static_cast<size_t>(avail);
    v.stages = stages_of(v, 1, bf16, 8);
    if (v.stages < v.min_stages) return;
    const long reserve = static_cast<long>(sm_smem) / 2 + 1024;   // more than half an SM: one CTA per SM
    const long cap = static_cast<long>(device_optin) - static_cast<long>(attr.sharedSizeBytes);
    v.smem = static_cast<size_t>(std::min(cap, std::max(avail, reserve)));
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(v.smem)) != cudaSuccess)
      return;
    cudaLaunchAttribute la[1];
    const cudaLaunchConfig_t cfg = pair_config(static_cast<unsigned>(num_sms & ~1), v.smem, nullptr, la);
    int clusters = 0;
    const cudaError_t err = bf16 ? cudaOccupancyMaxActiveClusters(&clusters, gmm::gmm_weight_grad_fp8_kernel<true>, &cfg)
                                 : cudaOccupancyMaxActiveClusters(&clusters, gmm::gmm_weight_grad_fp8_kernel<false>, &cfg);
    if (err != cudaSuccess || clusters < 1) return;
    v.grid = std::min(2 * clusters, num_sms & ~1);
  }
}

}  // namespace host
}  // namespace gmm

extern "C" int gmm_weight_grad_fp8(gmm_handle_t h, void *d_b, const void *d_t, const void *d_t_scales, const void *a_t,
                                   const void *a_t_scales, const uint32_t *a_offsets, int num_groups, int rows, int N,
                                   int K, int dtype, int accumulate, cudaStream_t stream) {
  if (!h || num_groups < 0 || rows < 0 || N < 16 || N % 16 || K < 16 || K % 16 || !dtype_bytes(dtype) ||
      (accumulate != 0 && accumulate != 1) || (accumulate && dtype != GMM_DTYPE_FP32))
    return GMM_ERR_INVALID_ARG;
  if (dtype == GMM_DTYPE_FP16 || N > (1 << 24) || K > (1 << 24) || num_groups > gmm::kMaxGroups || rows / 128 > (1 << 23))
    return GMM_ERR_UNSUPPORTED;
  if (num_groups == 0) return GMM_OK;
  if (!d_b || !aligned16(d_b)) return GMM_ERR_INVALID_ARG;
  if (rows > 0 && (!d_t || !d_t_scales || !a_t || !a_t_scales || !a_offsets || !aligned16(d_t) || !aligned16(a_t) ||
                   !aligned_to(a_offsets, 4)))
    return GMM_ERR_INVALID_ARG;
  const bool bf16 = dtype == GMM_DTYPE_BF16;
  const gmm_variant &v = h->var_weight_grad[bf16];
  if (v.grid == 0) return GMM_ERR_UNSUPPORTED;

  WeightGradParams p;
  std::memset(&p, 0, sizeof(p));
  const uint32_t units = static_cast<uint32_t>(K) / gmm::kWgUnit, most = gmm::kWgMaxK / gmm::kWgUnit;
  p.k_tiles = (units + most - 1) / most;
  p.width = units / p.k_tiles * gmm::kWgUnit;
  p.wide = units % p.k_tiles;
  p.n_tiles = (static_cast<uint32_t>(N) + gmm::kWgTileN - 1) / gmm::kWgTileN;
  const unsigned long long total = static_cast<unsigned long long>(p.k_tiles) * p.n_tiles * num_groups;
  if (total > 0x7fffffffull) return GMM_ERR_UNSUPPORTED;
  p.total = static_cast<uint32_t>(total);
  // The epilogue: warps and staging buffers of each, against stages of the operands' ring (a buffer is
  // 4 KB in fp32 and 2 in bf16).  A warp's way through 32 columns is latency, so where a tile has few
  // stages or a CTA few tiles, eight warps: bf16, 15 groups of 308 rows, N = 3120, K = 1152, 29.6 us
  // with eight and 39.1 with four; fp32, 16 groups, N = 1024, K = 512, 10.4 us with two buffers
  // each and 11.7 with four warps.  Long groups hide four (32768 rows over 8 groups, N = 14336,
  // K = 4096, bf16: 1094 us, 1116 with eight).  Many tiles in fp32 are bound by the gradient's bytes, and
  // the ring counts: 64 groups, N = 2816, K = 2048, 278 us with four warps of one buffer, 293 with
  // eight, 297 with four of two.
  const bool few = total <= 3u * static_cast<uint32_t>(v.grid / 2);
  p.epi_warps = (bf16 ? rows / num_groups < 1024 : few) ? 8 : 4;
  p.stg_bufs = (bf16 ? p.epi_warps == 4 : few) ? 2 : 1;
  p.num_stages = stages_of(v, num_groups, bf16, p.epi_warps * p.stg_bufs);
  if (p.num_stages < v.min_stages) return GMM_ERR_UNSUPPORTED;   // the offsets leave no room for the ring
  // As many n tiles a band as make the tiles that run side by side about as deep as they are wide.
  const uint32_t band = std::min(8u, p.n_tiles);
  p.band = gmm::Divisor::of(band);
  p.rest = gmm::Divisor::of(std::max(1u, p.n_tiles % band));
  p.whole = gmm::Divisor::of(band * p.k_tiles);
  p.per_group = gmm::Divisor::of(p.k_tiles * p.n_tiles);
  p.d_scales = static_cast<const uint8_t *>(d_t_scales);
  p.a_scales = static_cast<const uint8_t *>(a_t_scales);
  p.a_offsets = rows > 0 ? a_offsets : nullptr;
  p.status = reinterpret_cast<uint32_t *>(h->ws);
  p.num_groups = num_groups;
  p.rows = rows;
  p.N = N;
  p.K = K;
  p.accumulate = accumulate;
  if (const char *env = getenv("GMM_TEST_WAIT_LIMIT_NS")) p.wait_limit_ns = strtoull(env, nullptr, 10);

  int rc = GMM_OK;
  if (rows > 0) {
    const long long pitch = (static_cast<long long>(rows) / 128 + num_groups) * 128;
    rc = encode_codes(h, &p.d_map, d_t, pitch, N, gmm::kBlockN);
    if (!rc) rc = encode_codes(h, &p.a_map[0], a_t, pitch, K, p.width / 2);
    if (!rc) rc = p.wide ? encode_codes(h, &p.a_map[1], a_t, pitch, K, (p.width + gmm::kWgUnit) / 2) : (p.a_map[1] = p.a_map[0], GMM_OK);
    if (rc) return rc;
  }
  const int es = bf16 ? 2 : 4;
  for (int whole = 0; whole < 2; ++whole) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(num_groups)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(K) * es, static_cast<cuuint64_t>(N) * K * es};
    const cuuint32_t cols = whole ? 32 : 16, box[3] = {cols, 32, 1};
    const uint32_t row = cols * es;   // the staging buffer's row, swizzled over its whole width
    rc = encode_map(h, &p.out_map[whole], bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, d_b, dims,
                    strides, box,
                    row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : (row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B));
    if (rc) return rc;
  }

  DeviceGuard guard(h->device);
  const unsigned grid = std::min<unsigned>(static_cast<unsigned>(v.grid), 2u * p.total);
  cudaLaunchAttribute la[1];
  const cudaLaunchConfig_t cfg = pair_config(grid, v.smem, stream, la);
  const cudaError_t err = bf16 ? cudaLaunchKernelEx(&cfg, gmm::gmm_weight_grad_fp8_kernel<true>, p)
                               : cudaLaunchKernelEx(&cfg, gmm::gmm_weight_grad_fp8_kernel<false>, p);
  if (err != cudaSuccess) {
    debug_report("launch of the weight gradient kernel", static_cast<int>(err), cudaGetErrorString(err));
    cudaGetLastError();
    return GMM_ERR_CUDA;
  }
  return GMM_OK;
}
