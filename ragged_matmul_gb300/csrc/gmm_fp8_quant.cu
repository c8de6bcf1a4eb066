// Host side of the 8-bit quantisers (gmm_quantize_fp8, _tiles, _cols): argument checks, the
// kernel variant and the launch.
#include <type_traits>

#include "gmm_fp8_quant.cuh"
#include "gmm_host.h"

namespace {

using namespace gmm::host;
using gmm::Quant8Params;

constexpr int kMaxWidth = 1 << 24;
constexpr int kMaxRows = 1 << 30;

// Calls f with a value of the rows' type.
template <class F>
void by_dtype(int dtype, F f) {
  switch (dtype) {
    case GMM_DTYPE_BF16: f(__nv_bfloat16()); break;
    case GMM_DTYPE_FP16: f(__half()); break;
    default: f(float()); break;
  }
}

int alignment(const void *p, long long pitch) {
  const unsigned long long at = reinterpret_cast<uintptr_t>(p) | static_cast<unsigned long long>(pitch);
  return at % 32 == 0 ? 32 : (at % 16 == 0 ? 16 : 1);
}

template <class F>
void by_align(int align, F f) {
  if (align == 32) f(std::integral_constant<int, 32>());
  else if (align == 16) f(std::integral_constant<int, 16>());
  else f(std::integral_constant<int, 1>());
}

int check_quant8(gmm_ctx *h, Quant8Params &p, const void *x, long long x_stride, int src_rows, const int32_t *row_slots,
                 int top_k, int rows, int width, int dtype) {
  if (!h || !dtype_bytes(dtype) || rows < 0 || src_rows < 0 || x_stride < 0 || top_k < 1 || width < 16 || width % 16)
    return GMM_ERR_INVALID_ARG;
  if (width > kMaxWidth || rows > kMaxRows) return GMM_ERR_UNSUPPORTED;
  if (!row_slots && src_rows < rows) return GMM_ERR_INVALID_ARG;
  const int es = dtype_bytes(dtype);
  if (!aligned_to(x, es) || !aligned_to(row_slots, 4) || (rows > 0 && src_rows > 0 && !x)) return GMM_ERR_INVALID_ARG;
  std::memset(&p, 0, sizeof(p));
  p.x = static_cast<const uint8_t *>(x);
  p.x_pitch = x_stride * es;
  p.row_slots = row_slots;
  p.rows = rows;
  p.src_rows = src_rows;
  p.width = width;
  p.blocks = (width + gmm::kQ8Block - 1) / gmm::kQ8Block;
  p.by_blocks = gmm::Divisor::of(static_cast<uint32_t>(p.blocks));
  p.by_top_k = gmm::Divisor::of(static_cast<uint32_t>(top_k));
  p.status = reinterpret_cast<uint32_t *>(h->ws);
  return GMM_OK;
}

}  // namespace

extern "C" {

int gmm_quantize_fp8(gmm_handle_t h, void *q, float *scales, const void *x, long long x_stride, int src_rows,
                     const int32_t *row_slots, int top_k, int rows, int K, int dtype, int pow2, cudaStream_t stream) {
  Quant8Params p;
  const int rc = check_quant8(h, p, x, x_stride, src_rows, row_slots, top_k, rows, K, dtype);
  if (rc) return rc;
  if (pow2 != 0 && pow2 != 1) return GMM_ERR_INVALID_ARG;
  if (rows == 0) return GMM_OK;
  if (!q || !scales || !aligned16(q) || !aligned_to(scales, 4)) return GMM_ERR_INVALID_ARG;
  p.q = static_cast<uint8_t *>(q);
  p.scales = scales;
  // Units (a row's block) are numbered in 31 bits; longer calls go in slabs.
  constexpr int kUnits = gmm::kQ8Threads / gmm::kQ8RowLanes;   // of a CTA
  const int slab = static_cast<int>(((1ll << 31) - kUnits) / p.blocks);
  const int align = alignment(x, p.x_pitch);
  DeviceGuard guard(h->device);
  for (int row0 = 0; row0 < rows; row0 += std::min(slab, rows - row0)) {
    p.row0 = row0;
    p.rows = std::min(slab, rows - row0);
    const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.rows) * p.blocks + kUnits - 1) / kUnits);
    by_dtype(dtype, [&](auto t) {
      by_align(align, [&](auto a) {
        if (pow2) gmm::gmm_quantize_fp8_kernel<decltype(t), true, a.value><<<grid, gmm::kQ8Threads, 0, stream>>>(p);
        else gmm::gmm_quantize_fp8_kernel<decltype(t), false, a.value><<<grid, gmm::kQ8Threads, 0, stream>>>(p);
      });
    });
    const int launched = launch_status("launch of the 8-bit quantisation kernel");
    if (launched) return launched;
  }
  return GMM_OK;
}

int gmm_quantize_fp8_tiles(gmm_handle_t h, void *q, float *scales, const void *x, int batch, int N, int K, int dtype,
                           int pow2, cudaStream_t stream) {
  Quant8Params p;
  if (batch < 0 || N < 0) return GMM_ERR_INVALID_ARG;
  const int rc = check_quant8(h, p, x, K, N, nullptr, 1, batch > 0 ? N : 0, K, dtype);
  if (rc) return rc;
  if (pow2 != 0 && pow2 != 1) return GMM_ERR_INVALID_ARG;
  if (batch == 0 || N == 0) return GMM_OK;
  if (!x || !q || !scales || !aligned16(q) || !aligned_to(scales, 4)) return GMM_ERR_INVALID_ARG;
  p.row_blocks = (N - 1) / gmm::kQ8Block + 1;
  const long long tiles = static_cast<long long>(p.row_blocks) * p.blocks;
  if (tiles > 0x7fffffffll / batch) return GMM_ERR_UNSUPPORTED;   // tiles are numbered in 31 bits
  p.q = static_cast<uint8_t *>(q);
  p.scales = scales;
  const unsigned grid = static_cast<unsigned>(tiles * batch);
  DeviceGuard guard(h->device);
  by_dtype(dtype, [&](auto t) {
    by_align(alignment(x, p.x_pitch), [&](auto a) {
      if (pow2) gmm::gmm_quantize_fp8_tiles_kernel<decltype(t), true, a.value><<<grid, gmm::kQ8Threads, 0, stream>>>(p);
      else gmm::gmm_quantize_fp8_tiles_kernel<decltype(t), false, a.value><<<grid, gmm::kQ8Threads, 0, stream>>>(p);
    });
  });
  return launch_status("launch of the 8-bit tile quantisation kernel");
}

int gmm_quantize_fp8_cols(gmm_handle_t h, void *q_t, void *t_scales, void *q, float *scales, const void *x,
                          long long x_stride, int src_rows, const int32_t *row_slots, int top_k, const uint32_t *a_offsets,
                          int num_groups, int rows, int width, int dtype, cudaStream_t stream) {
  Quant8Params p;
  const int rc = check_quant8(h, p, x, x_stride, src_rows, row_slots, top_k, rows, width, dtype);
  if (rc) return rc;
  if (num_groups < 0 || !q != !scales) return GMM_ERR_INVALID_ARG;
  if (num_groups > gmm::kMaxGroups) return GMM_ERR_UNSUPPORTED;
  if (!aligned_to(a_offsets, 4) || !aligned16(q_t) || !aligned16(q) || !aligned_to(scales, 4)) return GMM_ERR_INVALID_ARG;
  if (rows == 0 || num_groups == 0) return GMM_OK;
  if (!a_offsets || !q_t || !t_scales) return GMM_ERR_INVALID_ARG;
  const long long blocks = rows / gmm::kQ8Block + num_groups;
  if (blocks > 0x7fffffffll / gmm::kQ8Block || blocks > 0x7fffffffll / p.blocks) return GMM_ERR_UNSUPPORTED;
  p.q_t = static_cast<uint8_t *>(q_t);
  p.t_scales = static_cast<uint8_t *>(t_scales);
  p.q = static_cast<uint8_t *>(q);
  p.scales = scales;
  p.a_offsets = a_offsets;
  p.groups = num_groups;
  p.pitch = static_cast<int>(blocks * gmm::kQ8Block);
  const unsigned grid = static_cast<unsigned>(blocks * p.blocks);
  DeviceGuard guard(h->device);
  const bool vec = alignment(x, p.x_pitch) >= 16;
  by_dtype(dtype, [&](auto t) {
    auto go = [&](auto v) {
      if (q) gmm::gmm_quantize_fp8_cols_kernel<decltype(t), v.value, true><<<grid, gmm::kQ8Threads, 0, stream>>>(p);
      else gmm::gmm_quantize_fp8_cols_kernel<decltype(t), v.value, false><<<grid, gmm::kQ8Threads, 0, stream>>>(p);
    };
    if (vec) go(std::true_type()); else go(std::false_type());
  });
  return launch_status("launch of the 8-bit column quantisation kernel");
}

}  // extern "C"
