// Shared host side of the C ABI's translation units: the handle, error reports, tensor-map
// encoding and the checks that several calls make.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "gmm.h"

// One launch configuration per kernel variant.  The grouped kernel keeps its group
// prefix (G + 1 words) in dynamic shared memory after the rings, so its configuration is
// chosen per launch: the first of its candidate layouts (in order of preference) whose
// minimum ring fits beside the prefix of that G, with as many stages as the rest holds.
struct gmm_variant {
  int stages = 0;           // depth of the W+T stage ring (grouped kernel: its first layout, one group)
  size_t smem = 0;          // dynamic shared memory of every launch
  size_t budget = 0;        // of which the kernel may use (the rest only keeps one CTA per SM)
  size_t stage_bytes = 0;   // grouped kernel: one stage of the ring
  int stage_mult = 1;       // grouped kernel: the ring depth is a multiple of this (4-bit: kAStages)
  int min_stages = 2;       // grouped kernel: the shallowest ring it runs with
  int layouts = 1;          // grouped kernel: candidate layouts, in order of preference
  size_t fixed[2] = {};     // per layout: everything but the stage ring and the prefix
  int q_stages[2] = {};     // per layout, 4-bit: packed-ring slots
  int grid = 0;             // CTAs: the SM count, or (pairs) twice the co-resident clusters of two
};

struct gmm_ctx {
  int device = 0;
  int num_experts = 0;
  int num_sms = 0;
  gmm_variant var[2][2];          // [4-bit][pair]
  gmm_variant var_fp8[2];         // e4m3 kernels, [pair]
  gmm_variant var_fp8_block;      // e4m3 with per-K-block scales (one CTA per tile)
  gmm_variant var_fp4[2];         // 4-bit floating point, [mxfp4], CTA pairs; grid 0: does not fit
  gmm_variant var_weight_grad[2]; // weight gradient on e4m3 operands, [bf16 result], CTA pairs; grid 0: does not fit
  int smem_per_sm = 0;            // shared memory of one SM (a launch reserves more than half: one CTA per SM)
  bool debug = false;             // GMM_DEBUG was set when the handle was created
  int use_pairs = 1;              // bf16 path: 1 = CTA-pair kernels (cta_group::2), 0 = one CTA per tile
  int use_pairs_int4 = 1;         // 4-bit path: the same
  uint8_t *ws = nullptr;          // [status word | per-CTA tensor-map slots | zero offsets | chunk counts]
  size_t ws_bytes = 0;
  const uint32_t *zero_offsets = nullptr;   // in ws: a_offsets of a call without rows, never written
  uint32_t *route_counts = nullptr;   // in ws; null with more experts than gmm_dispatch takes
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  PFN_cuMemsetD32Async_v3020 memset32 = nullptr;   // value writes that a captured CUDA graph replays as such
};

namespace gmm {
namespace host {

struct DeviceGuard {
  int prev = -1;
  bool switched = false;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) == cudaSuccess && prev != dev) switched = cudaSetDevice(dev) == cudaSuccess;
  }
  ~DeviceGuard() {
    if (switched) cudaSetDevice(prev);
  }
};

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// GMM_DEBUG=1: report the CUDA call behind a GMM_ERR_CUDA on stderr, and (when set as
// a handle is created) the handle's ring depths and each of its grouped-kernel launches'
// layout (diagnostics only).
inline void debug_report(const char *what, int code, const char *msg) {
  static const bool on = getenv("GMM_DEBUG") != nullptr;
  if (on) fprintf(stderr, "gmm: %s failed: %d %s\n", what, code, msg ? msg : "");
}

// A driver call.  It needs a current context, which a thread that has made no runtime call but
// cudaGetDevice lacks (autograd runs a backward pass on such a thread): the device's primary
// context is then made current, and the call made again.
template <class Call>
inline CUresult with_context(gmm_ctx *h, Call call) {
  const CUresult r = call();
  if (r != CUDA_ERROR_INVALID_CONTEXT) return r;
  DeviceGuard guard(h->device);
  if (cudaSetDevice(h->device) != cudaSuccess) {
    cudaGetLastError();
    return r;
  }
  return call();
}

inline int encode_map(gmm_ctx *h, CUtensorMap *m, CUtensorMapDataType type, uint32_t rank, const void *base,
               const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box,
               CUtensorMapSwizzle swizzle) {
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = with_context(h, [&] {
    return h->encode(m, type, rank, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  });
  if (r != CUDA_SUCCESS) debug_report("cuTensorMapEncodeTiled", static_cast<int>(r), nullptr);
  return r == CUDA_SUCCESS ? GMM_OK : GMM_ERR_CUDA;
}

inline int dtype_bytes(int dtype) {
  switch (dtype) {
    case GMM_DTYPE_BF16:
    case GMM_DTYPE_FP16: return 2;
    case GMM_DTYPE_FP32: return 4;
    default: return 0;
  }
}

inline bool aligned_to(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

inline int launch_status(const char *what) {
  const cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess) return GMM_OK;
  debug_report(what, static_cast<int>(err), cudaGetErrorString(err));
  return GMM_ERR_CUDA;
}

void configure_weight_grad(gmm_variant (&vars)[2], int optin, int sm_smem, int device_optin, int num_sms);

}  // namespace host
}  // namespace gmm
