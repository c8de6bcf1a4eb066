// Host side of a router's choice and its gradient (gmm_route, gmm_route_grad): argument checks.
#include <cmath>

#include "gmm_choose_launch.h"

namespace {

using namespace gmm::host;

int check_route(gmm_ctx *h, gmm::ChooseParams &p, const void *logits, long long logits_stride, int num_tokens, int top_k,
                int dtype, const gmm_route_options *o) {
  if (!h || !o || num_tokens < 0 || top_k < 1 || logits_stride < 0 || !dtype_bytes(dtype)) return GMM_ERR_INVALID_ARG;
  const int E = h->num_experts, es = dtype_bytes(dtype);
  if (top_k > E || (o->scoring != GMM_SCORE_SOFTMAX && o->scoring != GMM_SCORE_SIGMOID)) return GMM_ERR_INVALID_ARG;
  if (!(o->scale > 0.0f) || !(o->scale < INFINITY)) return GMM_ERR_INVALID_ARG;
  if (top_k > gmm::kRouteMaxTopK || E > gmm::kRouteMaxExperts || static_cast<long long>(num_tokens) * top_k > (1ll << 30))
    return GMM_ERR_UNSUPPORTED;
  if (num_tokens > 0 && (!logits || !aligned_to(logits, es))) return GMM_ERR_INVALID_ARG;
  std::memset(&p, 0, sizeof(p));
  p.logits = static_cast<const uint8_t *>(logits);
  p.logits_pitch = logits_stride * es;
  p.num_tokens = num_tokens;
  p.num_experts = E;
  p.top_k = top_k;
  p.scoring = o->scoring;
  p.groups = 1;
  p.group_size = E;
  p.top_groups = 1;
  p.group_top = 1;
  p.renormalise = o->renormalise != 0;
  p.scale = o->scale;
  p.status = reinterpret_cast<uint32_t *>(h->ws);
  return GMM_OK;
}

int run_choose_dtype(gmm_ctx *h, const gmm::ChooseParams &p, int dtype, bool score, bool grad, cudaStream_t stream) {
  DeviceGuard guard(h->device);
  switch (dtype) {
    case GMM_DTYPE_BF16: return run_choose_bf16(h, p, score, grad, stream);
    case GMM_DTYPE_FP16: return run_choose_fp16(h, p, score, grad, stream);
    default: return run_choose_fp32(h, p, score, grad, stream);
  }
}

}  // namespace

extern "C" {

int gmm_route(gmm_handle_t h, int32_t *slot_experts, float *weights, const void *logits, long long logits_stride,
              const float *bias, int num_tokens, int top_k, int dtype, const gmm_route_options *options,
              cudaStream_t stream) {
  static_assert(GMM_SCORE_SOFTMAX == gmm::kScoreSoftmax && GMM_SCORE_SIGMOID == gmm::kScoreSigmoid,
                "score functions of the C ABI and the kernel agree");
  gmm::ChooseParams p;
  int rc = check_route(h, p, logits, logits_stride, num_tokens, top_k, dtype, options);
  if (rc) return rc;
  const int E = h->num_experts, groups = options->expert_groups;
  if (groups < 1 || E % groups || options->top_groups < 1 || options->top_groups > groups ||
      (options->group_top != 1 && options->group_top != 2) || options->group_top > E / groups ||
      top_k > options->top_groups * (E / groups) || !aligned_to(bias, 4))
    return GMM_ERR_INVALID_ARG;
  if (groups > gmm::kChooseMaxGroups) return GMM_ERR_UNSUPPORTED;
  if (num_tokens > 0 && (!slot_experts || !weights || !aligned_to(slot_experts, 4) || !aligned_to(weights, 4)))
    return GMM_ERR_INVALID_ARG;
  p.bias = bias;
  p.bias_vec = aligned16(bias);
  p.ids = slot_experts;
  p.weights = weights;
  if (options->top_groups < groups) {   // else every group is kept
    p.groups = groups;
    p.group_size = E / groups;
    int lanes = 1;   // of a group, in a whole warp
    while (2 * lanes * groups <= 32) lanes *= 2;
    p.top_groups = options->top_groups;
    p.group_top = options->group_top;
    if ((p.group_size + lanes - 1) / lanes > gmm::kChooseMaxPerLane) return GMM_ERR_UNSUPPORTED;
  }
  if (num_tokens == 0) return GMM_OK;
  return run_choose_dtype(h, p, dtype, p.bias != nullptr, false, stream);
}

int gmm_route_grad(gmm_handle_t h, void *d_logits, long long d_logits_stride, const float *d_weights,
                   const int32_t *slot_experts, const void *logits, long long logits_stride, int num_tokens, int top_k,
                   int dtype, const gmm_route_options *options, cudaStream_t stream) {
  gmm::ChooseParams p;
  int rc = check_route(h, p, logits, logits_stride, num_tokens, top_k, dtype, options);
  if (rc) return rc;
  if (num_tokens == 0) return GMM_OK;
  const int es = dtype_bytes(dtype);
  if (!d_logits || !d_weights || !slot_experts || !aligned_to(d_logits, es) || !aligned_to(d_weights, 4) ||
      !aligned_to(slot_experts, 4) || d_logits_stride < 0)
    return GMM_ERR_INVALID_ARG;
  if (d_logits_stride < h->num_experts && num_tokens > 1) return GMM_ERR_INVALID_ARG;   // rows of the output overlap
  p.ids = const_cast<int32_t *>(slot_experts);
  p.weights = const_cast<float *>(d_weights);
  p.d_logits = static_cast<uint8_t *>(d_logits);
  p.d_pitch = d_logits_stride * es;
  return run_choose_dtype(h, p, dtype, false, true, stream);
}

}  // extern "C"
