#include "gmm_choose_launch.cuh"

namespace gmm {
namespace host {

int run_choose_fp32(gmm_ctx *h, const gmm::ChooseParams &p, bool score, bool grad, cudaStream_t stream) {
  return run_choose<float>(h, p, score, grad, stream);
}

}  // namespace host
}  // namespace gmm
