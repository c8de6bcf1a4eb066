#include "gmm_choose_launch.cuh"

namespace gmm {
namespace host {

int run_choose_fp16(gmm_ctx *h, const gmm::ChooseParams &p, bool score, bool grad, cudaStream_t stream) {
  return run_choose<__half>(h, p, score, grad, stream);
}

}  // namespace host
}  // namespace gmm
