// The launches of the router's kernels, one translation unit for each type of the logits.
#pragma once

#include "gmm_choose.cuh"
#include "gmm_host.h"

namespace gmm {
namespace host {

int run_choose_bf16(gmm_ctx *h, const gmm::ChooseParams &p, bool score, bool grad, cudaStream_t stream);
int run_choose_fp16(gmm_ctx *h, const gmm::ChooseParams &p, bool score, bool grad, cudaStream_t stream);
int run_choose_fp32(gmm_ctx *h, const gmm::ChooseParams &p, bool score, bool grad, cudaStream_t stream);

}  // namespace host
}  // namespace gmm
