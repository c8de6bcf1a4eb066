// The variants of the router's kernels and the rule that picks one, for one type of the logits.
#pragma once

#include <algorithm>
#include <type_traits>

#include "gmm_choose_launch.h"

namespace gmm {
namespace host {

// Warps a CTA: fewer where a warp's `smem` bytes (64-bit keys of every expert, rows of the
// gradient) and the kernel's own `own` would not fit the default 48 KB.
constexpr size_t kChooseSmem = 48 * 1024;
inline int choose_warps(size_t smem, size_t own) {
  return static_cast<int>(std::max<size_t>(1, std::min<size_t>(gmm::kChooseWarps, (kChooseSmem - own) / std::max<size_t>(1, smem))));
}

// The largest share of a token's experts that one of eight lanes takes where there is a bias.
constexpr int kScoreShare8 = 16;

template <class T, int L, int V>
int launch_choose(gmm::ChooseParams p, bool vec, bool score, bool grad, cudaStream_t stream) {
  for (p.group_lanes = L; p.group_lanes > 1 && p.group_lanes * p.groups > L;) p.group_lanes /= 2;
  const long long warps = (p.num_tokens + 32 / L - 1) / (32 / L);
  const bool dense = p.scoring == GMM_SCORE_SOFTMAX && !p.renormalise;
  const size_t per_warp = grad ? static_cast<size_t>(32) * V * 4 : (score ? static_cast<size_t>(32 / L) * p.num_experts * 8 : 0);
  const size_t own = grad ? 0 : 16 * static_cast<size_t>(score ? gmm::kChooseSlots<T, L, true> : gmm::kChooseSlots<T, L, false>);
  // One warp always fits: the keys of a whole warp's token, or of 32 / L tokens of as many experts as the layout is taken for.
  static_assert(16 * gmm::kChooseSlots<T, 32, true> + 8 * gmm::kRouteMaxExperts <= kChooseSmem, "a token's keys");
  static_assert(16 * gmm::kChooseSlots<T, 8, true> + 32 / 8 * 8 * (8 * kScoreShare8) <= kChooseSmem, "four tokens' keys");
  static_assert(32 * gmm::kChooseMaxPerLane * 4 <= kChooseSmem, "a row of the gradient");
  const int wc = choose_warps(per_warp, own);
  const unsigned grid = static_cast<unsigned>((warps + wc - 1) / wc), threads = 32u * wc;
  const size_t smem = per_warp * wc;
  auto go = [&](auto vec_c) {
    constexpr bool kVec = decltype(vec_c)::value;
    if (grad) {
      if (dense) gmm::gmm_route_grad_kernel<T, L, V, kVec, true><<<grid, threads, smem, stream>>>(p);
      else gmm::gmm_route_grad_kernel<T, L, V, kVec, false><<<grid, threads, smem, stream>>>(p);
    } else if constexpr (L == 32 || V <= kScoreShare8) {
      if (score) gmm::gmm_route_kernel<T, L, V, kVec, true><<<grid, threads, smem, stream>>>(p);
      else gmm::gmm_route_kernel<T, L, V, kVec, false><<<grid, threads, smem, stream>>>(p);
    } else {
      gmm::gmm_route_kernel<T, L, V, kVec, false><<<grid, threads, smem, stream>>>(p);
    }
  };
  if constexpr (V * sizeof(T) <= 128) {
    if (vec) go(std::true_type()); else go(std::false_type());
  } else {
    go(std::false_type());
  }
  return launch_status(grad ? "launch of the route gradient kernel" : "launch of the route kernel");
}

// The most logits that one of a token's `lanes` holds.
inline int choose_share(const gmm::ChooseParams &p, int lanes) {
  int per_group = lanes;
  while (per_group > 1 && per_group * p.groups > lanes) per_group /= 2;
  return per_group * p.groups > lanes ? 1 << 30 : (p.group_size + per_group - 1) / per_group;
}

template <class T>
int run_choose(gmm_ctx *h, const gmm::ChooseParams &p, bool score, bool grad, cudaStream_t stream) {
  // Lanes a token: a whole warp has the shortest way through one token; with many tokens eight
  // lanes leave fewer of them idle.
  const bool many = p.num_tokens > 16 * h->num_sms && p.top_k <= 8;
  const int need8 = choose_share(p, 8), need = choose_share(p, 32);
  const unsigned long long at = reinterpret_cast<uintptr_t>(p.logits) | static_cast<unsigned long long>(p.logits_pitch) |
                                reinterpret_cast<uintptr_t>(p.d_logits) | static_cast<unsigned long long>(p.d_pitch);
  auto vec = [&](int v) { return p.group_size % v == 0 && at % std::min<size_t>(16, v * sizeof(T)) == 0; };
  if (many && need8 <= 8) return launch_choose<T, 8, 8>(p, vec(8), score, grad, stream);
  if (many && need8 <= 16) return launch_choose<T, 8, 16>(p, vec(16), score, grad, stream);
  if (many && need8 <= 32 && !score) return launch_choose<T, 8, 32>(p, vec(32), score, grad, stream);
  if (need <= 2) return launch_choose<T, 32, 2>(p, vec(2), score, grad, stream);
  if (need <= 4) return launch_choose<T, 32, 4>(p, vec(4), score, grad, stream);
  if (need <= 8) return launch_choose<T, 32, 8>(p, vec(8), score, grad, stream);
  if (need <= 16) return launch_choose<T, 32, 16>(p, vec(16), score, grad, stream);
  if (need <= 32) return launch_choose<T, 32, 32>(p, vec(32), score, grad, stream);
  return launch_choose<T, 32, gmm::kChooseMaxPerLane>(p, false, score, grad, stream);
}

}  // namespace host
}  // namespace gmm
