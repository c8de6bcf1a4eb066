"""The weight gradient of one group so long that its contraction takes longer than a wait's limit."""
import os

import numpy as np
import pytest

from tests import fp8_util as fu

pytestmark = pytest.mark.gpu


def test_a_tile_that_outlasts_the_limit_of_a_wait():
    """2^24 rows are 131072 stages of one tile, some 30 ms; a limit of 5 ms stands for the default one of 2 s, which a
    group of 2^30 rows passes.  Nothing is stuck: the call completes."""
    import torch
    from ragged_matmul_gb300 import binding
    G, N, K, R, n = 1, 16, 16, 1 << 24, 200
    h = binding.gmm_create(G, 0)
    P = fu.pitch(R, G)
    d, a = (torch.zeros((w, P), dtype=torch.uint8, device="cuda") for w in (N, K))
    rng = np.random.default_rng(5)
    codes = [rng.choice([0x38, 0xB8, 0x40], (w, n)).astype(np.uint8) for w in (N, K)]        # 1, -1, 2: sums are exact
    at = torch.from_numpy(np.linspace(0, R - 1, n).astype(np.int64)).cuda()
    for x, q in zip((d, a), codes):
        x[:, at] = torch.from_numpy(q).cuda()
    ones = lambda w: torch.full((P // 128, w), 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    d_s, a_s, off = ones(N), ones(K), torch.tensor([0, R], dtype=torch.int32, device="cuda")
    out = torch.full((G, N, K), float("nan"), device="cuda")
    binding.gmm_weight_grad_fp8(h, out, d, d_s, a, a_s, off)       # with the limit that users have
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    out.fill_(float("nan"))
    os.environ["GMM_TEST_WAIT_LIMIT_NS"] = "5000000"
    try:
        start.record()
        binding.gmm_weight_grad_fp8(h, out, d, d_s, a, a_s, off)
        end.record()
        status = binding.gmm_query_status(h)
    finally:
        del os.environ["GMM_TEST_WAIT_LIMIT_NS"]
    assert status == binding.GMM_OK
    np.testing.assert_array_equal(out[0].double().cpu().numpy(), fu.E4M3[codes[0]] @ fu.E4M3[codes[1]].T)
    assert start.elapsed_time(end) > 8.0, "shorter than the limit and one suspension: this shows nothing"
    binding.gmm_destroy(h)
