"""Counts that are no whole numbers are refused by the router's and the 8-bit quantisers' calls, not cut off."""
import numpy as np
import pytest

from ragged_matmul_gb300 import binding


def test_route_options():
    for kw in (dict(groups=2.5), dict(groups=4, top_groups=1.5), dict(groups=4, top_groups=2, group_top=1.9)):
        with pytest.raises(ValueError, match="whole number"):
            binding._route_options("softmax", True, 1.0, **kw)
    o = binding._route_options("softmax", True, 1.0, np.int64(8), 4.0, np.int32(2))._obj
    assert (o.expert_groups, o.top_groups, o.group_top) == (8, 4, 2)


@pytest.mark.gpu
def test_top_k_of_the_quantisers():
    import torch
    h = binding.gmm_create(2, 0)
    x = torch.ones((3, 128), device="cuda")
    slots, off = torch.arange(6, dtype=torch.int32, device="cuda"), torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    P = binding.fp8_cols_pitch(6, 2)
    for top_k in (2, 2.0, np.int64(2)):
        binding.gmm_quantize_fp8(h, u8(6, 128), torch.zeros((6, 1), device="cuda"), x, row_slots=slots, top_k=top_k)
        binding.gmm_quantize_fp8_cols(h, u8(128, P), u8(P // 128, 128), x, off, row_slots=slots, top_k=top_k)
    with pytest.raises(ValueError, match="whole number"):
        binding.gmm_quantize_fp8(h, u8(6, 128), torch.zeros((6, 1), device="cuda"), x, row_slots=slots, top_k=2.5)
    with pytest.raises(ValueError, match="whole number"):
        binding.gmm_quantize_fp8_cols(h, u8(128, P), u8(P // 128, 128), x, off, row_slots=slots, top_k=2.5)
    assert binding.gmm_query_status(h) == binding.GMM_OK
    binding.gmm_destroy(h)
