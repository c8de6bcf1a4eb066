"""Blocks of zeros of either sign have zero codes in every form (s = 0 gives q = 0); a -0 beside other values keeps its sign."""
import numpy as np
import pytest

from tests import fp8_util as fu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("pad", [0, 1])
def test_negative_zeros(dtype, pad):
    import torch
    from ragged_matmul_gb300 import binding
    R, K = 300, 144
    off = [0, 130, 130, 300]
    h = binding.gmm_create(4, 0)
    wide = torch.zeros((R, K + pad), dtype=getattr(torch, dtype), device="cuda")
    x = wide[:, pad:]
    x[::3] = -0.0
    x[:, 5] = -0.0
    x[7, 9], x[200, 130] = 1.5, -2.0
    u8 = lambda *s: torch.full(s, 0x5A, dtype=torch.uint8, device="cuda")  # noqa: E731
    P = binding.fp8_cols_pitch(R, 3)
    q_t, t_s, q, s = u8(K, P), u8(P // 128, K), u8(R, K), torch.full((R, 2), 7.0, device="cuda")
    binding.gmm_quantize_fp8_cols(h, q_t, t_s, x, torch.tensor(off, dtype=torch.int32, device="cuda"), q=q, scales=s)
    q2, s2 = u8(R, K), torch.full((R, 2), 7.0, device="cuda")
    binding.gmm_quantize_fp8(h, q2, s2, x)
    assert binding.gmm_query_status(h) == binding.GMM_OK
    xs = x.float().cpu().numpy()
    want_q, want_s = fu.rows(xs, False)
    for got_q, got_s in ((q, s), (q2, s2)):
        np.testing.assert_array_equal(got_q.cpu().numpy(), want_q)
        np.testing.assert_array_equal(got_s.double().cpu().numpy(), want_s)
    got_t, got_ts = q_t.cpu().numpy(), t_s.cpu().numpy()
    for g in range(3):
        for b, r in enumerate(range(off[g], off[g + 1], 128)):
            part = xs[r:min(r + 128, off[g + 1])]
            scale = fu.scale_of(np.abs(part).max(0), True)
            want = np.zeros((128, K), np.uint8)
            want[:len(part)] = fu.codes(part, scale[None, :])
            at = off[g] // 128 + g + b
            np.testing.assert_array_equal(got_t[:, at * 128:at * 128 + 128], want.T)
            np.testing.assert_array_equal(got_ts[at], np.where(scale == 0, 0, np.log2(np.where(scale == 0, 1, scale)) + 127).astype(np.uint8))
    w = torch.full((1, 200, K), -0.0, dtype=x.dtype, device="cuda")
    w[0, 199, 143] = 1.0
    wq, ws = u8(1, 200, K), torch.full((1, 2, 2), 7.0, device="cuda")
    for pow2 in (False, True):
        binding.gmm_quantize_fp8_tiles(h, wq, ws, w, pow2=pow2)
        assert ((ws == 0).view(-1).tolist()) == [True, True, True, False]
        assert (wq[0, :128] == 0).all() and (wq[0, 128:, :128] == 0).all()
        assert (wq[0, 128:199, 128:] == 0x80).all() and wq[0, 199, 143] in (0x7E, 0x78)
    binding.gmm_destroy(h)
