"""Host-side argument checks of the dispatch, combine and 4-bit floating point calls: they
return before touching a GPU, so a null handle or a bad argument is answered on any machine."""
import ctypes

import pytest

from ragged_matmul_gb300 import binding
from ragged_matmul_gb300 import build as gbuild


@pytest.fixture(scope="module")
def lib():
    return binding.load_library(gbuild.build())


P = ctypes.c_void_p
BAD = binding.GMM_ERR_INVALID_ARG


def test_null_handles(lib):
    p = P(16)
    assert lib.gmm_dispatch(None, p, p, p, None, p, None, 0, 4, 2, 8, 0, None) == BAD
    assert lib.gmm_combine(None, p, 8, p, 8, p, p, 4, 2, 8, 0, None) == BAD
    assert lib.gmm_combine_grad(None, p, p, p, 8, p, 8, p, p, 4, 2, 8, 0, None) == BAD
    assert lib.gmm_quantize_fp4(None, p, p, p, 64, 4, None, 1, None, 4, 64, 0, 0, None) == BAD
    assert lib.gmm_dequantize_fp4(None, p, 64, p, p, None, 4, 64, 0, 0, None) == BAD
    assert lib.gmm_run_fp4(None, p, p, p, p, p, p, 1, 64, 64, p, p, 0, None, None, None, None) == BAD
    assert lib.gmm_run_fp4(None, p, p, p, p, p, p, 0, 64, 64, p, p, 0, None, None, None, None) == BAD


def test_scale_pitch():
    for fmt, block in (("nvfp4", 16), ("mxfp4", 32)):
        for K in (32, 64, 256, 512, 544, 4096, 7168):
            pitch = binding.fp4_scale_pitch(K, fmt)
            assert pitch % 16 == 0 and K // block <= pitch < K // block + 16
    with pytest.raises(ValueError):
        binding.fp4_scale_pitch(64, "fp4")


def test_tensors_on_another_device_are_refused():
    import torch
    x = torch.zeros((4, 64))
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    h = binding.Handle(None, 0, 2)
    for call in (lambda: binding.gmm_quantize_fp4(h, u8(4, 32), u8(4, 16), x),
                 lambda: binding.gmm_dequantize_fp4(h, x, u8(4, 32), u8(4, 16)),
                 lambda: binding.gmm_combine(h, x, x, i32(4, 1)),
                 lambda: binding.gmm_combine_grad(h, x, None, x, None, i32(4, 1)),
                 lambda: binding.gmm_dispatch(h, i32(3), i32(4, 1), i32(4), i32(4, 1))):
        with pytest.raises(ValueError, match="cuda:0"):
            call()
    with pytest.raises(TypeError):
        binding.gmm_combine(h, x, x, [1.0])


def test_the_gradient_states_that_its_rows_are_distinct():
    """Each row of d_rows has one writer only if no two slots name it: a condition of the call that the
    header and the binding both state."""
    import os
    with open(os.path.join(os.path.dirname(gbuild.PKG_DIR), "include", "gmm.h")) as f:
        header = f.read()
    comment = header[header.index(" * The gradient of gmm_combine:"):header.index("int gmm_combine_grad(")]
    for text in (comment, binding.gmm_combine_grad.__doc__):
        assert "must be distinct" in text and "not checked" in text
