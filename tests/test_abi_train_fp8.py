"""Host-side argument checks of the router's choice, the 8-bit quantisers and the weight gradient: they return
before touching a GPU, so a null handle or a bad argument is answered on any machine."""
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
    o = ctypes.byref(binding.GmmRouteOptions(0, 1, 1, 1, 1, 1.0))
    assert lib.gmm_route(None, p, p, p, 8, None, 4, 2, 0, o, None) == BAD
    assert lib.gmm_route_grad(None, p, 8, p, p, p, 8, 4, 2, 0, o, None) == BAD
    assert lib.gmm_quantize_fp8(None, p, p, p, 64, 4, None, 1, 4, 64, 0, 0, None) == BAD
    assert lib.gmm_quantize_fp8_tiles(None, p, p, p, 2, 64, 64, 0, 0, None) == BAD
    assert lib.gmm_quantize_fp8_cols(None, p, p, None, None, p, 64, 4, None, 1, p, 2, 4, 64, 0, None) == BAD
    assert lib.gmm_weight_grad_fp8(None, p, p, p, p, p, p, 2, 4, 64, 64, 2, 0, None) == BAD


def test_cols_pitch():
    """Each group's blocks lie behind those of the group before it, and inside the pitch."""
    import random
    rng = random.Random(0)
    for _ in range(200):
        loads = [rng.choice((0, 1, 127, 128, 129, rng.randrange(1000))) for _ in range(rng.randrange(1, 20))]
        first = rng.choice((0, 0, 5, 128, 300))
        behind = rng.choice((0, 100))
        end, r = 0, first
        for g, n in enumerate(loads):
            base = r // 128 + g
            assert base >= end
            end = base + -(-n // 128)
            r += n
        assert end * 128 <= binding.fp8_cols_pitch(r + behind, len(loads))


def test_tensors_on_another_device_are_refused():
    import torch
    x = torch.zeros((4, 64))
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    h = binding.Handle(None, 0, 64)
    for call in (lambda: binding.gmm_route(h, i32(4, 2), torch.zeros((4, 2)), x),
                 lambda: binding.gmm_route_grad(h, x, torch.zeros((4, 2)), i32(4, 2), x),
                 lambda: binding.gmm_quantize_fp8(h, u8(4, 64), torch.zeros((4, 1)), x),
                 lambda: binding.gmm_quantize_fp8_tiles(h, u8(1, 4, 64), torch.zeros((1, 1, 1)), x[None]),
                 lambda: binding.gmm_quantize_fp8_cols(h, u8(64, 128), u8(1, 64), x, i32(2)),
                 lambda: binding.gmm_weight_grad_fp8(h, torch.zeros((1, 64, 64)), u8(64, 128), u8(1, 64), u8(64, 128), u8(1, 64), i32(2))):
        with pytest.raises(ValueError, match="cuda:0"):
            call()
    with pytest.raises(TypeError):
        binding.gmm_route(h, i32(4, 2), torch.zeros((4, 2)), [1.0])


def test_options_are_the_headers():
    """The structure that the binding passes has the header's fields in its order."""
    import os
    import re
    with open(os.path.join(gbuild.INCLUDE_DIR, "gmm.h")) as f:
        body = re.search(r"typedef struct gmm_route_options \{(.*?)\}", f.read(), flags=re.S).group(1)
    fields = re.findall(r"(int|float) (\w+);", body)
    types = {"int": ctypes.c_int, "float": ctypes.c_float}
    assert [(n, types[t]) for t, n in fields] == list(binding.GmmRouteOptions._fields_)
    with pytest.raises(ValueError):
        binding._route_options("relu", True, 1.0)


def test_options_are_kept_by_value():
    """A setting given as a tensor counts with the value that it has at the call."""
    import torch
    scale, groups = torch.tensor(1.5), torch.tensor(4)
    first = binding._route_options("softmax", True, scale, groups, 2)._obj
    scale.fill_(2.5)
    groups.fill_(8)
    o = binding._route_options("softmax", True, scale, groups, 2)._obj
    assert (first.scale, first.expert_groups) == (1.5, 4) and (o.scale, o.expert_groups) == (2.5, 8)
    for scoring in (None, [], 2, 1.0):
        with pytest.raises(ValueError):
            binding._route_options(scoring, True, 1.0)


def test_reference_of_the_choice():
    """The tests' own reference on an example by hand."""
    import numpy as np

    from tests import choose_util as cu
    x = np.array([[0.0, 2.0, 1.0, -np.inf, 2.0, -1.0]])
    ids, w = cu.choose(x, 3, scoring="softmax")
    assert ids.tolist() == [[1, 4, 2]]
    np.testing.assert_allclose(w, np.array([[1, 1, np.exp(-1)]]) / (2 + np.exp(-1)))
    ids, _ = cu.choose(x, 3, scoring="sigmoid", bias=[1.0, 0, 0, 5, 0, 0])
    assert ids.tolist() == [[0, 1, 4]]
    ids, w = cu.choose(x, 3, scoring="sigmoid", groups=3, top_groups=1, group_top=2)      # group keys 1.38, 0.73, 1.15
    assert ids.tolist() == [[1, 0, -1]] and w[0, 2] == 0


def test_reference_of_the_quantisers():
    import numpy as np

    from tests import fp8_util as fu
    s = fu.scale_of(np.array([448.0, 449.0, 0.0, np.inf, 896.0, 2.0 ** -149]), True)
    np.testing.assert_array_equal(s, [1.0, 2.0, 0.0, np.nan, 2.0, 2.0 ** -127])
    x = np.zeros((1, 128), np.float32)
    x[0, :5] = (448, -1, 1.0625, 0.1, 17)
    q, s = fu.rows(x, True)
    np.testing.assert_allclose(fu.E4M3[q[0, :5]], (448, -1, 1.0, 0.1015625, 16))
    np.testing.assert_array_equal(fu.E4M3[q[0, 5:]], 0)
