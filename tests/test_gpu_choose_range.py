"""The router's choice and its gradient at the ends of what fp32 holds, against 64 bits: scores that leave the normal
range, and group sums that fp32 rounds coarsely or cannot hold.  Tolerances as in test_gpu_choose.py."""
import numpy as np
import pytest

from tests import choose_util as cu
from tests.test_gpu_choose import _check, _check_grad, _dtype, handles  # noqa: F401

pytestmark = pytest.mark.gpu


def _t():
    import torch
    return torch


def _cuda(x, dtype="fp32"):
    return _t().from_numpy(np.asarray(x, np.float32)).to(_dtype(dtype)).cuda()


@pytest.mark.parametrize("T", [40, 2561])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_sums_of_scores_below_the_normal_range(handles, scoring, dtype, T):  # noqa: F811
    """Groups' sums of two scores around 2^-126, where fp32 loses bits or the whole score."""
    rng = np.random.default_rng([T, 31])
    x = -87.5 + rng.uniform(-0.7, 0.7, (T, 32)) if scoring == "sigmoid" else rng.uniform(-104.0, -85.0, (T, 32))
    if scoring == "softmax":
        x[::2] = rng.uniform(-104.5, -99.0, x[::2].shape)        # a few bits are left of subnormal scores
        x[:, 5] = 0.0
    _check(handles(32), _cuda(x, dtype), 8, scoring=scoring, groups=8, top_groups=4, group_top=2)


def test_a_score_that_32_bits_drop(handles):  # noqa: F811
    """exp(-87.5) is below 2^-126, and the second group's sum is the larger one only with it."""
    x = [[-87.0, -87.0, -90.0, -90.0, -86.5, -87.5, -90.0, -90.0]]
    ids, _ = _check(handles(8), _cuda(x, "bf16"), 2, scoring="sigmoid", groups=2, top_groups=1, group_top=2)
    assert ids.tolist() == [[4, 5]]
