"""The router's choice and its gradient at the ends of what fp32 holds, against 64 bits: scores that leave the normal
range, and group sums that fp32 rounds coarsely or cannot hold.  Tolerances as in test_gpu_choose.py."""
import numpy as np
import pytest

from tests import choose_util as cu
from tests.test_gpu_choose import _check, _dtype, _rtol, handles  # noqa: F401

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


def _check_sigmoid_grad(h, x, ids, dw, renormalise):
    """As _check_grad, for distinct chosen experts.  Its reference takes 1 - s of a score s near 1, which is off by up to
    2^-53: of a logit of 29, whose 1 - s is 2.5e-13, more than the bound allows.  Here it is the sigmoid of -x."""
    from ragged_matmul_gb300 import binding
    d = _t().full_like(x, float("nan"))
    binding.gmm_route_grad(h, d, dw, ids, x, scoring="sigmoid", renormalise=renormalise)
    assert binding.gmm_query_status(h) == binding.GMM_OK
    xs, at, g = x.double().cpu().numpy(), ids.cpu().numpy(), dw.double().cpu().numpy()
    xj = np.take_along_axis(xs, at, 1)
    s, rest = 1.0 / (1.0 + np.exp(-xj)), 1.0 / (1.0 + np.exp(xj))
    if renormalise:
        u = s / s.sum(1, keepdims=True)
        dj, mj = u * (g - (u * g).sum(1, keepdims=True)) * rest, u * (np.abs(g) + (u * np.abs(g)).sum(1, keepdims=True)) * rest
    else:
        dj, mj = g * s * rest, np.abs(g) * s * rest
    want, mag = np.zeros_like(xs), np.zeros_like(xs)
    np.put_along_axis(want, at, dj, 1)
    np.put_along_axis(mag, at, mj, 1)
    info = _t().finfo(x.dtype)
    bound = mag * 3 * (_rtol(xs, xs.shape[1]) + 2.0 ** -24 * 40)
    err = np.abs(d.double().cpu().numpy() - want)
    assert np.all(err <= bound + (np.abs(want) + bound) * info.eps / 2 + info.tiny * info.eps + 1e-37), float((err - bound).max())


@pytest.mark.parametrize("T", [40, 2561])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_weights_of_sigmoids_around_the_smallest_normal(handles, dtype, T):  # noqa: F811
    """Chosen logits on both sides of ln 2^-126 = -87.3: a score that fp32 would drop has up to a thousandth of the weight."""
    torch = _t()
    rng = np.random.default_rng([T, 32])
    x = rng.uniform(-100.0, -86.0, (T, 12))
    x[:, 3:6] = rng.uniform(-81.0, -60.0, (T, 3))
    x[::5, 4] = rng.uniform(-30.0, 30.0, len(range(0, T, 5)))
    x = _cuda(x, dtype)
    for renormalise in (True, False):
        ids, _ = _check(handles(12), x, 8, scoring="sigmoid", renormalise=renormalise)
        dw = torch.from_numpy(rng.standard_normal((T, 8)).astype(np.float32)).cuda()
        _check_sigmoid_grad(handles(12), x, ids, dw, renormalise)


@pytest.mark.parametrize("T", [3, 2561])
def test_a_group_left_out_whose_terms_cancel(handles, T):  # noqa: F811
    """The last group's fp32 sum is 1.5, below the two before it, of which the better one is kept; its exact sum, 1.5003,
    is the largest.  Its error is far above that of the others."""
    logit = np.log1p(4e-4 * 2) * np.array([0.0, 0.0, 0.0, 0.0, -9.0, -9.0, 1.0, 0.5])       # scores 0.5 + 2e-4, 0.5 + 1e-4
    bias = np.array([0.25, 0.2501, 0.25, 0.25005, 0.0, 0.0, 4096.0, -4095.5], np.float32)
    ids, _ = _check(handles(8), _cuda(np.tile(logit, (T, 1))), 2, bias=bias, scoring="sigmoid", groups=4, top_groups=1, group_top=2)
    assert (ids.cpu() == _t().tensor([6, 7], dtype=_t().int32)).all()


@pytest.mark.parametrize("T", [3, 2561])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_group_sums_that_fp32_cannot_hold(handles, scoring, T):  # noqa: F811
    """Biases of the type's lowest and largest value: a sum of two is a finite 64-bit number, not -infinity (no expert at
    all) and not equal to another such sum."""
    low, inf = float(np.finfo(np.float32).min), np.inf
    x = _cuda(np.random.default_rng([T, 33]).standard_normal((T, 8)))
    for bias in ([0, 0, -inf, -inf, low, low, -inf, -inf],         # the third group has experts
                 [0, 0, low, low, low, 0.99 * low, -inf, -inf],
                 [0, 0, low, low, 0.99 * low, 0.99 * low, 2, 2],
                 [-low, -0.9 * low, 0, 0, -low, -low, -0.9 * low, -low],
                 [low, low, low, -inf, -inf, -inf, low, low]):
        for top_groups in (1, 2, 3):
            _check(handles(8), x, 2, bias=np.array(bias, np.float32), scoring=scoring, groups=4, top_groups=top_groups, group_top=2)
            if top_groups > 1:
                _check(handles(8), x, 4, bias=np.array(bias, np.float32), scoring=scoring, groups=4, top_groups=top_groups, group_top=2)
