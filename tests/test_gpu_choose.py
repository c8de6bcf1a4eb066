"""A router's choice and its gradient on the GPU against 64 bits: every size of the kernels' layouts,
ties, masks, biases, groups, keys that 32 bits do not tell apart, special values, strides, graphs, streams.

Tolerance of the weights.  With d the largest difference of two logits that enters (|x - m|, or |x| of a
sigmoid), an exponential is off by 2^-24 d (its argument's rounding) and 2 ulp (2^-22); numerator and sum
have one each, a sum of n terms adds a rounding per step (n at most), quotient and scale 2^-24 each:
2^-24 (2 d + 8 + n + 2) relative.  The gradient adds products and one more sum of at most 33 terms to the
magnitudes that it sums, and a rounding to its type (half a step)."""
import numpy as np
import pytest

from tests import choose_util as cu

pytestmark = pytest.mark.gpu


def _t():
    import torch
    return torch


@pytest.fixture(scope="module")
def handles():
    from ragged_matmul_gb300 import binding
    cache = {}

    def get(E):
        if E not in cache:
            cache[E] = binding.gmm_create(E, 0)
        return cache[E]
    yield get
    for h in cache.values():
        binding.gmm_destroy(h)


def _dtype(name):
    torch = _t()
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _logits(rng, T, E, dtype, spread=1.5):
    torch = _t()
    return torch.from_numpy((spread * rng.standard_normal((T, E))).astype(np.float32)).to(_dtype(dtype)).cuda()


def _route(h, x, top_k, bias=None, stream=None, **kw):
    torch = _t()
    from ragged_matmul_gb300 import binding
    T = x.shape[0]
    ids = torch.full((T, top_k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, top_k), float("nan"), device="cuda")
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    binding.gmm_route(h, ids, w, x, bias=b, stream=stream, **kw)
    return ids, w


def _rtol(x, n):
    finite = np.where(np.isfinite(x), x, 0.0)
    d = min(float(np.max(finite) - np.min(finite)) + float(np.max(np.abs(finite))), 200.0) if finite.size else 0.0
    return 2.0 ** -24 * (2 * d + 10 + n)


def _check(h, x, top_k, bias=None, groups=1, top_groups=None, group_top=1, **kw):
    from ragged_matmul_gb300 import binding
    ids, w = _route(h, x, top_k, bias=bias, expert_groups=groups, top_groups=top_groups, group_top=group_top, **kw)
    status = binding.gmm_query_status(h)
    xs = x.double().cpu().numpy()
    want_ids, want_w = cu.choose(xs, top_k, bias=None if bias is None else np.asarray(bias, np.float32), groups=groups,
                                 top_groups=top_groups, group_top=group_top, **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    np.testing.assert_allclose(w.cpu().numpy(), want_w, rtol=_rtol(xs, xs.shape[1]), atol=1e-37)
    assert status == binding.GMM_OK
    return ids, w


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("E,top_k", [(1, 1), (2, 2), (7, 3), (8, 8), (64, 8), (65, 6), (100, 1), (128, 12), (161, 8), (256, 8),
                                     (257, 32), (500, 5), (1000, 8), (1024, 4), (4096, 8)])
@pytest.mark.parametrize("scoring,renormalise", [("softmax", True), ("sigmoid", False)])
def test_without_a_bias(handles, E, top_k, dtype, scoring, renormalise):
    rng = np.random.default_rng([E, top_k])
    for T in (1, 5):
        _check(handles(E), _logits(rng, T, E, dtype), top_k, scoring=scoring, renormalise=renormalise, scale=2.5)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E,top_k", [(5, 2), (64, 8), (63, 8), (128, 16), (100, 6)])
def test_many_tokens(handles, E, top_k, dtype):
    """From some thousand tokens on, several share a warp; their number leaves one warp partly empty."""
    rng = np.random.default_rng(E)
    _check(handles(E), _logits(rng, 2501, E, dtype), top_k, scoring="softmax", renormalise=False)
    _check(handles(E), _logits(rng, 2501, E, dtype), top_k, scoring="sigmoid", renormalise=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,top_k", [(3, 2), (64, 6), (160, 8), (256, 8), (1000, 32), (4096, 3)])
def test_with_a_bias(handles, E, top_k, scoring, dtype):
    rng = np.random.default_rng([E, 3])
    bias = np.round(50 * rng.standard_normal(E)) * 0.001
    for renormalise in (True, False):
        _check(handles(E), _logits(rng, 9, E, dtype), top_k, bias=bias, scoring=scoring, renormalise=renormalise)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups,top_k", [(64, 1, 1, 8), (30, 1, 1, 3), (100, 1, 1, 8), (256, 8, 4, 8), (120, 3, 2, 6),
                                                       (160, 8, 3, 8), (256, 1, 1, 8), (48, 6, 2, 4), (9, 3, 1, 3)])
def test_many_tokens_with_a_bias_or_groups(handles, E, groups, top_groups, top_k, scoring, dtype):
    """Several tokens a warp: near keys, ties, masks and NaN of one leave its neighbours alone."""
    torch = _t()
    from ragged_matmul_gb300 import binding
    rng = np.random.default_rng([E, groups])
    T = 2561
    x = _logits(rng, T, E, "fp32")
    x[5::9] = torch.from_numpy(rng.integers(-2, 3, (len(range(5, T, 9)), E)).astype(np.float32)).cuda()      # ties
    x[6::9] = 1.0 + 2.0 ** -22 * torch.from_numpy(rng.integers(-3, 4, (len(range(6, T, 9)), E)).astype(np.float32)).cuda()
    x[7::9, 3:] = -float("inf")
    x[8::18] = -float("inf")
    x = x.to(_dtype(dtype))
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
    for b in (None, bias, np.zeros(E)):
        for group_top in (1, 2):
            _check(handles(E), x, top_k, bias=b, scoring=scoring, groups=groups, top_groups=top_groups, group_top=group_top)
    x[40, E - 1] = float("nan")
    xs = x.double().cpu().numpy()
    ids, w = _route(handles(E), x, top_k, bias=bias, scoring=scoring, expert_groups=groups, top_groups=top_groups, group_top=2)
    assert binding.gmm_query_status(handles(E)) == binding.GMM_ERR_BAD_INPUT
    clean = [t for t in range(30, 50) if t != 40]
    want_ids, _ = cu.choose(xs[clean], top_k, bias=bias, scoring=scoring, groups=groups, top_groups=top_groups, group_top=2)
    np.testing.assert_array_equal(ids.cpu().numpy()[clean], want_ids)
    assert (ids[40] == -1).all() and (w[40] == 0).all()


@pytest.mark.parametrize("T", [70, 2561])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [24, 64, 256])
def test_biases_that_even_out_scores(handles, E, scoring, T):
    """Keys near one another whose logits and biases are not, and keys that 64 bits hold equal though the scores differ."""
    torch = _t()
    rng = np.random.default_rng([E, T])
    x = (1.5 * rng.standard_normal(E)).astype(np.float32)
    e = np.exp(x.astype(np.float64) - x.max())
    s = e / e.sum() if scoring == "softmax" else 1 / (1 + np.exp(-x.astype(np.float64)))
    rows = torch.from_numpy(x).cuda() + 2.0 ** -21 * torch.from_numpy(rng.integers(-2, 3, (T, E)).astype(np.float32)).cuda()
    for step in (0.0, 1e-7, 1e-6, 3e-5):
        _check(handles(E), rows, 8, bias=(1.0 - s + step * rng.integers(-9, 10, E)).astype(np.float32), scoring=scoring)
    far = torch.from_numpy((rng.uniform(-60, -50, (T, E))).astype(np.float32)).cuda()
    if scoring == "softmax":
        far[:, E // 2] = 0.0
    _check(handles(E), far, 8, bias=np.ones(E, np.float32), scoring=scoring, renormalise=False)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups,top_k", [(64, 1, 1, 8), (100, 1, 1, 5), (128, 1, 1, 8), (40, 8, 5, 8)])
def test_many_tokens_with_a_few_near_keys(handles, E, groups, top_groups, top_k, scoring):
    """Some keys more than a token's lanes, of which 32 bits do not tell all apart."""
    rng = np.random.default_rng([E, 5])
    T = 2561
    x = -3.0 + 0.1 * rng.standard_normal((T, E))
    for t in range(T):
        near = rng.permutation(E)[:rng.integers(top_k, 24)]
        x[t, near] = 1.0 + 2.0 ** -22 * rng.integers(-3, 4, len(near))
    x = _t().from_numpy(x.astype(np.float32)).cuda()
    for bias in (np.zeros(E), 2.0 ** -26 * rng.integers(-3, 4, E)):
        _check(handles(E), x, top_k, bias=bias.astype(np.float32), scoring=scoring, groups=groups, top_groups=top_groups, group_top=2)


@pytest.mark.parametrize("E", [1500, 1536, 2000, 2048, 4000])
def test_shared_memory_at_every_number_of_experts(handles, E):
    """The 64-bit keys of a token and the gradient's rows, where fewer warps share a block."""
    torch = _t()
    rng = np.random.default_rng(E)
    x = _logits(rng, 9, E, "fp32")
    ids, _ = _check(handles(E), x, 8, bias=np.full(E, 2.0), scoring="softmax", renormalise=False)
    _check_grad(handles(E), x, ids, torch.ones((9, 8), device="cuda"), scoring="softmax", renormalise=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("E,groups,top_groups,top_k", [(256, 8, 4, 8), (60, 3, 2, 6), (64, 32, 5, 10), (160, 5, 1, 8),
                                                       (8, 4, 3, 6), (1024, 4, 2, 8), (4096, 32, 3, 8)])
def test_groups(handles, E, groups, top_groups, top_k, group_top, with_bias, dtype):
    rng = np.random.default_rng([E, groups, group_top])
    bias = 0.05 * rng.standard_normal(E) if with_bias else None
    for scoring in ("sigmoid", "softmax"):
        _check(handles(E), _logits(rng, 11, E, dtype), top_k, bias=bias, scoring=scoring, groups=groups,
               top_groups=top_groups, group_top=group_top)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [None, "zeros", "steps"])
def test_ties_go_to_the_lowest_expert(handles, scoring, dtype, bias):
    torch = _t()
    rng = np.random.default_rng(4)
    E = 96
    b = None if bias is None else (np.zeros(E) if bias == "zeros" else rng.integers(0, 3, E) * 0.25)
    few = rng.integers(-2, 3, (40, E)).astype(np.float32)       # five values, -0 among the zeros
    few[::3] *= -1.0
    x = torch.from_numpy(few).to(_dtype(dtype)).cuda()
    _check(handles(E), x, 8, bias=b, scoring=scoring)
    _check(handles(E), x, 8, bias=b, scoring=scoring, groups=8, top_groups=3, group_top=2)
    _check(handles(E), torch.zeros_like(x), 8, bias=b, scoring=scoring, groups=8, top_groups=3, group_top=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_keys_that_32_bits_do_not_tell_apart(handles, scoring):
    """Logits one step apart, whose scores plus bias round to the same fp32 or in the wrong order."""
    torch = _t()
    rng = np.random.default_rng(5)
    E, T = 128, 60
    x = np.full((T, E), 1.0, np.float32)
    steps = rng.integers(-40, 41, (T, E))
    x = (x.view(np.int32) + steps.astype(np.int32)).view(np.float32)
    x = torch.from_numpy(x).cuda()
    _check(handles(E), x, 8, bias=np.full(E, 3.0), scoring=scoring)
    _check(handles(E), x, 8, bias=0.5 + rng.integers(0, 2, E) * 2.0 ** -24, scoring=scoring)
    _check(handles(E), x, 8, bias=None, scoring=scoring, groups=16, top_groups=4, group_top=2)
    _check(handles(E), x, 8, bias=np.full(E, 3.0), scoring=scoring, groups=16, top_groups=4, group_top=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top_k", [6, 12])
def test_more_near_keys_than_lanes(handles, scoring, top_k):
    """Every expert's key within the fp32 error of every other's, and all of them equal."""
    torch = _t()
    rng = np.random.default_rng(15)
    E, T = 200, 12
    x = (np.full((T, E), -1.5, np.float32).view(np.int32) + rng.integers(-3, 4, (T, E)).astype(np.int32)).view(np.float32)
    x = torch.from_numpy(x).cuda()
    bias = np.full(E, 1.0) + rng.integers(0, 2, E) * 2.0 ** -23
    for b in (None, bias, np.zeros(E)):
        _check(handles(E), x, top_k, bias=b, scoring=scoring)
        _check(handles(E), x, top_k, bias=b, scoring=scoring, groups=10, top_groups=4, group_top=2)
        _check(handles(E), torch.zeros_like(x), top_k, bias=b, scoring=scoring, groups=10, top_groups=4, group_top=1)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_groups_whose_terms_cancel(handles, scoring):
    """Biases of opposite signs, far larger than the scores: a group's sum is small and its fp32 error is not."""
    rng = np.random.default_rng(18)
    E = 16
    bias = np.where(np.arange(E) % 2 == 0, 1000.0, -1000.0)
    _check(handles(E), _logits(rng, 1500, E, "fp32", spread=0.5), 4, bias=bias, scoring=scoring, groups=8, top_groups=3, group_top=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_groups_far_below(handles, scoring, dtype):
    """Groups of logits so low that their scores are tiny or underflow, some with one expert left."""
    torch = _t()
    rng = np.random.default_rng(16)
    E, T = 64, 30
    x = _logits(rng, T, E, "fp32")
    x[:10] -= 20.0
    x[10:20, ::2] -= 60.0
    x[20:] *= 20.0
    x[:, 8:15] = -float("inf")
    x = x.to(_dtype(dtype))
    bias = 0.01 * rng.standard_normal(E)
    bias[40:47] = -np.inf
    bias[50] = np.inf
    for b in (None, bias):
        for group_top in (1, 2):
            _check(handles(E), x, 8, bias=b, scoring=scoring, groups=8, top_groups=3, group_top=group_top)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_experts(handles, scoring, dtype, with_bias):
    """Masked by -infinity (nothing, some, nearly all and all of a token's), and by the type's lowest value,
    which is an ordinary logit; biases of -infinity and NaN mask an expert for every token."""
    torch = _t()
    rng = np.random.default_rng(6)
    E, T = 40, 24
    x = _logits(rng, T, E, dtype)
    x[2:8, ::2] = -float("inf")
    x[8:12, 3:] = -float("inf")
    x[12:14] = -float("inf")
    x[14:18, 5:] = torch.finfo(x.dtype).min
    x[18:20] = torch.finfo(x.dtype).min
    bias = None
    if with_bias:
        bias = 0.1 * rng.standard_normal(E)
        bias[7] = -np.inf
        bias[9] = np.nan
    for renormalise in (True, False):
        _check(handles(E), x, 6, bias=bias, scoring=scoring, renormalise=renormalise)
    ids, w = _check(handles(E), x, 6, bias=bias, scoring=scoring, groups=5, top_groups=2, group_top=2)
    assert (ids[12:14] == -1).all() and (w[12:14] == 0).all()


def test_equal_keys_between_near_ones(handles):
    """An expert whose exact key belongs among the chosen ones, behind equal keys that its fp32 key follows."""
    torch = _t()
    E = 40
    x = np.full((64, E), -3.0, np.float32)
    bias = np.zeros(E, np.float32)
    rng = np.random.default_rng(17)
    for t in range(64):
        at = rng.permutation(E)[:6]
        x[t, at[:4]] = 1.0                                  # equal
        x[t, at[4:]] = np.nextafter(np.float32(1.0), np.float32(2.0)) if t % 2 else np.nextafter(np.float32(1.0), np.float32(0.0))
    for top_k in (1, 2, 3, 4, 5):
        _check(handles(E), torch.from_numpy(x).cuda(), top_k, bias=bias, scoring="sigmoid")
        _check(handles(E), torch.from_numpy(x).cuda(), top_k, bias=bias + 1, scoring="softmax")


def test_every_key_infinite(handles):
    """Biases of +infinity force experts; among them the lowest come first."""
    rng = np.random.default_rng(8)
    E = 50
    bias = np.zeros(E)
    bias[[3, 17, 30, 41]] = np.inf
    _check(handles(E), _logits(rng, 7, E, "fp32"), 3, bias=bias, scoring="sigmoid")
    _check(handles(E), _logits(rng, 7, E, "bf16"), 6, bias=bias, scoring="softmax")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_far_logits(handles, scoring):
    """Scores that underflow, and all-equal tokens far from zero."""
    torch = _t()
    rng = np.random.default_rng(9)
    x = _logits(rng, 12, 64, "fp32")
    x[0:3] -= 200.0
    x[3:6] -= 95.0
    x[6:8] += 60.0
    x[8] *= 30.0
    for renormalise in (True, False):
        _check(handles(64), x, 8, scoring=scoring, renormalise=renormalise)
    if scoring == "sigmoid":
        x[9, 5] = float("inf")
        _check(handles(64), x, 8, scoring=scoring)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_nan_logits_give_no_expert_and_are_reported(handles, dtype, many):
    from ragged_matmul_gb300 import binding
    rng = np.random.default_rng(10)
    E, T = 48, 3001 if many else 10
    x = _logits(rng, T, E, dtype)
    x[3, 47] = float("nan")
    x[6, 0] = float("inf")
    h = handles(E)
    clean = [t for t in range(T) if t not in (3, 6)]
    xs = x.double().cpu().numpy()
    want_ids, want_w = cu.choose(xs[clean], 4, scoring="softmax")
    for bias in (None, np.zeros(E)):
        ids, w = _route(h, x, 4, bias=bias, scoring="softmax")
        assert binding.gmm_query_status(h) == binding.GMM_ERR_BAD_INPUT
        assert (ids[[3, 6]] == -1).all() and (w[[3, 6]] == 0).all()
        np.testing.assert_array_equal(ids.cpu().numpy()[clean], want_ids)
        np.testing.assert_allclose(w.cpu().numpy()[clean], want_w, rtol=_rtol(xs[clean], E), atol=1e-37)
    ids, _ = _route(h, x, 4, scoring="sigmoid")
    assert binding.gmm_query_status(h) == binding.GMM_ERR_BAD_INPUT
    assert (ids[3] == -1).all() and ids[6, 0] == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("top_k", [3, 12])
def test_the_smallest_logits_keep_their_order(handles, dtype, top_k):
    """Subnormal values of both signs, zeros of both signs and the smallest normal ones."""
    torch = _t()
    rng = np.random.default_rng(13)
    E, T = 32, 12
    if dtype == "fp32":
        bits = rng.integers(0, 20, (T, E)).astype(np.int32)
        x = torch.from_numpy((bits | (rng.integers(0, 2, (T, E)) << 31).astype(np.int64)).astype(np.int64).astype(np.uint32).view(np.float32)).cuda()
    else:
        bits = rng.integers(0, 20, (T, E)) | (rng.integers(0, 2, (T, E)) << 15)
        x = torch.from_numpy(bits.astype(np.uint16).view(np.int16)).cuda().view(_dtype(dtype))
    _check(handles(E), x, top_k, scoring="sigmoid")
    _check(handles(E), x, top_k, scoring="softmax", groups=4, top_groups=2)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("top_k", [4, 12])
def test_nan_of_either_sign(handles, dtype, top_k):
    torch = _t()
    from ragged_matmul_gb300 import binding
    rng = np.random.default_rng(14)
    x = _logits(rng, 6, 64, dtype)
    nan = torch.tensor([float("nan")], device="cuda").to(x.dtype)
    x[1, 60], x[4, 0] = nan[0], -nan[0].abs()
    view = x.view(torch.int32 if dtype == "fp32" else torch.int16)
    view[4, 0] = -1                        # a NaN with every bit set
    for groups, kept in ((1, 1), (8, 6)):
        ids, w = _route(handles(64), x, top_k, scoring="sigmoid", expert_groups=groups, top_groups=kept)
        assert binding.gmm_query_status(handles(64)) == binding.GMM_ERR_BAD_INPUT
        assert (ids[[1, 4]] == -1).all() and (w[[1, 4]] == 0).all() and (ids[[0, 2, 3, 5]] >= 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E", [64, 100, 128, 200, 256])
def test_many_tokens_with_ties_and_masks(handles, E, dtype):
    """Tokens of few different logits, next to masked ones, where several share a warp."""
    torch = _t()
    rng = np.random.default_rng([E, 5])
    x = torch.from_numpy(rng.integers(-3, 4, (2600, E)).astype(np.float32)).to(_dtype(dtype)).cuda()
    x[::7, 5:] = -float("inf")
    x[3::11] = -float("inf")
    _check(handles(E), x, 8, scoring="softmax")
    _check(handles(E), x, 3, scoring="sigmoid", renormalise=False)


def test_strides_and_one_row_for_all(handles):
    torch = _t()
    rng = np.random.default_rng(11)
    wide = _logits(rng, 33, 131, "bf16")
    _check(handles(64), wide[:, 1:65], 8)
    _check(handles(64), wide[::2, 64:128], 8, scoring="sigmoid", bias=0.1 * rng.standard_normal(64))
    one = _logits(rng, 1, 64, "fp32").expand(7, 64)
    _check(handles(64), one, 4)
    _check(handles(64), one.half(), 4)


def test_no_tokens(handles):
    torch = _t()
    ids, w = _route(handles(64), torch.zeros((0, 64), device="cuda"), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)


def test_graph_replay_and_streams(handles):
    """A captured call follows its inputs; two streams with a handle each; the same bits every time."""
    torch = _t()
    from ragged_matmul_gb300 import binding
    rng = np.random.default_rng(12)
    E, T, k = 256, 300, 8
    h = handles(E)
    x = _logits(rng, T, E, "bf16")
    b = torch.zeros(E, device="cuda")
    ids, w = torch.zeros((T, k), dtype=torch.int32, device="cuda"), torch.zeros((T, k), device="cuda")
    d = torch.zeros_like(x)
    g = torch.ones((T, k), device="cuda").cumsum(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        binding.gmm_route(h, ids, w, x, bias=b, scoring="sigmoid", expert_groups=8, top_groups=4, group_top=2)
        binding.gmm_route_grad(h, d, g, ids, x, scoring="sigmoid")
    for seed in (1, 2):
        x.copy_(_logits(np.random.default_rng(seed), T, E, "bf16"))
        b.normal_(0, 0.05)
        graph.replay()
        torch.cuda.synchronize()
        xs = x.double().cpu().numpy()
        want_ids, want_w = cu.choose(xs, k, scoring="sigmoid", bias=b.cpu().numpy(), groups=8, top_groups=4, group_top=2)
        np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
        np.testing.assert_allclose(w.cpu().numpy(), want_w, rtol=_rtol(xs, E))
        again = [t.clone() for t in (ids, w, d)]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(again, (ids, w, d)))
    h2 = binding.gmm_create(E, 0)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        ids2, w2 = torch.empty_like(ids), torch.empty_like(w)
        binding.gmm_route(h2, ids2, w2, x, bias=b, scoring="sigmoid", expert_groups=8, top_groups=4, group_top=2)
    binding.gmm_route(h, ids, w, x, bias=b, scoring="sigmoid", expert_groups=8, top_groups=4, group_top=2)
    torch.cuda.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    binding.gmm_destroy(h2)


# ---------------------------------------------------------------- the gradient

def _check_grad(h, x, ids, dw, x_out=None, **kw):
    torch = _t()
    from ragged_matmul_gb300 import binding
    d = torch.full_like(x, float("nan")) if x_out is None else x_out
    binding.gmm_route_grad(h, d, dw, ids, x, **kw)
    assert binding.gmm_query_status(h) == binding.GMM_OK
    xs = x.double().cpu().numpy()
    want, mag = cu.grad(xs, ids.cpu().numpy(), dw.cpu().numpy(), **kw)
    err = np.abs(d.double().cpu().numpy() - want)
    half = torch.finfo(x.dtype).eps / 2
    tiny = torch.finfo(x.dtype).tiny * torch.finfo(x.dtype).eps + 1e-37      # below the smallest step of the type
    bound = mag * 3 * (_rtol(xs, xs.shape[1]) + 2.0 ** -24 * 40)
    assert np.all(err <= bound + (np.abs(want) + bound) * half + tiny), float((err - bound).max())
    return d


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("E,top_k,T", [(1, 1, 3), (8, 3, 5), (64, 8, 2503), (63, 6, 9), (128, 12, 2501), (161, 8, 7), (1000, 32, 4),
                                       (4096, 8, 3)])
def test_gradient(handles, E, top_k, T, scoring, renormalise, dtype):
    torch = _t()
    rng = np.random.default_rng([E, top_k, T])
    x = _logits(rng, T, E, dtype)
    ids, _ = _route(handles(E), x, top_k, scoring=scoring)
    dw = torch.from_numpy(rng.standard_normal((T, top_k)).astype(np.float32)).cuda()
    _check_grad(handles(E), x, ids, dw, scoring=scoring, renormalise=renormalise, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_gradient_of_dropped_masked_and_repeated_slots(handles, scoring, renormalise):
    torch = _t()
    from ragged_matmul_gb300 import binding
    rng = np.random.default_rng(20)
    E, T, k = 24, 12, 5
    x = _logits(rng, T, E, "fp32")
    x[1:4, 6:] = -float("inf")
    x[4] = -float("inf")
    x[5] -= 150.0
    ids = torch.from_numpy(rng.integers(0, E, (T, k)).astype(np.int32)).cuda()
    ids[0] = -1                       # a token without experts
    ids[6, 1:3] = -1
    ids[7] = 11                       # the same expert in every slot
    ids[8, 3] = ids[8, 0]
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    dw[0, 0] = float("nan")           # a dropped slot's gradient is not read into anything
    h = handles(E)
    d = _check_grad(h, x, ids, dw, scoring=scoring, renormalise=renormalise)
    assert (d[0] == 0).all() and (d[4] == 0).all()
    ids[9, 2] = E                     # out of range: left out and reported
    d2 = torch.empty_like(x)
    binding.gmm_route_grad(h, d2, dw, ids, x, scoring=scoring, renormalise=renormalise)
    assert binding.gmm_query_status(h) == binding.GMM_ERR_BAD_INPUT
    want, _ = cu.grad(x.double().cpu().numpy(), ids.cpu().numpy(), dw.cpu().numpy(), scoring=scoring, renormalise=renormalise)
    np.testing.assert_allclose(d2.double().cpu().numpy(), want, atol=1e-4)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_gradient_by_differences(handles, scoring, renormalise):
    """The 64-bit reference's own weights, two sides of each logit: the gradient's formula, not its rounding."""
    torch = _t()
    rng = np.random.default_rng(21)
    E, T, k = 12, 6, 4
    x = _logits(rng, T, E, "fp32")
    ids, _ = _route(handles(E), x, k, scoring=scoring)
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    d = _check_grad(handles(E), x, ids, dw, scoring=scoring, renormalise=renormalise, scale=1.5)
    xs, chosen, g = x.double().cpu().numpy(), ids.cpu().numpy(), dw.double().cpu().numpy()

    def loss(v):
        w = np.take_along_axis(cu.scores(v, scoring), chosen, 1)
        if renormalise:
            w = w / w.sum(1, keepdims=True)
        return (1.5 * w * g).sum(1)

    step = 1e-5
    for e in range(E):
        hi, lo = xs.copy(), xs.copy()
        hi[:, e] += step
        lo[:, e] -= step
        np.testing.assert_allclose(d[:, e].double().cpu().numpy(), (loss(hi) - loss(lo)) / (2 * step), atol=2e-5)


def test_gradient_strides_and_reported_tokens(handles):
    torch = _t()
    from ragged_matmul_gb300 import binding
    rng = np.random.default_rng(22)
    E, T, k = 64, 19, 6
    h = handles(E)
    wide, out = _logits(rng, T, 131, "bf16"), torch.zeros((T, 200), dtype=torch.bfloat16, device="cuda")
    x = wide[:, 3:67]
    ids, _ = _route(h, x, k)
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    for renormalise in (True, False):
        _check_grad(h, x, ids, dw, x_out=out[:, 100:164], renormalise=renormalise)
    assert (out[:, :100] == 0).all() and (out[:, 164:] == 0).all()       # nothing beside the view is written
    x = _logits(rng, T, E, "fp32")
    x[2, 9] = float("nan")
    d = torch.full_like(x, 5.0)
    ids, _ = _route(h, x, k, renormalise=False)
    assert binding.gmm_query_status(h) == binding.GMM_ERR_BAD_INPUT
    binding.gmm_route_grad(h, d, dw, ids, x, renormalise=False)
    assert (d[2] == 0).all() and torch.isfinite(d).all()
    binding.gmm_query_status(h)


# ---------------------------------------------------------------- refusals

def test_refusals(handles):
    torch = _t()
    from ragged_matmul_gb300 import binding
    h = handles(64)
    x = torch.zeros((5, 64), device="cuda")
    ids, w = torch.zeros((5, 4), dtype=torch.int32, device="cuda"), torch.zeros((5, 4), device="cuda")
    ok = dict(scoring="softmax")
    binding.gmm_route(h, ids, w, x, **ok)
    for kw in (dict(expert_groups=3), dict(expert_groups=0), dict(expert_groups=8, top_groups=9), dict(expert_groups=8, top_groups=0),
               dict(expert_groups=64, top_groups=2), dict(group_top=3), dict(group_top=0), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(expert_groups=64, top_groups=8, group_top=2)):
        with pytest.raises(binding.GmmError) as e:
            binding.gmm_route(h, ids, w, x, **kw)
        assert e.value.code == binding.GMM_ERR_INVALID_ARG, kw
    with pytest.raises(binding.GmmError) as e:      # more than 32 groups
        binding.gmm_route(h, ids, w, x, expert_groups=64, top_groups=8)
    assert e.value.code == binding.GMM_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        binding.gmm_route(h, ids, w, x, scoring="relu")
    with pytest.raises(ValueError):
        binding.gmm_route(h, ids, w, x[:, :63])
    with pytest.raises(ValueError):
        binding.gmm_route(h, ids[:4], w, x)
    with pytest.raises(ValueError):
        binding.gmm_route(h, ids, w[:, :3], x)
    with pytest.raises(ValueError):
        binding.gmm_route(h, ids, w, x, bias=torch.zeros(63, device="cuda"))
    with pytest.raises(TypeError):
        binding.gmm_route(h, ids, w, x.double())
    with pytest.raises(TypeError):
        binding.gmm_route(h, ids.long(), w, x)
    with pytest.raises(ValueError):
        binding.gmm_route(h, ids, w, x.t().contiguous().t())
    with pytest.raises(binding.GmmError) as e:
        binding.gmm_route(handles(3), torch.zeros((5, 4), dtype=torch.int32, device="cuda"), w, x[:, :3].contiguous())
    assert e.value.code == binding.GMM_ERR_INVALID_ARG
    with pytest.raises(binding.GmmError) as e:
        binding.gmm_route(h, torch.zeros((5, 33), dtype=torch.int32, device="cuda"), torch.zeros((5, 33), device="cuda"), x)
    assert e.value.code == binding.GMM_ERR_UNSUPPORTED
    d = torch.zeros_like(x)
    binding.gmm_route_grad(h, d, w, ids, x)
    with pytest.raises(TypeError):
        binding.gmm_route_grad(h, d.half(), w, ids, x)
    with pytest.raises(ValueError):
        binding.gmm_route_grad(h, d[:4], w, ids, x)
    with pytest.raises(ValueError):
        binding.gmm_route_grad(h, torch.zeros((1, 64), device="cuda").expand(5, 64), w, ids, x)
    with pytest.raises(ValueError):
        binding.gmm_route_grad(h, d, w[:, :3], ids, x)
    assert binding.gmm_query_status(h) == binding.GMM_OK
