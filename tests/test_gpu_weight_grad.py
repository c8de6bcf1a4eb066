"""The weight gradient on 8-bit operands against 64 bits: tile edges in n and k, groups without rows, of one
row and of many blocks, scales of every row and column, both result types, accumulation, special values,
graphs, streams, refusals.

Tolerance.  The operands are exact in the tensor core (products of two e4m3 values have 8 bits, powers of two
scale them), sums are fp32: with n products of a result and the tensor core adding 32 of them at a time onto
its accumulator, each addition is off by one step at most (2^-23, aligned sums are cut off) of what is summed,
so an error of up to (n / 32 + 33) 2^-23 times the sum of the products' magnitudes; then one rounding."""
import numpy as np
import pytest

from tests import fp8_util as fu

pytestmark = pytest.mark.gpu


def _t():
    import torch
    return torch


@pytest.fixture(scope="module")
def h():
    from ragged_matmul_gb300 import binding
    handle = binding.gmm_create(4, 0)
    yield handle
    binding.gmm_destroy(handle)


def _offsets(loads, first=0):
    return np.concatenate([[first], first + np.cumsum(loads)]).astype(np.int64)


def _operand(rng, width, offsets, rows, exponents=(90, 160)):
    """Random codes and scales (numpy): zeros behind a group's last row; blocks that no group uses hold NaN codes."""
    G = len(offsets) - 1
    P = fu.pitch(rows, G)
    q = np.full((width, P), 0x7F, np.uint8)
    s = np.full((P // 128, width), 0xFF, np.uint8)
    for g in range(G):
        n = int(offsets[g + 1] - offsets[g])
        nb = -(-n // 128)
        at = int(offsets[g]) // 128 + g
        c = rng.integers(0, 256, (width, nb * 128)).astype(np.uint8)
        c[(c & 0x7F) == 0x7F] = 0x7E
        c[:, n:] = 0
        q[:, at * 128:(at + nb) * 128] = c
        s[at:at + nb] = rng.integers(*exponents, (nb, width))
    return q, s


def _dev(x):
    torch = _t()
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _run(h, d, ds, a, as_, offsets, dtype="fp32", out=None, accumulate=False, stream=None):
    torch = _t()
    from ragged_matmul_gb300 import binding
    G = len(offsets) - 1
    if out is None:
        out = torch.full((G, d.shape[0], a.shape[0]), float("nan"), dtype=torch.float32 if dtype == "fp32" else torch.bfloat16,
                         device="cuda")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    binding.gmm_weight_grad_fp8(h, out, _dev(d), _dev(ds), _dev(a), _dev(as_), off, accumulate=accumulate, stream=stream)
    return out


def _check(out, d, ds, a, as_, offsets, base=0.0):
    torch = _t()
    want, mag = fu.weight_grad(d, ds, a, as_, offsets)
    n = np.diff(offsets).reshape(-1, 1, 1)
    bound = (n / 32 + 33) * 2.0 ** -23 * (mag + np.abs(base)) + 1e-37
    want = want + base
    got = out.double().cpu().numpy()
    err = np.abs(got - want)
    half = torch.finfo(out.dtype).eps / 2
    assert np.all(err <= bound + half * (np.abs(want) + bound)), (float(np.nanmax(err / (mag + 1e-300))), int(np.isnan(got).sum()))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N,K", [(16, 16), (128, 240), (256, 256), (272, 48), (144, 496), (512, 720), (48, 1008)])
@pytest.mark.parametrize("loads", [(128,), (1, 0, 300, 127)])
def test_shapes(h, N, K, loads, dtype):
    from ragged_matmul_gb300 import binding
    rng = np.random.default_rng([N, K, len(loads)])
    off = _offsets(loads)
    rows = int(off[-1])
    d, ds = _operand(rng, N, off, rows)
    a, as_ = _operand(rng, K, off, rows)
    out = _run(h, d, ds, a, as_, off, dtype)
    assert binding.gmm_query_status(h) == binding.GMM_OK
    _check(out, d, ds, a, as_, off)


@pytest.mark.parametrize("loads,first,behind", [((0, 0), 0, 0), ((1,), 0, 0), ((129, 255, 256), 3, 70), (tuple([2] * 130), 0, 1),
                                                ((2000, 0, 5, 700), 0, 0), (tuple([0] * 50 + [64]), 127, 0)])
def test_groups(h, loads, first, behind):
    """Groups of every length, rows before the first and behind the last."""
    from ragged_matmul_gb300 import binding
    rng = np.random.default_rng(len(loads))
    off = _offsets(loads, first)
    rows = int(off[-1]) + behind
    d, ds = _operand(rng, 64, off, rows)
    a, as_ = _operand(rng, 96, off, rows)
    out = _run(h, d, ds, a, as_, off)
    assert binding.gmm_query_status(h) == binding.GMM_OK
    _check(out, d, ds, a, as_, off)


def test_many_groups(h):
    """As many groups as the library takes; most of them empty."""
    from ragged_matmul_gb300 import binding
    rng = np.random.default_rng(2)
    loads = np.zeros(4096, int)
    loads[[0, 17, 2000, 4095]] = (3, 140, 1, 9)
    off = _offsets(loads)
    rows = int(off[-1])
    d, ds = _operand(rng, 32, off, rows)
    a, as_ = _operand(rng, 16, off, rows)
    out = _run(h, d, ds, a, as_, off)
    assert binding.gmm_query_status(h) == binding.GMM_OK
    _check(out, d, ds, a, as_, off)


def test_every_scale_reaches_its_row_and_block(h):
    """One-hot codes: each result is one product of two scales, exactly."""
    N, K, rows = 400, 272, 700
    off = np.array([0, 300, 700])
    rng = np.random.default_rng(3)
    d, ds = _operand(rng, N, off, rows, (100, 150))
    a, as_ = _operand(rng, K, off, rows, (100, 150))
    for r in (0, 127, 128, 299, 300, 427, 428, 699):
        g = int(r >= 300)
        col = (off[g] // 128 + g) * 128 + r - off[g]
        one_d, one_a = np.zeros_like(d), np.zeros_like(a)
        one_d[:, col] = 0x38              # 1.0
        one_a[:, col] = 0x40              # 2.0
        out = _run(h, one_d, ds, one_a, as_, off).double().cpu().numpy()
        want = np.zeros((2, N, K))
        want[g] = 2.0 * np.outer(fu.E8M0[ds[col // 128]], fu.E8M0[as_[col // 128]])
        np.testing.assert_array_equal(out, want)


@pytest.mark.parametrize("loads", [(200, 0, 1), (0, 0, 0)])
def test_accumulate(h, loads):
    """Adds to d_b; groups without rows stay as they are."""
    torch = _t()
    rng = np.random.default_rng(4)
    off = _offsets(loads)
    rows = int(off[-1])
    d, ds = _operand(rng, 272, off, rows, (120, 130))
    a, as_ = _operand(rng, 144, off, rows, (120, 130))
    base = 100.0 * rng.standard_normal((3, 272, 144)).astype(np.float32)
    out = _run(h, d, ds, a, as_, off, out=torch.from_numpy(base).cuda(), accumulate=True)
    _check(out, d, ds, a, as_, off, base=base.astype(np.float64))
    assert np.array_equal(out[1].cpu().numpy(), base[1])


def test_a_block_that_is_not_finite_spoils_its_row_of_the_gradient(h):
    rng = np.random.default_rng(5)
    off = _offsets((140, 20))
    d, ds = _operand(rng, 80, off, 160)
    a, as_ = _operand(rng, 64, off, 160)
    ds[1, 33] = 255                       # group 0's second block
    as_[off[1] // 128 + 1, 7] = 255       # group 1's
    out = _run(h, d, ds, a, as_, off).cpu().numpy()
    nan = np.isnan(out)
    want = np.zeros_like(nan)
    want[0, 33, :] = True
    want[1, :, 7] = True
    np.testing.assert_array_equal(nan, want)


def test_from_the_quantiser(h):
    """Rows of a batch sorted by expert, quantised along the rows, to the gradient of the weights."""
    torch = _t()
    from ragged_matmul_gb300 import binding
    rng = np.random.default_rng(6)
    T, k, E, N, K = 333, 2, 4, 272, 400
    ids = torch.from_numpy(rng.integers(-1, E, (T, k)).astype(np.int32)).cuda()
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).cuda().bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    off, sr, rs = torch.zeros(E + 1, **i32), torch.zeros((T, k), **i32), torch.zeros(T * k, **i32)
    binding.gmm_dispatch(h, off, sr, rs, ids)
    dc = torch.from_numpy(rng.standard_normal((T * k, N)).astype(np.float32)).cuda().bfloat16()
    P = binding.fp8_cols_pitch(T * k, E)
    u8 = lambda *s: torch.full(s, 0x7F, dtype=torch.uint8, device="cuda")  # noqa: E731
    a, as_, d, ds = u8(K, P), u8(P // 128, K), u8(N, P), u8(P // 128, N)
    binding.gmm_quantize_fp8_cols(h, a, as_, x, off, row_slots=rs, top_k=k)
    binding.gmm_quantize_fp8_cols(h, d, ds, dc, off)
    out = torch.full((E, N, K), float("nan"), device="cuda")
    binding.gmm_weight_grad_fp8(h, out, d, ds, a, as_, off)
    assert binding.gmm_query_status(h) == binding.GMM_OK
    offs = off.cpu().numpy().astype(np.int64)
    _check(out, d.cpu().numpy(), ds.cpu().numpy(), a.cpu().numpy(), as_.cpu().numpy(), offs)
    # Against the unquantised product: each operand is off by half a step of e4m3, 2^-4 of the value or
    # 2^-10 times its block's scale, which is at most amax / 224.
    rows = x.double().cpu().numpy()[np.maximum(rs.cpu().numpy(), 0) // k]
    dcs = dc.double().cpu().numpy()
    for g in range(E):
        r = slice(offs[g], offs[g + 1])
        exact = dcs[r].T @ rows[r]
        da, dd = np.abs(rows[r]) * 2.0 ** -4 + np.abs(rows[r]).max() / 224 * 2.0 ** -10, np.abs(dcs[r]) * 2.0 ** -4 + np.abs(dcs[r]).max() / 224 * 2.0 ** -10
        bound = dd.T @ np.abs(rows[r]) + np.abs(dcs[r]).T @ da + dd.T @ da
        assert np.all(np.abs(out[g].double().cpu().numpy() - exact) <= bound * 1.01)


def test_bad_offsets_write_nothing(h):
    torch = _t()
    from ragged_matmul_gb300 import binding
    rng = np.random.default_rng(7)
    good = _offsets((30, 20, 14))
    d, ds = _operand(rng, 32, good, 64)
    a, as_ = _operand(rng, 32, good, 64)
    for off in ([0, 30, 20, 64], [0, 10, 20, 900], [0, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], [0, -1, 5, 6]):
        out = torch.full((3, 32, 32), 7.0, device="cuda")
        _run(h, d, ds, a, as_, off, out=out)
        assert binding.gmm_query_status(h) == binding.GMM_ERR_BAD_INPUT
        assert (out == 7.0).all()


def test_without_rows(h):
    """No rows at all: zeros, or nothing when the call accumulates."""
    torch = _t()
    from ragged_matmul_gb300 import binding
    P = binding.fp8_cols_pitch(0, 2)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((2, 48, 80), 3.0, dtype=dtype, device="cuda")
        binding.gmm_weight_grad_fp8(h, out, u8(48, P), u8(2, 48), u8(80, P), u8(2, 80), off)
        assert (out == 0).all()
    out = torch.full((2, 48, 80), 3.0, device="cuda")
    binding.gmm_weight_grad_fp8(h, out, u8(48, P), u8(2, 48), u8(80, P), u8(2, 80), off, accumulate=True)
    assert (out == 3.0).all()
    lib = binding.load_library()          # the C call without operands
    rc = lib.gmm_weight_grad_fp8(h.ptr, out.data_ptr(), None, None, None, None, None, 2, 0, 48, 80, binding.GMM_DTYPE_FP32, 0,
                                 binding.stream_handle(0))
    assert rc == binding.GMM_OK and binding.gmm_query_status(h) == binding.GMM_OK
    assert (out == 0).all()


def test_graph_replay_and_streams(h):
    torch = _t()
    from ragged_matmul_gb300 import binding
    rng = np.random.default_rng(8)
    off = _offsets((300, 40, 0, 260))
    d, ds = _operand(rng, 528, off, 600)
    a, as_ = _operand(rng, 496, off, 600)
    t = [_dev(x) for x in (d, ds, a, as_)]
    offt = torch.tensor(off, dtype=torch.int32, device="cuda")
    out = torch.zeros((4, 528, 496), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        binding.gmm_weight_grad_fp8(h, out, *t, offt)
    graph.replay()
    torch.cuda.synchronize()
    _check(out, d, ds, a, as_, off)
    first = out.clone()
    d2, ds2 = _operand(rng, 528, off, 600)
    t[0].copy_(_dev(d2))
    t[1].copy_(_dev(ds2))
    graph.replay()
    torch.cuda.synchronize()
    _check(out, d2, ds2, a, as_, off)
    t[0].copy_(_dev(d))
    t[1].copy_(_dev(ds))
    h2 = binding.gmm_create(4, 0)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    out2 = torch.zeros_like(out)
    torch.cuda.synchronize()
    for _ in range(3):                    # two handles, two streams, the same bits
        binding.gmm_weight_grad_fp8(h, out, *t, offt)
        binding.gmm_weight_grad_fp8(h2, out2, *t, offt, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(out2, first)
    binding.gmm_destroy(h2)


def test_refusals(h):
    torch = _t()
    from ragged_matmul_gb300 import binding
    P = binding.fp8_cols_pitch(100, 2)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.zeros((2, 48, 80), device="cuda")
    ok = (u8(48, P), u8(P // 128, 48), u8(80, P), u8(P // 128, 80), off)
    binding.gmm_weight_grad_fp8(h, out, *ok)
    with pytest.raises(binding.GmmError) as e:      # accumulation in fewer bits
        binding.gmm_weight_grad_fp8(h, out.bfloat16(), *ok, accumulate=True)
    assert e.value.code == binding.GMM_ERR_INVALID_ARG
    with pytest.raises(TypeError):
        binding.gmm_weight_grad_fp8(h, out.half(), *ok)
    with pytest.raises(binding.GmmError) as e:      # 40 is not a multiple of 16
        binding.gmm_weight_grad_fp8(h, torch.zeros((2, 40, 80), device="cuda"), u8(40, P), u8(P // 128, 40), *ok[2:])
    assert e.value.code == binding.GMM_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        binding.gmm_weight_grad_fp8(h, out[0], *ok)
    with pytest.raises(ValueError):
        binding.gmm_weight_grad_fp8(h, out, u8(48, P + 16), *ok[1:])
    with pytest.raises(ValueError):
        binding.gmm_weight_grad_fp8(h, out, ok[0], u8(P // 128 + 1, 48), *ok[2:])
    with pytest.raises(ValueError):
        binding.gmm_weight_grad_fp8(h, out, ok[0], ok[1], u8(80, P + 128), *ok[3:])
    with pytest.raises(ValueError):
        binding.gmm_weight_grad_fp8(h, out, *ok[:4], off[:2])
    with pytest.raises(ValueError):
        binding.gmm_weight_grad_fp8(h, out.transpose(1, 2), *ok)
    with pytest.raises(binding.GmmError) as e:      # d_b not on 16 bytes
        binding.gmm_weight_grad_fp8(h, torch.zeros(2 * 48 * 80 + 1, device="cuda")[1:].view(2, 48, 80), *ok)
    assert e.value.code == binding.GMM_ERR_INVALID_ARG
    assert binding.gmm_query_status(h) == binding.GMM_OK
