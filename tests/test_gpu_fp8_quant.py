"""The 8-bit quantisers on the GPU against their definitions, codes and scales bit for bit: every type, short
and odd sizes, last blocks that are not whole, gathers, groups of every length, values at the border between
two codes and two powers of two, special values, strides, graphs, refusals."""
import numpy as np
import pytest

from tests import fp8_util as fu

pytestmark = pytest.mark.gpu
TYPES = ["bf16", "fp16", "fp32"]


def _t():
    import torch
    return torch


@pytest.fixture(scope="module")
def h():
    from ragged_matmul_gb300 import binding
    handle = binding.gmm_create(8, 0)
    yield handle
    binding.gmm_destroy(handle)


def _dtype(name):
    torch = _t()
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _values(rng, shape, dtype):
    """Normal values of very different sizes from channel to channel and row to row, some zero."""
    torch = _t()
    x = rng.standard_normal(shape) * 2.0 ** rng.integers(-6, 7, shape[-1:])
    x *= 2.0 ** rng.integers(-3, 4, shape[:-1] + (1,))
    x[rng.random(shape) < 0.05] = 0.0
    return torch.from_numpy(x.astype(np.float32)).to(_dtype(dtype)).cuda()


def _f32(x):
    return x.float().cpu().numpy()


def _u8(*shape, fill=0x5A):
    torch = _t()
    return torch.full(shape, fill, dtype=torch.uint8, device="cuda")


def _same_scales(got, want):
    np.testing.assert_array_equal(got.double().cpu().numpy(), want)      # NaN where NaN


def _rows(h, x, pow2=False, **kw):
    torch = _t()
    from ragged_matmul_gb300 import binding
    n = kw["row_slots"].numel() if kw.get("row_slots") is not None else x.shape[0]
    q, s = _u8(n, x.shape[1]), torch.full((n, -(-x.shape[1] // 128)), -5.0, device="cuda")
    binding.gmm_quantize_fp8(h, q, s, x, pow2=pow2, **kw)
    return q, s


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("R,K", [(1, 16), (3, 128), (5, 144), (1, 2048), (70, 256), (129, 1424), (33, 4096), (1000, 112)])
def test_rows(h, R, K, pow2, dtype):
    from ragged_matmul_gb300 import binding
    x = _values(np.random.default_rng([R, K]), (R, K), dtype)
    q, s = _rows(h, x, pow2)
    want_q, want_s = fu.rows(_f32(x), pow2)
    _same_scales(s, want_s)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)
    q8 = _t().empty((R, K), dtype=_t().float8_e4m3fn, device="cuda")     # the other type of buffer
    binding.gmm_quantize_fp8(h, q8, s, x, pow2=pow2)
    assert _t().equal(q8.view(_t().uint8), q)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (2, 128, 128), (3, 200, 144), (1, 257, 1424), (5, 16, 272), (2, 384, 512)])
def test_tiles(h, E, N, K, pow2, dtype):
    torch = _t()
    from ragged_matmul_gb300 import binding
    w = _values(np.random.default_rng([E, N, K]), (E, N, K), dtype)
    q, s = _u8(E, N, K), torch.full((E, -(-N // 128), -(-K // 128)), -5.0, device="cuda")
    binding.gmm_quantize_fp8_tiles(h, q, s, w, pow2=pow2)
    want_q, want_s = fu.tiles(_f32(w), pow2)
    _same_scales(s, want_s)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)


def _offsets(loads, first=0):
    return np.concatenate([[first], first + np.cumsum(loads)]).astype(np.int64)


def _dev(offsets):
    return _t().tensor(offsets, dtype=_t().int32, device="cuda")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("loads,width", [((1,), 16), ((128,), 128), ((127, 1, 129), 144), ((0, 0, 300, 0), 272), ((5, 0, 0, 2), 1424),
                                         ((256, 255, 1, 513), 400), ((0,), 32), (tuple([3] * 300), 48)])
def test_cols(h, loads, width, both, dtype):
    torch = _t()
    from ragged_matmul_gb300 import binding
    rng = np.random.default_rng([len(loads), width])
    G, R = len(loads), sum(loads) + 5          # rows behind the last group
    for first in (0, 3):
        off = _offsets(loads, first)
        rows = max(R, int(off[-1]))
        x = _values(rng, (rows, width), dtype)
        P = fu.pitch(rows, G)
        q_t, ts = _u8(width, P), _u8(P // 128, width, fill=0x33)
        q, s = (_u8(rows, width), torch.full((rows, -(-width // 128)), -5.0, device="cuda")) if both else (None, None)
        binding.gmm_quantize_fp8_cols(h, q_t, ts, x, _dev(off), q=q, scales=s)
        assert binding.gmm_query_status(h) == binding.GMM_OK
        want, want_s = fu.cols(_f32(x), off, rows, np.full((width, P), 0x5A, np.uint8), np.full((P // 128, width), 0x33, np.uint8))
        np.testing.assert_array_equal(ts.cpu().numpy(), want_s)
        np.testing.assert_array_equal(q_t.cpu().numpy(), want)
        if both:
            want_q, want_rs = fu.rows(_f32(x), False)
            live = (np.arange(rows) >= off[0]) & (np.arange(rows) < off[-1])
            want_q[~live], want_rs[~live] = 0x5A, -5.0
            _same_scales(s, want_rs)
            np.testing.assert_array_equal(q.cpu().numpy(), want_q)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gathered(h, dtype):
    """Rows picked by slots, some without a source, and one past the tokens."""
    torch = _t()
    from ragged_matmul_gb300 import binding
    rng = np.random.default_rng(7)
    T, k, K = 90, 3, 272
    x = _values(rng, (T, K), dtype)
    slots = rng.permutation(T * k).astype(np.int32)
    slots[[4, 100]] = -1
    rs = torch.from_numpy(slots).cuda()
    xs = _f32(x)[np.maximum(slots, 0) // k]
    xs[slots < 0] = 0.0
    want_q, want_s = fu.rows(xs, False)
    want_q[slots < 0], want_s[slots < 0] = 0x5A, -5.0
    q, s = _rows(h, x, row_slots=rs, top_k=k)
    _same_scales(s, want_s)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)
    loads = (100, 0, 1, 169)
    off, R = _offsets(loads), T * k
    P = fu.pitch(R, 4)
    q_t, ts = _u8(K, P), _u8(P // 128, K)
    q, s = _u8(R, K), torch.full((R, -(-K // 128)), -5.0, device="cuda")
    binding.gmm_quantize_fp8_cols(h, q_t, ts, x, _dev(off), row_slots=rs, top_k=k, q=q, scales=s)
    assert binding.gmm_query_status(h) == binding.GMM_OK
    want_t, want_ts = fu.cols(xs, off, R, np.full((K, P), 0x5A, np.uint8), np.full((P // 128, K), 0x5A, np.uint8))
    np.testing.assert_array_equal(ts.cpu().numpy(), want_ts)
    np.testing.assert_array_equal(q_t.cpu().numpy(), want_t)
    _same_scales(s, want_s)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)
    slots[7] = T * k                       # past the tokens: as without a source, and reported
    rs = torch.from_numpy(slots).cuda()
    q, s = _rows(h, x, row_slots=rs, top_k=k)
    assert binding.gmm_query_status(h) == binding.GMM_ERR_BAD_INPUT
    assert (q[7] == 0x5A).all() and (s[7] == -5.0).all()
    binding.gmm_quantize_fp8_cols(h, q_t, ts, x, _dev(off), row_slots=rs, top_k=k)
    assert binding.gmm_query_status(h) == binding.GMM_ERR_BAD_INPUT
    assert (q_t[:, 7] == 0).all()


@pytest.mark.parametrize("pow2", [False, True])
def test_borders(h, pow2):
    """Quotients at and next to the middle between two codes, and largest magnitudes at and next to 448 times
    a power of two, over the whole range of exponents."""
    torch = _t()
    from ragged_matmul_gb300 import binding
    mids = (fu.GRID[1:] + fu.GRID[:-1]) / 2
    at = np.concatenate([mids, np.nextafter(mids.astype(np.float32), np.float32(0)), np.nextafter(mids.astype(np.float32), np.float32(1e9))])
    x = []
    for ex in list(range(-149, -100)) + [-60, -1, 0, 3, 60] + list(range(100, 119)):
        for top in (448.0, np.nextafter(np.float32(448), np.float32(0)), np.nextafter(np.float32(448), np.float32(500)), 447.0, 300.0, 256.0):
            row = np.zeros(128 * 3)
            row[:at.size] = at[:384]
            row[::128] = top
            with np.errstate(under="ignore", over="ignore"):
                x.append(np.ldexp(row * np.where(np.arange(384) % 3 == 0, -1, 1), ex).astype(np.float32))
    x = np.array(x)
    x = x[:, :384]
    x[~np.isfinite(x)] = 0.0
    xt = torch.from_numpy(x).cuda()
    q, s = _rows(h, xt, pow2)
    want_q, want_s = fu.rows(x, pow2)
    _same_scales(s, want_s)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)
    if pow2:                               # the same values as columns
        rows = x.shape[0] - x.shape[0] % 128
        xc = np.ascontiguousarray(x[:rows].reshape(-1, 128).T[:, :1440])
        xt = torch.from_numpy(xc).cuda()
        P = fu.pitch(128, 1)
        q_t, ts = _u8(xc.shape[1], P), _u8(P // 128, xc.shape[1])
        binding.gmm_quantize_fp8_cols(h, q_t, ts, xt, _dev([0, 128]))
        want, want_ts = fu.cols(xc, [0, 128], 128, np.full((xc.shape[1], P), 0x5A, np.uint8), np.full((P // 128, xc.shape[1]), 0x5A, np.uint8))
        np.testing.assert_array_equal(ts.cpu().numpy(), want_ts)
        np.testing.assert_array_equal(q_t.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", TYPES)
def test_special_values(h, dtype):
    """Infinities and NaN spoil their own block only; blocks of zeros; the type's largest values."""
    torch = _t()
    from ragged_matmul_gb300 import binding
    rng = np.random.default_rng(9)
    x = _values(rng, (260, 400), dtype)
    x[0, 5] = float("inf")
    x[1, 130] = -float("inf")
    x[2, 399] = float("nan")
    x[3, :128] = 0.0
    x[4] = -0.0
    x[5, 0], x[5, 200] = torch.finfo(x.dtype).max, torch.finfo(x.dtype).min
    x[6, :16] = torch.finfo(x.dtype).tiny
    x[7] = 0.0
    x[7, 3] = torch.finfo(x.dtype).tiny * torch.finfo(x.dtype).eps
    x[10:200, 17] = 0.0
    xs = _f32(x)
    for pow2 in (False, True):
        q, s = _rows(h, x, pow2)
        want_q, want_s = fu.rows(xs, pow2)
        _same_scales(s, want_s)
        np.testing.assert_array_equal(q.cpu().numpy(), want_q)
        tq, tsc = _u8(1, 260, 400), torch.zeros((1, 3, 4), device="cuda")
        binding.gmm_quantize_fp8_tiles(h, tq, tsc, x[None].contiguous(), pow2=pow2)
        want_q, want_s = fu.tiles(xs[None], pow2)
        _same_scales(tsc, want_s)
        np.testing.assert_array_equal(tq.cpu().numpy(), want_q)
    off = _offsets((2, 130, 0, 128))
    P = fu.pitch(260, 4)
    q_t, ts = _u8(400, P), _u8(P // 128, 400)
    q, s = _u8(260, 400), torch.full((260, 4), -5.0, device="cuda")
    binding.gmm_quantize_fp8_cols(h, q_t, ts, x, _dev(off), q=q, scales=s)
    want, want_ts = fu.cols(xs, off, 260, np.full((400, P), 0x5A, np.uint8), np.full((P // 128, 400), 0x5A, np.uint8))
    np.testing.assert_array_equal(ts.cpu().numpy(), want_ts)
    np.testing.assert_array_equal(q_t.cpu().numpy(), want)
    want_q, want_s = fu.rows(xs, False)
    _same_scales(s, want_s)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_strides(h, dtype, shift):
    """Rows any distance apart and on any element, and one row for all."""
    torch = _t()
    from ragged_matmul_gb300 import binding
    rng = np.random.default_rng(11)
    wide = _values(rng, (150, 331), dtype)
    x = wide[::2, shift:shift + 272]
    for pow2 in (False, True):
        q, s = _rows(h, x, pow2)
        want_q, want_s = fu.rows(_f32(x), pow2)
        _same_scales(s, want_s)
        np.testing.assert_array_equal(q.cpu().numpy(), want_q)
    off = _offsets((30, 45))
    P = fu.pitch(75, 2)
    q_t, ts = _u8(272, P), _u8(P // 128, 272)
    binding.gmm_quantize_fp8_cols(h, q_t, ts, x, _dev(off))
    want, want_ts = fu.cols(_f32(x), off, 75, np.full((272, P), 0x5A, np.uint8), np.full((P // 128, 272), 0x5A, np.uint8))
    np.testing.assert_array_equal(ts.cpu().numpy(), want_ts)
    np.testing.assert_array_equal(q_t.cpu().numpy(), want)
    one = wide[:1, shift:shift + 48].expand(9, 48)
    q, s = _rows(h, one)
    want_q, want_s = fu.rows(_f32(one), False)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)
    flat = _values(rng, (3 * 40 * 48 + 1,), dtype)
    w = flat[1:].view(3, 40, 48)          # weights on any element
    q, s = _u8(3, 40, 48), torch.zeros((3, 1, 1), device="cuda")
    binding.gmm_quantize_fp8_tiles(h, q, s, w)
    want_q, want_s = fu.tiles(_f32(w), False)
    _same_scales(s, want_s)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)


def test_bad_offsets_write_nothing(h):
    torch = _t()
    from ragged_matmul_gb300 import binding
    x = _values(np.random.default_rng(3), (64, 32), "bf16")
    P = fu.pitch(64, 3)
    for off in ([0, 30, 20, 64], [0, 10, 20, 65], [0, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], [0, -1, 5, 6]):
        q_t, ts, q, s = _u8(32, P), _u8(P // 128, 32), _u8(64, 32), torch.full((64, 1), -5.0, device="cuda")
        binding.gmm_quantize_fp8_cols(h, q_t, ts, x, _dev(off), q=q, scales=s)
        assert binding.gmm_query_status(h) == binding.GMM_ERR_BAD_INPUT
        assert (q_t == 0x5A).all() and (ts == 0x5A).all() and (q == 0x5A).all() and (s == -5.0).all()


def test_no_rows(h):
    torch = _t()
    from ragged_matmul_gb300 import binding
    x = torch.zeros((0, 64), device="cuda")
    _rows(h, x)
    P = fu.pitch(0, 3)
    q_t, ts = _u8(64, P), _u8(3, 64)
    binding.gmm_quantize_fp8_cols(h, q_t, ts, x, _dev([0, 0, 0, 0]))
    assert (q_t == 0x5A).all()
    binding.gmm_quantize_fp8_tiles(h, _u8(0, 128, 64), torch.zeros((0, 1, 1), device="cuda"), torch.zeros((0, 128, 64), device="cuda"))
    assert binding.gmm_query_status(h) == binding.GMM_OK


def test_graph_replay(h):
    torch = _t()
    from ragged_matmul_gb300 import binding
    x = _values(np.random.default_rng(1), (300, 272), "bf16")
    off = _dev(_offsets((100, 200)))
    P = fu.pitch(300, 2)
    q_t, ts, q, s = _u8(272, P), _u8(P // 128, 272), _u8(300, 272), torch.zeros((300, 3), device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        binding.gmm_quantize_fp8_cols(h, q_t, ts, x, off, q=q, scales=s)
    x.copy_(_values(np.random.default_rng(2), (300, 272), "bf16"))
    off.copy_(_dev(_offsets((190, 110))))
    graph.replay()
    torch.cuda.synchronize()
    want, want_ts = fu.cols(_f32(x), _offsets((190, 110)), 300, np.full((272, P), 0x5A, np.uint8), np.full((P // 128, 272), 0x5A, np.uint8))
    np.testing.assert_array_equal(ts.cpu().numpy()[[0, 1, 2, 3]], want_ts[[0, 1, 2, 3]])
    np.testing.assert_array_equal(q_t.cpu().numpy(), want)


def test_refusals(h):
    torch = _t()
    from ragged_matmul_gb300 import binding
    x = torch.zeros((8, 64), device="cuda")
    q, s = _u8(8, 64), torch.zeros((8, 1), device="cuda")
    binding.gmm_quantize_fp8(h, q, s, x)
    with pytest.raises(binding.GmmError) as e:       # 24 is not a multiple of 16
        binding.gmm_quantize_fp8(h, _u8(8, 24), s, x[:, :24])
    assert e.value.code == binding.GMM_ERR_INVALID_ARG
    with pytest.raises(binding.GmmError) as e:       # q not on 16 bytes
        binding.gmm_quantize_fp8(h, _u8(8 * 64 + 1)[1:].view(8, 64), s, x)
    assert e.value.code == binding.GMM_ERR_INVALID_ARG
    with pytest.raises(binding.GmmError):
        binding.gmm_quantize_fp8(h, q, s, x, row_slots=torch.zeros(8, dtype=torch.int32, device="cuda"), top_k=0)
    with pytest.raises(ValueError):
        binding.gmm_quantize_fp8(h, q, torch.zeros((8, 2), device="cuda"), x)
    with pytest.raises(ValueError):
        binding.gmm_quantize_fp8(h, q[:7], s, x)
    with pytest.raises(TypeError):
        binding.gmm_quantize_fp8(h, q, s, x.double())
    with pytest.raises(TypeError):
        binding.gmm_quantize_fp8(h, q.to(torch.int8), s, x)
    w = torch.zeros((2, 64, 32), device="cuda")
    with pytest.raises(ValueError):
        binding.gmm_quantize_fp8_tiles(h, _u8(2, 64, 32), torch.zeros((2, 1), device="cuda"), w)
    with pytest.raises(ValueError):
        binding.gmm_quantize_fp8_tiles(h, _u8(2, 32, 64), torch.zeros((2, 1, 1), device="cuda"), w.transpose(1, 2))
    off = _dev([0, 4, 8])
    P = fu.pitch(8, 2)
    binding.gmm_quantize_fp8_cols(h, _u8(64, P), _u8(2, 64), x, off)
    with pytest.raises(ValueError):
        binding.gmm_quantize_fp8_cols(h, _u8(64, P + 128), _u8(2, 64), x, off)
    with pytest.raises(ValueError):
        binding.gmm_quantize_fp8_cols(h, _u8(64, P), _u8(1, 64), x, off)
    with pytest.raises(ValueError):
        binding.gmm_quantize_fp8_cols(h, _u8(64, P), _u8(2, 64), x, off, q=q)
    with pytest.raises(binding.GmmError) as e:
        big = torch.zeros(4098, dtype=torch.int32, device="cuda")
        binding.gmm_quantize_fp8_cols(h, _u8(64, fu.pitch(8, 4097)), _u8(4097, 64), x, big)
    assert e.value.code == binding.GMM_ERR_UNSUPPORTED
    assert binding.gmm_query_status(h) == binding.GMM_OK
