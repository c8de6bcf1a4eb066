"""The 4-bit floating point calls (quantise, dequantise, grouped product) against a 64-bit
reference.

Tolerances, derived from the arithmetic:
- codes: equal, except where the real quotient lies within 2^-22 (relative) of a rounding
  boundary, where either neighbour is right (the kernels' quotients are fp32, half an ulp is
  2^-24, and the divisor s g is itself rounded);
- dequantised values: one fp32 rounding of s g, one of the product, one to the type;
- the product: every instruction adds 64 exact products to the fp32 sum; with S the sum of
  magnitudes, |error| <= (K / 64 + 6) 2^-22 S with the roundings of the scales and of the
  epilogue, before the rounding to bf16 (2^-8 of the result).
"""
import numpy as np
import pytest

import fp4_util as ref

pytestmark = pytest.mark.gpu
FMTS = ("nvfp4", "mxfp4")


def _mods():
    import torch
    from ragged_matmul_gb300 import binding
    from ragged_matmul_gb300 import build as gbuild
    gbuild.build()
    return torch, binding


_handles = {}


def handle(E):
    _, binding = _mods()
    if E not in _handles:
        _handles[E] = binding.gmm_create(E, 0)
    return _handles[E]


def dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def quantise(x, fmt, g=None, row_slots=None, top_k=1, rows=None):
    torch, binding = _mods()
    K = x.shape[1]
    R = x.shape[0] if rows is None else rows
    packed = torch.full((R, K // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((R, ref.pitch(K, fmt)), 0x5A, dtype=torch.uint8, device="cuda")
    h = handle(4)
    gt = None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda")
    rs = None if row_slots is None else dev(np.asarray(row_slots, np.int32))
    binding.gmm_quantize_fp4(h, packed, scales, x, fmt=fmt, row_slots=rs, top_k=top_k, global_scale=gt)
    return packed.cpu().numpy(), scales.cpu().numpy(), binding.gmm_query_status(h)


def check_codes(x, packed, scales, fmt, g=1.0):
    """Exact up to the boundary rule of the module's docstring; x in 64 bits."""
    R, K = x.shape
    b = ref.BLOCK[fmt]
    blocks = x.reshape(R, K // b, b)
    amax = np.abs(blocks).max(-1)
    eps = 2.0 ** -22
    got_s = scales[:, : K // b].astype(np.int64)
    lo, hi = ref.scale_codes(amax * (1 - eps), fmt, g), ref.scale_codes(amax * (1 + eps), fmt, g)
    if fmt == "mxfp4":
        lo = hi = ref.scale_codes(amax, fmt)
    assert ((got_s == lo) | (got_s == hi)).all()
    assert (scales[:, K // b:] == 0).all(), "padding"
    d = (ref.SCALES[fmt][got_s] * (g if fmt == "nvfp4" else 1.0))[..., None]
    got = ref.unpack(packed).reshape(blocks.shape)
    if fmt == "mxfp4" or g == 1.0:      # x / d is decided exactly: every rounding boundary of it is hit or missed exactly
        want = ref.codes(blocks, d)
        near = (ref.codes(blocks * (1 - eps), d) != want) | (ref.codes(blocks * (1 + eps), d) != want)
        assert ((got == want) | near).all()
        if np.array_equal(x, x.astype(np.float16)):
            assert np.array_equal(got, want)
    else:
        a, c = ref.codes(blocks * (1 - eps), d), ref.codes(blocks * (1 + eps), d)
        assert ((got == a) | (got == c)).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (17, 4096), (130, 608), (1, 8192)])
def test_quantise(fmt, dtype, rows, K):
    torch, _ = _mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(rows * K)
    x = (torch.randn((rows, K), generator=g, device="cuda") * 2.5).to(getattr(torch, dtype))
    packed, scales, status = quantise(x, fmt)
    assert status == 0
    check_codes(x.double().cpu().numpy(), packed, scales, fmt)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("g", [0.37, 1.0 / 3.0, 1e-6, 4096.0])
def test_quantise_global_scale(dtype, g):
    torch, _ = _mods()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    g = float(np.float32(g))
    x = (torch.randn((33, 1024), generator=gen, device="cuda") * g * 900).to(getattr(torch, dtype))
    packed, scales, _ = quantise(x, "nvfp4", g=g)
    check_codes(x.double().cpu().numpy(), packed, scales, "nvfp4", g)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantise_ties_and_every_scale(fmt):
    """Blocks whose quotients are exactly the seven rounding boundaries, for scales of every mantissa."""
    torch, _ = _mods()
    bounds = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    b = ref.BLOCK[fmt]
    rows = []
    scales = (np.arange(8, 16) / 8.0)[:, None] * 2.0 ** np.arange(-4, 5)[None] if fmt == "nvfp4" else 2.0 ** np.arange(-20.0, 21.0)
    for s in np.ravel(scales):
        blk = np.zeros(b)
        blk[0] = 6.0
        blk[1:8] = bounds
        blk[8:15] = -bounds
        blk[15] = -0.0
        rows.append(np.tile(blk * s, 32 // b))
    x = np.array(rows)
    assert np.array_equal(x, x.astype(np.float32))
    packed, sc, _ = quantise(torch.from_numpy(x.astype(np.float32)).cuda(), fmt)
    want_s = ref.scale_codes(np.abs(x.reshape(len(x), -1, b)).max(-1), fmt)
    assert np.array_equal(sc[:, : 32 // b].astype(np.int64), want_s)
    d = np.repeat(ref.SCALES[fmt][want_s], b, 1)
    assert np.array_equal(ref.unpack(packed), ref.codes(x, d))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_quantise_special_blocks(fmt, dtype):
    """Zeros, the smallest and largest numbers, infinities and NaN; every block by itself."""
    torch, _ = _mods()
    t = getattr(torch, dtype)
    fi = torch.finfo(t)
    x = torch.zeros((1, 32 * 8), dtype=t, device="cuda")
    x[0, 32] = fi.tiny
    x[0, 64] = fi.max
    x[0, 65] = -fi.max
    x[0, 96] = float("inf")
    x[0, 97] = 1.0
    x[0, 128] = float("nan")
    x[0, 160] = -float("inf")
    x[0, 192:224] = 3.0
    x[0, 224] = fi.tiny / 4        # a subnormal
    packed, scales, _ = quantise(x, fmt)
    b = ref.BLOCK[fmt]
    n = 32 // b
    nan = 0x7F if fmt == "nvfp4" else 0xFF
    s = scales[0, : 8 * n]
    for i in (3, 4, 5):
        assert s[i * n] == nan and (ref.unpack(packed)[0, 32 * i:32 * i + b] == 0).all()
    finite = np.array([0, 1, 2, 6, 7])
    xd = x.double().cpu().numpy().reshape(8, 32)[finite].reshape(len(finite), n, b)
    want = ref.scale_codes(np.abs(xd).max(-1), fmt)
    assert np.array_equal(s.reshape(8, n)[finite], want)
    d = ref.SCALES[fmt][want][..., None]
    assert np.array_equal(ref.unpack(packed).reshape(8, n, b)[finite], ref.codes(xd, d))


@pytest.mark.parametrize("fmt", FMTS)
def test_quantise_gathers_rows(fmt):
    torch, _ = _mods()
    x = torch.randn((5, 224), device="cuda").bfloat16()
    slots = [14, 0, -1, 7, 3, 3, -1]
    packed, scales, status = quantise(x, fmt, row_slots=slots, top_k=3, rows=7)
    assert status == 0
    live = [i for i, s in enumerate(slots) if s >= 0]
    src = x.double().cpu().numpy()[[slots[i] // 3 for i in live]]
    check_codes(src, packed[live], scales[live], fmt)
    for i in (2, 6):
        assert (packed[i] == 0xA5).all() and (scales[i] == 0x5A).all()
    packed, scales, status = quantise(x, fmt, row_slots=[15, 1], top_k=3, rows=2)   # source row 5 of 5
    assert status == -5
    assert (packed[0] == 0xA5).all() and not (packed[1] == 0xA5).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_quantise_strided_and_unaligned(fmt):
    torch, _ = _mods()
    base = torch.randn((9, 200), device="cuda").bfloat16()
    for x in (base[:, 1:161], base[:, 8:168], base[2:3, 3:35].expand(6, 32)):
        packed, scales, _ = quantise(x, fmt)
        check_codes(x.double().cpu().numpy(), packed, scales, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("shift,pitch", [(0, 160), (8, 168), (4, 164), (1, 163), (0, 161), (2, 162)])
def test_quantise_every_alignment(fmt, dtype, shift, pitch):
    """Rows that start on 32 bytes, on 16, on 8, 4 and 2, of each type, gathered and not: the codes and
    scales of the same values in rows on 32 bytes, which the tests above compare with the reference."""
    torch, _ = _mods()
    R, K = 11, 160
    gen = torch.Generator(device="cuda")
    gen.manual_seed(shift + pitch)
    values = (torch.randn((R, K), generator=gen, device="cuda") * 3).to(getattr(torch, dtype))
    values[3, 40] = float("inf")
    buf = torch.full((shift + R * pitch,), 1e4, dtype=values.dtype, device="cuda")
    x = buf[shift:].as_strided((R, K), (pitch, 1))
    x.copy_(values)
    slots = [4, 21, -1, 0, 13, 7]
    for kw in ({}, dict(row_slots=slots, top_k=2, rows=len(slots))):
        got, want = quantise(x, fmt, **kw), quantise(values, fmt, **kw)
        assert got[2] == want[2] == 0
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    finite = [r for r in range(R) if r != 3]
    packed, scales, _ = quantise(x, fmt)
    check_codes(x.double().cpu().numpy()[finite], packed[finite], scales[finite], fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("off", [0, 1])
def test_dequantise_every_code(fmt, dtype, off):
    """All 16 codes under all scale codes; NaN scales give NaN."""
    torch, binding = _mods()
    b = ref.BLOCK[fmt]
    packed = np.tile(ref.pack(np.arange(16)), (256, 32 // 16))
    scales = ref.pad_scales(np.repeat(np.arange(256)[:, None], 32 // b, 1).astype(np.uint8), 32, fmt)
    y = torch.zeros((256, 40), dtype=getattr(torch, dtype), device="cuda")[:, off:off + 32]
    h = handle(4)
    binding.gmm_dequantize_fp4(h, y, dev(packed), dev(scales), fmt=fmt)
    with np.errstate(over="ignore", invalid="ignore"):
        want = torch.from_numpy(ref.values(packed, scales, fmt).astype(np.float32)).to(getattr(torch, dtype))
    assert torch.equal(torch.nan_to_num(y.cpu(), nan=77.0), torch.nan_to_num(want, nan=77.0))
    assert torch.equal(torch.isnan(y.cpu()), torch.isnan(want))


def test_dequantise_global_scale():
    torch, binding = _mods()
    rng = np.random.default_rng(3)
    packed, scales = ref.random_operand(rng, (7,), 320, "nvfp4")
    y = torch.zeros((7, 320), device="cuda")
    g = np.float32(0.123)
    binding.gmm_dequantize_fp4(handle(4), y, dev(packed), dev(scales), global_scale=dev(np.array([g])))
    want = ref.values(packed, scales, "nvfp4", float(g))
    assert (np.abs(y.double().cpu().numpy() - want) <= 2.0 ** -22 * np.abs(want)).all()


# ---------------------------------------------------------------- product

def run_product(a, a_s, off, b, b_s, ids, fmt, ga=None, gb=None, c=None, **epi):
    torch, binding = _mods()
    E, N = b.shape[:2]
    rows = a.shape[0]
    h = handle(E)
    if c is None:
        c = torch.full((rows, N), 0x7FA5, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    stats = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    binding.gmm_run_fp4(h, c, dev(a), dev(np.asarray(off, np.int32)), dev(b), dev(np.asarray(ids, np.int32)), stats,
                        dev(a_s), dev(b_s), fmt=fmt, a_global=None if ga is None else dev(np.array([ga], np.float32)),
                        b_global=None if gb is None else dev(np.asarray(gb, np.float32)), **epi)
    status = binding.gmm_query_status(h)
    return c, stats.cpu().numpy(), status


def check_product(c, C, S, live, K, where=""):
    import torch
    got = c.double().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(C) + (K / 64 + 6) * 2.0 ** -22 * S
    bad = ~(np.abs(got - C) <= tol)[live]
    assert not bad.any(), f"{where}: {bad.sum()} of {bad.size} off, worst {np.abs(got - C)[live].max()}"
    bits = c.view(torch.int16).cpu().numpy()
    assert (bits[~live] == 0x7FA5).all(), f"{where}: rows outside active groups changed"


LOADS = [
    ([1], [0]),
    ([40], [1]),
    ([3, 17, 0, 40], [2, 0, -1, 3]),
    ([129, 224, 225, 31], [3, 1, 1, 0]),
    ([700, 1, 0, 33], [0, -1, 2, 3]),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("loads,ids", LOADS)
@pytest.mark.parametrize("N,K", [(256, 256), (8, 32), (264, 96), (776, 1312)])
def test_product(fmt, loads, ids, N, K):
    rng = np.random.default_rng([N, K, len(loads), sum(loads)])
    off = np.concatenate([[0], np.cumsum(loads)])
    a, a_s = ref.random_operand(rng, (off[-1],), K, fmt)
    b, b_s = ref.random_operand(rng, (4, N), K, fmt, 0.3)
    C, S, live = ref.product(a, a_s, off, b, b_s, ids, fmt)
    c, stats, status = run_product(a, a_s, off, b, b_s, ids, fmt)
    assert status == 0 and stats[1] == sum(0 <= e < 4 for e in ids) and (stats[[0, 2, 3]] == -1).all()
    check_product(c, C, S, live, K)


@pytest.mark.parametrize("fmt", FMTS)
def test_product_exact_integers(fmt):
    """Integer values, scales of one, sums below 256: exact."""
    rng = np.random.default_rng(9)
    K, N, off, ids = 96, 40, [0, 5, 77, 300], [1, 0, 1]
    one = 0x38 if fmt == "nvfp4" else 127
    small = np.array([0, 2, 4, 10, 12])     # 0, 1, 2, -1, -2
    a, b = ref.pack(small[rng.integers(0, 5, (300, K))]), ref.pack(small[rng.integers(0, 5, (2, N, K))])
    a_s = ref.pad_scales(np.full((300, K // ref.BLOCK[fmt]), one, np.uint8), K, fmt)
    b_s = ref.pad_scales(np.full((2, N, K // ref.BLOCK[fmt]), one, np.uint8), K, fmt)
    C, _, live = ref.product(a, a_s, off, b, b_s, ids, fmt)
    c, _, _ = run_product(a, a_s, off, b, b_s, ids, fmt)
    assert np.abs(C).max() < 256 and live.all()
    assert np.array_equal(c.double().cpu().numpy(), C)


@pytest.mark.parametrize("fmt", FMTS)
def test_product_every_scale_position(fmt):
    """One-hot activations: C[r, n] is one weight value times one pair of scales, so a scale
    taken from another row, block, CTA or stage shows at once."""
    rng = np.random.default_rng(11)
    K, N, R = 1088, 520, 450
    b = ref.BLOCK[fmt]
    a_codes = np.zeros((R, K), np.int64)
    k_of = rng.integers(0, K, R)
    a_codes[np.arange(R), k_of] = 2
    def scales(shape):
        if fmt == "nvfp4":
            return rng.integers(8, 0x70, shape).astype(np.uint8)
        return rng.integers(107, 140, shape).astype(np.uint8)
    a_s, b_s = (ref.pad_scales(scales((*lead, K // b)), K, fmt) for lead in ((R,), (2, N)))
    a, w = ref.pack(a_codes), ref.pack(rng.integers(1, 8, (2, N, K)))
    off, ids = [0, 210, 450], [1, 0]
    C, _, _ = ref.product(a, a_s, off, w, b_s, ids, fmt)
    c, _, _ = run_product(a, a_s, off, w, b_s, ids, fmt)
    got = c.double().cpu().numpy()
    assert (np.abs(got - C) <= 2.0 ** -8 * np.abs(C)).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_product_padding_scales_are_not_used(fmt):
    rng = np.random.default_rng(12)
    K, N, off, ids = 160, 72, [0, 50], [0]
    a, a_s = ref.random_operand(rng, (50,), K, fmt)
    b, b_s = ref.random_operand(rng, (1, N), K, fmt)
    n = K // ref.BLOCK[fmt]
    a_s[:, n:] = 0xFF
    b_s[..., n:] = 0x7F if fmt == "nvfp4" else 0xFF
    C, S, live = ref.product(a, a_s, off, b, b_s, ids, fmt)
    c, _, _ = run_product(a, a_s, off, b, b_s, ids, fmt)
    check_product(c, C, S, live, K)


@pytest.mark.parametrize("fmt", FMTS)
def test_product_nan_scale_stays_in_its_row(fmt):
    rng = np.random.default_rng(13)
    K, N, off, ids = 320, 136, [0, 60], [0]
    a, a_s = ref.random_operand(rng, (60,), K, fmt)
    b, b_s = ref.random_operand(rng, (1, N), K, fmt)
    a_s[7, 3] = b_s[0, 100, 2] = 0x7F if fmt == "nvfp4" else 0xFF
    C, S, live = ref.product(a, a_s, off, b, b_s, ids, fmt)
    c, _, _ = run_product(a, a_s, off, b, b_s, ids, fmt)
    got = c.double().cpu().numpy()
    nan = np.zeros_like(C, bool)
    nan[7], nan[:, 100] = True, True
    assert np.array_equal(np.isnan(C), nan) and np.array_equal(np.isnan(got), nan)
    assert (np.abs(got - C)[~nan] <= (2.0 ** -8 * np.abs(C) + (K / 64 + 6) * 2.0 ** -22 * S)[~nan]).all()


def test_product_global_scales_and_epilogue():
    import torch
    rng = np.random.default_rng(14)
    K, N, off, ids = 544, 200, [0, 90, 90, 333], [2, 1, 0]
    a, a_s = ref.random_operand(rng, (333,), K, "nvfp4")
    b, b_s = ref.random_operand(rng, (3, N), K, "nvfp4")
    ga, gb = np.float32(0.07), np.array([0.5, 1.25, 0.031], np.float32)
    bias = rng.standard_normal((3, N)).astype(np.float32)
    scale = rng.uniform(0.1, 1, 333).astype(np.float32)
    C, S, live = ref.product(a, a_s, off, b, b_s, ids, "nvfp4", ga, gb)
    bias_t = torch.from_numpy(bias).bfloat16().cuda()
    c, _, _ = run_product(a, a_s, off, b, b_s, ids, "nvfp4", ga, gb, bias=bias_t,
                          row_scale=torch.from_numpy(scale).cuda(), activation="relu")
    bd = bias_t.double().cpu().numpy()
    want = np.zeros_like(C)
    for g, e in enumerate(ids):
        r = slice(off[g], off[g + 1])
        want[r] = np.maximum(C[r] + bd[e], 0) * scale[r, None]
        S[r] = (S[r] + np.abs(bd[e])) * scale[r, None]
    check_product(c, want, S, live, K)


@pytest.mark.parametrize("fmt", FMTS)
def test_product_long_k_and_many_groups(fmt):
    rng = np.random.default_rng(15)
    K, N, G, E = 8224, 64, 300, 7
    loads = rng.integers(0, 3, G)
    ids = rng.integers(-1, E, G)
    off = np.concatenate([[0], np.cumsum(loads)])
    a, a_s = ref.random_operand(rng, (off[-1],), K, fmt)
    b, b_s = ref.random_operand(rng, (E, N), K, fmt)
    C, S, live = ref.product(a, a_s, off, b, b_s, ids, fmt)
    c, stats, _ = run_product(a, a_s, off, b, b_s, ids, fmt)
    assert stats[1] == (ids >= 0).sum()
    check_product(c, C, S, live, K)


def test_product_bad_inputs_are_reported():
    rng = np.random.default_rng(16)
    a, a_s = ref.random_operand(rng, (40,), 64, "nvfp4")
    b, b_s = ref.random_operand(rng, (2, 16), 64, "nvfp4")
    c, stats, status = run_product(a, a_s, [0, 20, 10, 40], b, b_s, [0, 1, 0], "nvfp4")
    assert status == -5 and stats[1] == 3 and (c.view(__import__("torch").int16).cpu().numpy() == 0x7FA5).all()
    c, stats, status = run_product(a, a_s, [0, 20, 40], b, b_s, [0, 2], "nvfp4")
    C, S, live = ref.product(a, a_s, [0, 20, 40], b, b_s, [0, 2], "nvfp4")
    assert status == -5 and stats[1] == 1
    check_product(c, C, S, live, 64)


def test_product_no_groups():
    torch, binding = _mods()
    a, a_s = ref.random_operand(np.random.default_rng(1), (0,), 64, "nvfp4")
    b, b_s = ref.random_operand(np.random.default_rng(1), (2, 16), 64, "nvfp4")
    c, stats, status = run_product(a, a_s, [0], b, b_s, [], "nvfp4")
    assert status == 0 and stats[1] == 0


def test_product_replays_in_a_graph():
    torch, binding = _mods()
    rng = np.random.default_rng(17)
    K, N, E = 512, 264, 3
    h = handle(E)
    loads = [[100, 0, 60], [5, 150, 5]]
    ops = [(*ref.random_operand(rng, (160,), K, "nvfp4"), *ref.random_operand(rng, (E, N), K, "nvfp4")) for _ in loads]
    bufs = [dev(x) for x in ops[0]]
    off = dev(np.concatenate([[0], np.cumsum(loads[0])]).astype(np.int32))
    ids = dev(np.arange(E, dtype=np.int32))
    stats = torch.zeros(2, dtype=torch.int32, device="cuda")
    c = torch.zeros((160, N), dtype=torch.bfloat16, device="cuda")
    args = (h, c, bufs[0], off, bufs[2], ids, stats, bufs[1], bufs[3])
    binding.gmm_run_fp4(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.gmm_run_fp4(*args)
    for l, o in zip(loads, ops):
        for x, y in zip(bufs, o):
            x.copy_(dev(y))
        off.copy_(dev(np.concatenate([[0], np.cumsum(l)]).astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        C, S, live = ref.product(o[0], o[1], np.concatenate([[0], np.cumsum(l)]), o[2], o[3], range(E), "nvfp4")
        check_product(c, C, S, live, K)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("budget", [200 * 1024, 170 * 1024])
def test_product_with_less_shared_memory(fmt, budget, monkeypatch):
    """Shallower rings on a device that offers a block less shared memory."""
    _, binding = _mods()
    monkeypatch.setenv("GMM_SMEM_BUDGET", str(budget))
    h = binding.gmm_create(2, 0)
    monkeypatch.delenv("GMM_SMEM_BUDGET")
    monkeypatch.setitem(_handles, 2, h)
    rng = np.random.default_rng(18)
    K, N, off, ids = 1600, 328, [0, 250, 611], [1, 0]
    a, a_s = ref.random_operand(rng, (611,), K, fmt)
    b, b_s = ref.random_operand(rng, (2, N), K, fmt)
    C, S, live = ref.product(a, a_s, off, b, b_s, ids, fmt)
    c, _, status = run_product(a, a_s, off, b, b_s, ids, fmt)
    assert status == 0
    check_product(c, C, S, live, K)


def test_product_most_groups():
    """4096 groups (the limit) of zero to two rows, repeated experts, some skipped; one more is refused."""
    torch, binding = _mods()
    rng = np.random.default_rng(19)
    K, N, G, E = 96, 24, 4096, 5
    loads, ids = rng.integers(0, 3, G), rng.integers(-1, E, G)
    off = np.concatenate([[0], np.cumsum(loads)])
    a, a_s = ref.random_operand(rng, (off[-1],), K, "mxfp4")
    b, b_s = ref.random_operand(rng, (E, N), K, "mxfp4")
    C, S, live = ref.product(a, a_s, off, b, b_s, ids, "mxfp4")
    c, stats, status = run_product(a, a_s, off, b, b_s, ids, "mxfp4")
    assert status == 0 and stats[1] == (ids >= 0).sum()
    check_product(c, C, S, live, K)
    with pytest.raises(binding.GmmError) as err:
        run_product(a, a_s, np.append(off, off[-1]), b, b_s, np.append(ids, 0), "mxfp4")
    assert err.value.code == binding.GMM_ERR_UNSUPPORTED


def test_product_launches_leave_the_handle_clean():
    """Launches that claim tiles from the handle's counter, from one end and from both, one after
    the other and between other products of the handle: each finds the counter at zero."""
    torch, binding = _mods()
    rng = np.random.default_rng(20)
    K, N, E = 64, 2048, 8
    h = handle(E)
    w16 = torch.randn((E, N, K), device="cuda").bfloat16()
    for loads in ([900] * 8, [6000, 1, 5, 900, 0, 240, 241, 33], [6000, 1, 5, 900, 0, 240, 241, 33]):
        off = np.concatenate([[0], np.cumsum(loads)])
        a, a_s = ref.random_operand(rng, (off[-1],), K, "nvfp4")
        b, b_s = ref.random_operand(rng, (E, N), K, "nvfp4")
        C, S, live = ref.product(a, a_s, off, b, b_s, range(E), "nvfp4")
        for _ in range(2):
            c, stats, status = run_product(a, a_s, off, b, b_s, range(E), "nvfp4")
            assert status == 0
            check_product(c, C, S, live, K)
        x = torch.randn((int(off[-1]), K), device="cuda").bfloat16()
        y = torch.zeros((int(off[-1]), N), dtype=torch.bfloat16, device="cuda")
        st = torch.zeros(2, dtype=torch.int32, device="cuda")
        binding.gmm_run(h, y, x, dev(off.astype(np.int32)), w16, dev(np.arange(E, dtype=np.int32)), st)
        want = torch.cat([x[off[e]:off[e + 1]].double() @ w16[e].double().t() for e in range(E)])
        assert binding.gmm_query_status(h) == 0
        assert float((y.double() - want).abs().max()) <= float(want.abs().max()) * 2.0 ** -7


def test_two_handles_on_two_streams():
    torch, binding = _mods()
    rng = np.random.default_rng(21)
    K, N, E, R = 512, 1024, 2, 900
    jobs = []
    for i in range(2):
        a, a_s = ref.random_operand(rng, (R,), K, "nvfp4")
        b, b_s = ref.random_operand(rng, (E, N), K, "nvfp4")
        off = [0, 300 + 100 * i, R]
        jobs.append((a, a_s, off, b, b_s, binding.gmm_create(E, 0), torch.cuda.Stream(),
                     torch.zeros((R, N), dtype=torch.bfloat16, device="cuda"),
                     [dev(x) for x in (a, np.asarray(off, np.int32), b, np.arange(E, dtype=np.int32), np.zeros(2, np.int32), a_s, b_s)]))
    torch.cuda.synchronize()
    for _ in range(3):
        for a, a_s, off, b, b_s, h, s, c, d in jobs:
            binding.gmm_run_fp4(h, c, *d, stream=s)
    for a, a_s, off, b, b_s, h, s, c, d in jobs:
        assert binding.gmm_query_status(h, s) == 0
        C, S, live = ref.product(a, a_s, off, b, b_s, range(E), "nvfp4")
        check_product(c, C, S, live, K)
        binding.gmm_destroy(h)


def test_refusals():
    torch, binding = _mods()
    h = handle(2)
    u8 = dict(dtype=torch.uint8, device="cuda")
    x = torch.zeros((4, 64), device="cuda")
    p, s = torch.zeros((4, 32), **u8), torch.zeros((4, 16), **u8)
    for bad in (dict(fmt="int4"), dict(packed=p[:, :31]), dict(scales=s[:3]), dict(x=x.t()), dict(x=x[0]),
                dict(global_scale=torch.ones(2, device="cuda"))):
        kw = dict(packed=p, scales=s, x=x, fmt="nvfp4", global_scale=None)
        kw.update(bad)
        with pytest.raises(ValueError):
            binding.gmm_quantize_fp4(h, **kw)
    with pytest.raises(TypeError):
        binding.gmm_quantize_fp4(h, p, s, x.double())
    with pytest.raises(binding.GmmError):      # mxfp4 has no global scale
        binding.gmm_quantize_fp4(h, p, s, x, fmt="mxfp4", global_scale=torch.ones(1, device="cuda"))
    with pytest.raises(binding.GmmError):      # K not a multiple of 32
        binding.gmm_quantize_fp4(h, torch.zeros((4, 24), **u8), s, x[:, :48])
    with pytest.raises(binding.GmmError):
        binding.gmm_quantize_fp4(h, p, s, x, row_slots=torch.zeros(4, dtype=torch.int32, device="cuda"), top_k=0)
    with pytest.raises(ValueError):            # an output whose rows overlap
        binding.gmm_dequantize_fp4(h, x[:1].expand(4, 64), p, s)
    b, bs = torch.zeros((2, 16, 32), **u8), torch.zeros((2, 16, 16), **u8)
    c = torch.zeros((4, 16), dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    ids = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (dict(fmt="mxfp8"), dict(a_scales=s[:, :8]), dict(b_scales=bs[:1]), dict(b=b[:, :, :16]),
                dict(b_global=torch.ones(3, device="cuda")), dict(c=c[:3])):
        kw = dict(c=c, a=p, a_offsets=off, b=b, expert_ids=ids, expert_usage_stats=st, a_scales=s, b_scales=bs)
        kw.update(bad)
        with pytest.raises(ValueError):
            binding.gmm_run_fp4(h, **kw)
    with pytest.raises(binding.GmmError):      # N not a multiple of 8
        binding.gmm_run_fp4(h, c[:, :12].contiguous(), p, off, b[:, :12].contiguous(), ids, st, s,
                            bs[:, :12].contiguous())
