"""Dispatch, combine and its gradient against a 64-bit reference.

Tolerances: the sort and the copies are exact.  combine sums k products by fused
multiply-adds in fp32: |error| <= k 2^-24 S (S the sum of magnitudes), then one rounding to
the type: the result lies between the roundings of the ends of that interval.  d_rows: the
fp32 product (error 2^-24 of it), rounded to the type likewise.  d_weights: n terms in some
order, |error| <= n 2^-24 S.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
DTYPES = ("bfloat16", "float16", "float32")


def rounded_between(got, lo, hi, dtype):
    """got (a tensor of `dtype`) against the interval [lo, hi] in 64 bits, its ends rounded to the type
    (through fp32, moved one step outwards for that rounding; half of fp32's smallest subnormal is added)."""
    import torch
    t = getattr(torch, dtype)
    ends = []
    for x, away in ((lo, -np.inf), (hi, np.inf)):
        f = np.nextafter(np.asarray(x, np.float64).astype(np.float32), np.float32(away))
        ends.append(torch.from_numpy(f).to(t).double().numpy())
    g = got.double().cpu().numpy()
    return (g >= ends[0]) & (g <= ends[1])


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


def sort_reference(e, E):
    T, k = e.shape
    flat = e.reshape(-1).astype(np.int64)
    ok = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(ok, flat, E), kind="stable")[: ok.sum()]
    slot_rows = np.full(T * k, -1, np.int32)
    slot_rows[order] = np.arange(order.size)
    row_slots = np.full(T * k, -1, np.int32)
    row_slots[: order.size] = order
    off = np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=E))])
    return off, slot_rows.reshape(T, k), row_slots


def run_dispatch(e, E, tokens=None, rows=None):
    torch, binding = _mods()
    T, k = e.shape
    h = handle(E)
    off = torch.full((E + 3,), -7, dtype=torch.int32, device="cuda")
    sr = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    rs = torch.full((T * k,), -7, dtype=torch.int32, device="cuda")
    binding.gmm_dispatch(h, off, sr, rs, torch.from_numpy(np.ascontiguousarray(e, np.int32)).cuda(), rows=rows, tokens=tokens)
    status = binding.gmm_query_status(h)
    assert (off[E + 1:] == -7).all()
    return off[: E + 1].cpu().numpy(), sr.cpu().numpy(), rs.cpu().numpy(), status


def experts(rng, T, k, E, drop=0.0, skew=0.0):
    p = (np.arange(1, E + 1.0)) ** -skew
    e = rng.choice(E, size=(T, k), p=p / p.sum()).astype(np.int32)
    e[rng.random((T, k)) < drop] = -1
    return e


SORTS = [
    (1, 1, 1, 0.0), (1, 8, 64, 0.0), (5, 2, 3, 0.5), (256, 8, 64, 0.0), (512, 8, 64, 0.1), (4096, 1, 8, 0.0),
    (513, 8, 64, 0.1), (4097, 1, 1, 0.0), (3001, 6, 255, 0.1), (20000, 2, 8, 0.0), (700, 32, 4096, 0.0),
    (1500, 3, 1025, 0.2), (70000, 1, 5, 0.0), (300, 4, 700, 1.0), (5000, 4, 700, 1.0),
]


@pytest.mark.parametrize("T,k,E,drop", SORTS)
def test_sort(T, k, E, drop):
    rng = np.random.default_rng([T, k, E])
    e = experts(rng, T, k, E, drop, skew=1.0)
    off, sr, rs, status = run_dispatch(e, E)
    want = sort_reference(e, E)
    assert status == 0
    assert np.array_equal(off, want[0]) and np.array_equal(sr, want[1]) and np.array_equal(rs, want[2])


@pytest.mark.parametrize("T,k", [(40, 4), (3000, 4)])
def test_sort_all_to_one_expert_and_bad_ids(T, k):
    e = np.full((T, k), 2, np.int32)
    for bad in (None, 5, 1 << 30):
        x = e.copy()
        if bad is not None:
            x[T // 2, 1] = bad
            x[T - 1, k - 1] = -(1 << 31)
        off, sr, rs, status = run_dispatch(x, 5)
        want = sort_reference(x, 5)
        assert status == (0 if bad is None else -5)
        assert np.array_equal(off, want[0]) and np.array_equal(sr, want[1]) and np.array_equal(rs, want[2])


def test_sort_no_tokens():
    off, _, _, status = run_dispatch(np.zeros((0, 3), np.int32), 4)
    assert status == 0 and (off == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,width", [(1, 1, 2, 1), (7, 3, 4, 33), (200, 8, 16, 2048), (100, 2, 8, 1411),
                                         (2500, 2, 8, 136), (2100, 4, 70, 65)])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_copy(dtype, T, k, E, width, pad):
    torch, _ = _mods()
    rng = np.random.default_rng([T, k, width])
    e = experts(rng, T, k, E, 0.15)
    base = torch.randn((T, width + pad), device="cuda").to(getattr(torch, dtype))
    tokens = base[:, pad // 3: pad // 3 + width]
    rows = torch.full((T * k, width), 7.0, dtype=tokens.dtype, device="cuda")
    off, sr, rs, _ = run_dispatch(e, E, tokens, rows)
    want = sort_reference(e, E)
    assert np.array_equal(sr, want[1]) and np.array_equal(rs, want[2])
    n = int(want[0][-1])
    src = torch.from_numpy(want[2][:n] // k).cuda().long()
    assert torch.equal(rows[:n], tokens[src]) and (rows[n:] == 7.0).all()


def test_copy_keeps_special_values_and_broadcast_rows():
    torch, _ = _mods()
    e = np.array([[0, 1], [1, 0], [1, -1]], np.int32)
    t = torch.tensor([float("nan"), float("inf"), -0.0, 1e-45], device="cuda").expand(3, 4)
    rows = torch.zeros((6, 4), device="cuda")
    run_dispatch(e, 2, t, rows)
    assert torch.equal(rows[:5].view(torch.int32), t[:1].expand(5, 4).contiguous().view(torch.int32))


def slots_for(rng, T, k, drop, extra=0):
    """A random injective map of slots to rows, some dropped."""
    n = T * k + extra
    sr = rng.permutation(n)[: T * k].reshape(T, k).astype(np.int32)
    sr[rng.random((T, k)) < drop] = -1
    return sr, n


COMBINES = [(1, 1, 1), (1, 8, 2048), (3, 5, 33), (129, 2, 264), (200, 8, 1411), (33, 32, 72), (5, 11, 4096), (2000, 2, 64)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,width", COMBINES)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(dtype, T, k, width, weighted):
    torch, binding = _mods()
    rng = np.random.default_rng([T, k, width])
    sr, n = slots_for(rng, T, k, 0.2, 5)
    sr[T // 2] = -1                                   # a token without any row
    rows = torch.from_numpy(rng.standard_normal((n, width)).astype(np.float32)).cuda().to(getattr(torch, dtype))
    w = rng.standard_normal((T, k)).astype(np.float32) if weighted else None
    out = torch.full((T, width + 3), 9.0, dtype=rows.dtype, device="cuda")[:, 1:1 + width] if T % 2 else \
        torch.full((T, width), 9.0, dtype=rows.dtype, device="cuda")
    binding.gmm_combine(handle(4), out, rows, torch.from_numpy(sr).cuda(), None if w is None else torch.from_numpy(w).cuda())
    assert binding.gmm_query_status(handle(4)) == 0
    x = rows.double().cpu().numpy()
    ww = np.where(sr >= 0, 1.0 if w is None else w.astype(np.float64), 0.0)
    terms = ww[:, :, None] * x[np.maximum(sr, 0)]
    want, S = terms.sum(1), np.abs(terms).sum(1)
    e32 = k * 2.0 ** -24 * S
    assert rounded_between(out, want - e32, want + e32, dtype).all()
    assert (out[T // 2] == 0).all()


def test_combine_ignores_what_dropped_slots_would_hold():
    """NaN and infinities in rows and weights that no kept slot names do not reach the sums."""
    torch, binding = _mods()
    rows = torch.tensor([[1.0, 2.0], [float("nan"), float("inf")], [4.0, 8.0]], device="cuda")
    sr = torch.tensor([[0, -1], [-1, 2], [-1, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, float("nan")], [float("inf"), 2.0], [float("nan"), 1.0]], device="cuda")
    out = torch.full((3, 2), -1.0, device="cuda")
    binding.gmm_combine(handle(4), out, rows, sr, w)
    assert torch.equal(out.cpu(), torch.tensor([[0.5, 1.0], [8.0, 16.0], [0.0, 0.0]]))
    d_rows, d_w = torch.full((3, 2), 3.0, device="cuda"), torch.full((3, 2), 3.0, device="cuda")
    binding.gmm_combine_grad(handle(4), d_rows, d_w, torch.ones((3, 2), device="cuda"), rows, sr, w)
    assert torch.equal(d_rows.cpu(), torch.tensor([[0.5, 0.5], [3.0, 3.0], [2.0, 2.0]]))
    assert torch.equal(d_w.cpu(), torch.tensor([[3.0, 0.0], [0.0, 12.0], [0.0, 0.0]]))


def test_combine_reports_rows_past_the_end():
    torch, binding = _mods()
    rows = torch.ones((2, 8), device="cuda")
    sr = torch.tensor([[0, 2], [1, 1 << 30]], dtype=torch.int32, device="cuda")
    out = torch.zeros((2, 8), device="cuda")
    binding.gmm_combine(handle(4), out, rows, sr)
    assert binding.gmm_query_status(handle(4)) == -5 and (out == 1).all()
    d_rows, d_w = torch.zeros((2, 8), device="cuda"), torch.ones((2, 2), device="cuda")
    binding.gmm_combine_grad(handle(4), d_rows, d_w, out, rows, sr)
    assert binding.gmm_query_status(handle(4)) == -5 and (d_rows == 1).all()
    assert torch.equal(d_w.cpu(), torch.tensor([[8.0, 0.0], [8.0, 0.0]]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,width", COMBINES)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_grad(dtype, T, k, width, weighted):
    torch, binding = _mods()
    rng = np.random.default_rng([T, k, width, 1])
    sr, n = slots_for(rng, T, k, 0.2, 5)
    mk = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda().to(getattr(torch, dtype))
    rows = mk(n, width)
    d_out = mk(T, width + 5)[:, 2:2 + width] if T % 2 else mk(T, width)
    w = rng.standard_normal((T, k)).astype(np.float32) if weighted else None
    d_rows = torch.full((n, width), 7.0, dtype=rows.dtype, device="cuda")
    d_w = torch.full((T, k), 7.0, device="cuda")
    args = (torch.from_numpy(sr).cuda(), None if w is None else torch.from_numpy(w).cuda())
    binding.gmm_combine_grad(handle(4), d_rows, d_w, d_out, rows, *args)
    g, x = d_out.double().cpu().numpy(), rows.double().cpu().numpy()
    kept = sr >= 0
    want = np.full((n, width), 7.0)
    named = np.zeros(n, bool)
    for t, j in zip(*np.nonzero(kept)):
        want[sr[t, j]] = (1.0 if w is None else float(w[t, j])) * g[t]
        named[sr[t, j]] = True
    e32 = 2.0 ** -24 * np.abs(want)
    got = d_rows.double().cpu().numpy()
    assert rounded_between(d_rows, want - e32, want + e32, dtype)[named].all() and (got[~named] == 7.0).all()
    terms = g[:, None, :] * x[np.maximum(sr, 0)]
    want_w = np.where(kept, terms.sum(2), 0.0)
    tol_w = np.where(kept, width * 2.0 ** -24 * np.abs(terms).sum(2), 0.0)
    assert (np.abs(d_w.double().cpu().numpy() - want_w) <= tol_w).all()
    again = torch.full_like(d_rows, 7.0)
    binding.gmm_combine_grad(handle(4), again, None, d_out, None, *args)
    assert torch.equal(again, d_rows)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("width", [1, 2, 3, 62, 63, 64, 65, 66, 127, 129, 513, 2047, 4098])
@pytest.mark.parametrize("shift", [0, 1])
def test_rows_on_any_two_bytes(dtype, width, shift):
    """Rows of 2-byte elements whose words do not coincide: every parity of the source, the result
    and the gradients, and nothing written beside them (exact values: integers, weights 1 and 2)."""
    torch, binding = _mods()
    rng = np.random.default_rng([width, shift])
    dt, h = getattr(torch, dtype), handle(4)
    for T, k in ((5, 1), (6, 2), (7, 3), (4, 7)):
        sr = rng.permutation(T * k).astype(np.int32).reshape(T, k)
        sr[rng.random((T, k)) < 0.2] = -1
        srt = torch.from_numpy(sr).cuda()
        w = rng.integers(1, 3, (T, k)).astype(np.float32)
        n = T * k

        def flat(count, at, fill=None):
            """`count` elements `at` elements into a buffer, and the buffer."""
            buf = torch.full((count + 8,), 99.0, dtype=dt, device="cuda")
            view = buf[at:at + count]
            if fill is not None:
                view.copy_(fill)
            return view, buf

        ints = lambda *s: torch.from_numpy(rng.integers(-4, 5, s).astype(np.float32)).cuda()
        rows = flat(n * width, shift, ints(n * width).to(dt))[0].view(n, width)
        x = rows.double().cpu().numpy()
        ww = np.where(sr >= 0, w, 0.0)
        for at in (0, 1, 2, 3):
            for pitch in (width, width + 1, width + 2):
                out_v, out_b = flat((T - 1) * pitch + width, at)
                out = out_v.as_strided((T, width), (pitch, 1))
                binding.gmm_combine(h, out, rows, srt, torch.from_numpy(w).cuda())
                want = torch.full_like(out_b, 99.0)
                want[at:at + out_v.numel()].as_strided((T, width), (pitch, 1)).copy_(
                    torch.from_numpy((ww[:, :, None] * x[np.maximum(sr, 0)]).sum(1)).cuda().to(dt))
                assert torch.equal(out_b, want), (T, k, at, pitch)
            g_v, _ = flat((T - 1) * (width + 1) + width, at, ints((T - 1) * (width + 1) + width).to(dt))
            d_out = g_v.as_strided((T, width), (width + 1, 1))
            g = d_out.double().cpu().numpy()
            d_v, d_b = flat(n * width, (at + shift) % 3)
            d_w = torch.full((T, k), 7.0, device="cuda")
            binding.gmm_combine_grad(h, d_v.view(n, width), d_w, d_out, rows, srt, torch.from_numpy(w).cuda())
            want = torch.full_like(d_b, 99.0)
            wr = want[(at + shift) % 3:(at + shift) % 3 + n * width].view(n, width)
            for t, j in zip(*np.nonzero(sr >= 0)):
                wr[int(sr[t, j])] = torch.from_numpy(w[t, j] * g[t]).cuda().to(dt)
            assert torch.equal(d_b, want), (T, k, at)
            want_w = np.where(sr >= 0, (g[:, None, :] * x[np.maximum(sr, 0)]).sum(2), 0.0)
            assert (d_w.cpu().numpy() == want_w).all(), (T, k, at)


def test_gradient_against_differences():
    """The weighted sum is linear in the rows and in the weights, so a central difference of the
    forward call with step 1 is its derivative up to rounding: with L = <out, G> and every
    |term| of out at most B, the difference is off by at most 2 (k + 1) 2^-24 k B sum|G|."""
    torch, binding = _mods()
    rng = np.random.default_rng(8)
    T, k, width, h = 6, 3, 20, handle(4)
    sr, n = slots_for(rng, T, k, 0.2)
    srt = torch.from_numpy(sr).cuda()
    rows = rng.uniform(-1, 1, (n, width)).astype(np.float32)
    w = rng.uniform(-1, 1, (T, k)).astype(np.float32)
    G = rng.uniform(-1, 1, (T, width)).astype(np.float32)

    def loss(r, ww):
        out = torch.empty((T, width), device="cuda")
        binding.gmm_combine(h, out, torch.from_numpy(r).cuda(), srt, torch.from_numpy(ww).cuda())
        return float((out.double().cpu().numpy() * G).sum())

    d_rows, d_w = torch.zeros((n, width), device="cuda"), torch.zeros((T, k), device="cuda")
    binding.gmm_combine_grad(h, d_rows, d_w, torch.from_numpy(G).cuda(), torch.from_numpy(rows).cuda(), srt,
                             torch.from_numpy(w).cuda())
    tol = 2 * (k + 1) * 2.0 ** -24 * k * 4 * np.abs(G).sum()
    for t in range(T):
        for j in range(k):
            up, dn = w.copy(), w.copy()
            up[t, j] += 1
            dn[t, j] -= 1
            step = float(up[t, j]) - float(dn[t, j])
            assert abs((loss(rows, up) - loss(rows, dn)) / step - float(d_w[t, j])) <= tol
    for r in range(n):
        c = int(rng.integers(width))
        up, dn = rows.copy(), rows.copy()
        up[r, c] += 1
        dn[r, c] -= 1
        step = float(up[r, c]) - float(dn[r, c])
        assert abs((loss(up, w) - loss(dn, w)) / step - float(d_rows[r, c])) <= tol


def test_gradient_of_the_copy_is_combine():
    torch, binding = _mods()
    rng = np.random.default_rng(9)
    T, k, E, width = 50, 4, 6, 40
    e = experts(rng, T, k, E, 0.1)
    off, sr, rs, _ = run_dispatch(e, E)
    d_rows = rng.standard_normal((T * k, width)).astype(np.float32)
    out = torch.zeros((T, width), device="cuda")
    binding.gmm_combine(handle(E), out, torch.from_numpy(d_rows).cuda(), torch.from_numpy(sr).cuda())
    want, S = np.zeros((T, width)), np.zeros((T, width))
    for r, s in enumerate(rs):
        if s >= 0:
            want[s // k] += d_rows[r]
            S[s // k] += np.abs(d_rows[r])
    assert (np.abs(out.double().cpu().numpy() - want) <= (k + 1) * 2.0 ** -24 * S).all()


def test_stream_and_graph():
    """The calls follow the given stream and replay in a CUDA graph on new inputs."""
    torch, binding = _mods()
    rng = np.random.default_rng(10)
    h, E, k = handle(6), 6, 2
    for T in (60, 3000):
        e = torch.zeros((T, k), dtype=torch.int32, device="cuda")
        tokens = torch.zeros((T, 24), device="cuda")
        off, sr = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros((T, k), dtype=torch.int32, device="cuda")
        rs, rows = torch.zeros(T * k, dtype=torch.int32, device="cuda"), torch.zeros((T * k, 24), device="cuda")
        out = torch.zeros((T, 24), device="cuda")
        s = torch.cuda.Stream()
        torch.cuda.synchronize()

        def calls(stream=None):
            binding.gmm_dispatch(h, off, sr, rs, e, rows=rows, tokens=tokens, stream=stream)
            binding.gmm_combine(h, out, rows, sr, stream=stream)
        calls(s)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls()
        for i in range(2):
            ids = experts(rng, T, k, E, 0.0)
            e.copy_(torch.from_numpy(ids).cuda())
            tokens.copy_(torch.randn((T, 24), device="cuda"))
            graph.replay()
            torch.cuda.synchronize()
            assert np.array_equal(rs.cpu().numpy(), sort_reference(ids, E)[2])
            assert torch.equal(out, tokens * 2)


def test_refusals():
    torch, binding = _mods()
    h = handle(4)
    i32 = dict(dtype=torch.int32, device="cuda")
    e = torch.zeros((5, 2), **i32)
    off, sr, rs = torch.zeros(5, **i32), torch.zeros((5, 2), **i32), torch.zeros(10, **i32)
    t, r = torch.zeros((5, 8), device="cuda"), torch.zeros((10, 8), device="cuda")
    for bad in (dict(off=off[:4]), dict(sr=sr[:4]), dict(rs=rs[:9]), dict(tokens=None), dict(rows=r[:9]),
                dict(tokens=t[:4]), dict(tokens=torch.zeros((8, 5), device="cuda").t()), dict(e=e[0])):
        kw = dict(off=off, sr=sr, rs=rs, e=e, rows=r, tokens=t)
        kw.update(bad)
        with pytest.raises(ValueError):
            binding.gmm_dispatch(h, kw["off"], kw["sr"], kw["rs"], kw["e"], rows=kw["rows"], tokens=kw["tokens"])
    with pytest.raises(TypeError):
        binding.gmm_dispatch(h, off, sr, rs, e, rows=r.half(), tokens=t)
    with pytest.raises(TypeError):
        binding.gmm_dispatch(h, off, sr, rs, e.long(), rows=r, tokens=t)
    big = torch.zeros((2, 33), **i32)
    with pytest.raises(binding.GmmError) as err:
        binding.gmm_dispatch(h, off, big.clone(), torch.zeros(66, **i32), big)
    assert err.value.code == binding.GMM_ERR_UNSUPPORTED
    out = torch.zeros((5, 8), device="cuda")
    for bad in (dict(out=out[:4]), dict(out=out[:1].expand(5, 8)), dict(rows=r[:, :4].contiguous()),
                dict(weights=torch.ones((5, 3), device="cuda"))):
        kw = dict(out=out, rows=r, weights=None)
        kw.update(bad)
        with pytest.raises(ValueError):
            binding.gmm_combine(h, kw["out"], kw["rows"], sr, kw["weights"])
    with pytest.raises(ValueError):
        binding.gmm_combine_grad(h, r, torch.zeros((5, 2), device="cuda"), out, None, sr)
