"""The router's choice, the 8-bit quantisers and the weight gradient at their ends: buffers whose offsets pass 32
bits, calls that are the first of their thread, another current stream, one handle's calls side by side."""
import threading

import numpy as np
import pytest

from tests import choose_util as cu
from tests import fp8_util as fu

pytestmark = pytest.mark.gpu


def _t():
    import torch
    return torch


def test_logits_past_32_bits():
    """Rows whose byte offsets pass 2^32 and element offsets 2^31."""
    torch = _t()
    from ragged_matmul_gb300 import binding
    E, T = 4096, 600_001
    h = binding.gmm_create(E, 0)
    x = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    at = torch.arange(T, device="cuda")
    best, second = at.remainder(4093), (at + 7).remainder(4093)
    x[at, best] = 3.0
    x[at, second] = 2.0
    ids, w = torch.zeros((T, 2), dtype=torch.int32, device="cuda"), torch.zeros((T, 2), device="cuda")
    binding.gmm_route(h, ids, w, x)
    assert torch.equal(ids[:, 0].long(), best) and torch.equal(ids[:, 1].long(), second)
    d = torch.full_like(x, 5.0)
    dw = torch.tensor([1.0, 0.0], device="cuda").expand(T, 2).contiguous()
    binding.gmm_route_grad(h, d, dw, ids, x)
    p = 1 / (1 + np.exp(-1.0))
    want = torch.tensor(p * (1 - p), device="cuda").to(torch.bfloat16)
    assert (d[at, best] == want).all() and (d[at, second] == -want).all()
    d[at, best] = 0.0
    d[at, second] = 0.0
    assert not d.any()
    assert binding.gmm_query_status(h) == binding.GMM_OK
    binding.gmm_destroy(h)


def test_quantisers_past_32_bits():
    torch = _t()
    from ragged_matmul_gb300 import binding
    E, R, K = 3, 600_100, 8192
    h = binding.gmm_create(E, 0)
    x = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda")
    x += torch.arange(R, device="cuda").remainder(13).sub(6).to(torch.bfloat16)[:, None]
    off = torch.tensor([0, 5, 400_003, R], dtype=torch.int32, device="cuda")
    P = binding.fp8_cols_pitch(R, E)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    q, s, q_t, ts = u8(R, K), torch.zeros((R, K // 128), device="cuda"), u8(K, P), u8(P // 128, K)
    binding.gmm_quantize_fp8_cols(h, q_t, ts, x, off, q=q, scales=s)
    assert binding.gmm_query_status(h) == binding.GMM_OK
    q2, s2 = u8(R, K), torch.zeros_like(s)
    binding.gmm_quantize_fp8(h, q2, s2, x)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    for r in (0, 262_143, 262_144, 400_002, 400_003, 524_288, R - 1):
        want_q, want_s = fu.rows(x[r:r + 1].float().cpu().numpy(), False)
        np.testing.assert_array_equal(q[r].cpu().numpy(), want_q[0])
        np.testing.assert_array_equal(s[r].double().cpu().numpy(), want_s[0])
        g = int(np.searchsorted(off.cpu().numpy(), r, side="right")) - 1
        first = int(off[g])
        col = (first // 128 + g) * 128 + r - first
        value = fu.E4M3[q_t[:, col].cpu().numpy()] * fu.E8M0[ts[col // 128].cpu().numpy()]
        np.testing.assert_array_equal(value, x[r].double().cpu().numpy())        # small whole numbers are exact
    binding.gmm_destroy(h)


def test_weight_gradient_past_32_bits():
    torch = _t()
    from ragged_matmul_gb300 import binding
    G, N, K = 40, 8208, 8208
    h = binding.gmm_create(G, 0)
    loads = np.arange(1, G + 1)
    off = np.concatenate([[0], np.cumsum(loads)])
    R = int(off[-1])
    rng = np.random.default_rng(3)
    P = fu.pitch(R, G)
    u8 = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    d, a = rng.choice([0x38, 0xB8, 0x40], (N, P)).astype(np.uint8), rng.choice([0x38, 0xB8, 0x30], (K, P)).astype(np.uint8)
    live = np.zeros(P, bool)
    for g in range(G):
        c = (int(off[g]) // 128 + g) * 128
        live[c:c + loads[g]] = True
    d[:, ~live] = 0
    a[:, ~live] = 0
    ones = lambda w: np.full((P // 128, w), 127, np.uint8)  # noqa: E731
    out = torch.full((G, N, K), float("nan"), device="cuda")
    binding.gmm_weight_grad_fp8(h, out, u8(d), u8(ones(N)), u8(a), u8(ones(K)), torch.tensor(off, dtype=torch.int32, device="cuda"))
    assert binding.gmm_query_status(h) == binding.GMM_OK
    for g in (0, 7, 15, 16, 31, 32, 39):       # 2^30 elements are 15.9 groups, 2^31 31.9
        c = (int(off[g]) // 128 + g) * 128
        rows = [0, 1, 4000, N - 1]
        want = fu.E4M3[d[rows, c:c + loads[g]]] @ fu.E4M3[a[:, c:c + loads[g]]].T
        np.testing.assert_array_equal(out[g, rows].double().cpu().numpy(), want)
    assert not torch.isnan(out.sum())
    binding.gmm_destroy(h)


@pytest.mark.slow
def test_weight_gradient_of_the_longest_pitch():
    """2^30 rows, the most that gmm_quantize_fp8_cols takes: the last block's columns lie behind 2^33 bytes."""
    torch = _t()
    from ragged_matmul_gb300 import binding
    G, N, K, R, n = 1, 16, 16, 1 << 30, 200
    h = binding.gmm_create(G, 0)
    P = fu.pitch(R, G)
    d, a = (torch.zeros((w, P), dtype=torch.uint8, device="cuda") for w in (N, K))
    rng = np.random.default_rng(4)
    codes = [rng.choice([0x38, 0xB8, 0x40], (w, n)).astype(np.uint8) for w in (N, K)]
    c = (R - n) // 128 * 128
    for x, q in zip((d, a), codes):
        x[:, c:c + n] = torch.from_numpy(q).cuda()
    ones = lambda w: torch.full((P // 128, w), 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    out = torch.full((G, N, K), float("nan"), device="cuda")
    binding.gmm_weight_grad_fp8(h, out, d, ones(N), a, ones(K), torch.tensor([R - n, R], dtype=torch.int32, device="cuda"))
    assert binding.gmm_query_status(h) == binding.GMM_OK
    np.testing.assert_array_equal(out[0].double().cpu().numpy(), fu.E4M3[codes[0]] @ fu.E4M3[codes[1]].T)
    binding.gmm_destroy(h)


def _calls(h, E):
    """Each call on inputs of its own: (name, call, result)."""
    torch = _t()
    from ragged_matmul_gb300 import binding
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    T, k, K, N = 70, 2, 144, 272
    logits, ids, w = rnd(T, E), torch.zeros((T, k), dtype=torch.int32, device="cuda"), torch.zeros((T, k), device="cuda")
    chosen = rnd(T, E).topk(k, dim=1).indices.to(torch.int32)
    d = torch.zeros_like(logits)
    x = rnd(T, K).bfloat16()
    q, s = u8(T, K), torch.zeros((T, 2), device="cuda")
    wt, wq, ws = rnd(E, N, K).bfloat16(), u8(E, N, K), torch.zeros((E, 3, 2), device="cuda")
    off = torch.linspace(0, T, E + 1, device="cuda").to(torch.int32)
    P = binding.fp8_cols_pitch(T, E)
    a, a_s, dt, dt_s = u8(K, P), u8(P // 128, K), u8(N, P), u8(P // 128, N)
    dc = rnd(T, N)
    binding.gmm_quantize_fp8_cols(h, dt, dt_s, dc, off)
    a2, a2_s = u8(K, P), u8(P // 128, K)
    binding.gmm_quantize_fp8_cols(h, a2, a2_s, x, off)
    out = torch.zeros((E, N, K), device="cuda")
    torch.cuda.synchronize()
    return {
        "route": (lambda **o: binding.gmm_route(h, ids, w, logits, bias=logits[0], **o), w),
        "route_grad": (lambda **o: binding.gmm_route_grad(h, d, w, chosen, logits, **o), d),
        "rows": (lambda **o: binding.gmm_quantize_fp8(h, q, s, x, **o), q),
        "tiles": (lambda **o: binding.gmm_quantize_fp8_tiles(h, wq, ws, wt, **o), wq),
        "cols": (lambda **o: binding.gmm_quantize_fp8_cols(h, a, a_s, x, off, **o), a),
        "weight_grad": (lambda **o: binding.gmm_weight_grad_fp8(h, out, dt, dt_s, a2, a2_s, off, **o), out),
    }


@pytest.mark.parametrize("name", ["route", "route_grad", "rows", "tiles", "cols", "weight_grad"])
def test_first_call_of_a_thread(name):
    torch = _t()
    from ragged_matmul_gb300 import binding
    h = binding.gmm_create(5, 0)
    call, result = _calls(h, 5)[name]
    call()
    torch.cuda.synchronize()
    want = result.clone()
    if name != "route":
        result.zero_()
    torch.cuda.synchronize()
    got = []

    def run():
        try:
            got.append(call())
        except Exception as err:       # noqa: BLE001
            got.append(err)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    assert got == [0]
    torch.cuda.synchronize()
    assert torch.equal(result, want)
    binding.gmm_destroy(h)


def test_one_handles_calls_side_by_side():
    """These calls keep nothing in the handle but the status word: on several streams at once they give the
    same bits."""
    torch = _t()
    from ragged_matmul_gb300 import binding
    h = binding.gmm_create(5, 0)
    calls = _calls(h, 5)
    want = {}
    for name, (call, result) in calls.items():
        if name != "route_grad":       # it reads the weights that `route` writes
            call()
    torch.cuda.synchronize()
    calls["route_grad"][0]()
    torch.cuda.synchronize()
    want = {n: r.clone() for n, (_, r) in calls.items()}
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        for s, (call, _) in zip(streams, calls.values()):
            call(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(r, want[n]) for n, (_, r) in calls.items())
    assert binding.gmm_query_status(h) == binding.GMM_OK
    binding.gmm_destroy(h)


def test_two_graphs_of_one_handle_in_turn():
    torch = _t()
    from ragged_matmul_gb300 import binding
    E, T, k = 64, 333, 6
    h = binding.gmm_create(E, 0)
    pool = []
    for seed in (1, 2):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        x = torch.randn((T, E), generator=g, device="cuda")
        ids, w, d = torch.zeros((T, k), dtype=torch.int32, device="cuda"), torch.zeros((T, k), device="cuda"), torch.zeros_like(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            binding.gmm_route(h, ids, w, x, scoring="sigmoid", renormalise=bool(seed % 2))
            binding.gmm_route_grad(h, d, w, ids, x, scoring="sigmoid", renormalise=bool(seed % 2))
        pool.append((graph, x, ids, w, d, bool(seed % 2)))
    for _ in range(3):
        for p in pool:
            p[0].replay()
    torch.cuda.synchronize()
    for _, x, ids, w, d, r in pool:
        xs = x.double().cpu().numpy()
        want_ids, want_w = cu.choose(xs, k, scoring="sigmoid", renormalise=r)
        np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
        np.testing.assert_allclose(w.cpu().numpy(), want_w, rtol=2.0 ** -24 * 200)
        want_d, mag = cu.grad(xs, want_ids, w.cpu().numpy(), scoring="sigmoid", renormalise=r)
        assert (np.abs(d.double().cpu().numpy() - want_d) <= mag * 2.0 ** -24 * 200 + 1e-30).all()
    binding.gmm_destroy(h)
