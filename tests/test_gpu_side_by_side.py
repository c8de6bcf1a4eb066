"""Calls that share a handle, run at once on streams of their own or as the first one of a thread.  Every result is
overwritten before, so that a call which writes nothing, or a part, is seen; every call has operands of its own."""
import threading

import pytest

pytestmark = pytest.mark.gpu


def _calls(h, E):
    """{name: (call, results)}."""
    import torch
    from ragged_matmul_gb300 import binding
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    T, k, K, N = 333, 2, 144, 272
    logits, ids, w = rnd(T, E), torch.zeros((T, k), dtype=torch.int32, device="cuda"), torch.zeros((T, k), device="cuda")
    bias = 0.1 * rnd(E)
    chosen, dw, d = rnd(T, E).topk(k, dim=1).indices.to(torch.int32), rnd(T, k), torch.zeros((T, E), device="cuda")
    grad_of = logits.clone()
    x, q, s = rnd(T, K).bfloat16(), u8(T, K), torch.zeros((T, 2), device="cuda")
    wt, wq, ws = rnd(E, N, K).bfloat16(), u8(E, N, K), torch.zeros((E, 3, 2), device="cuda")
    off = torch.linspace(0, T, E + 1, device="cuda").to(torch.int32)
    P = binding.fp8_cols_pitch(T, E)
    xc, a, a_s, aq, aqs = rnd(T, K).half(), u8(K, P), u8(P // 128, K), u8(T, K), torch.zeros((T, 2), device="cuda")
    d_t, d_ts, a_t, a_ts = u8(N, P), u8(P // 128, N), u8(K, P), u8(P // 128, K)
    binding.gmm_quantize_fp8_cols(h, d_t, d_ts, rnd(T, N), off)
    binding.gmm_quantize_fp8_cols(h, a_t, a_ts, rnd(T, K), off)
    out = torch.zeros((E, N, K), device="cuda")
    torch.cuda.synchronize()
    return {
        "route": (lambda **o: binding.gmm_route(h, ids, w, logits, bias=bias, **o), (ids, w)),
        "route_grad": (lambda **o: binding.gmm_route_grad(h, d, dw, chosen, grad_of, **o), (d,)),
        "rows": (lambda **o: binding.gmm_quantize_fp8(h, q, s, x, **o), (q, s)),
        "tiles": (lambda **o: binding.gmm_quantize_fp8_tiles(h, wq, ws, wt, **o), (wq, ws)),
        "cols": (lambda **o: binding.gmm_quantize_fp8_cols(h, a, a_s, xc, off, q=aq, scales=aqs, **o), (a, a_s, aq, aqs)),
        "weight_grad": (lambda **o: binding.gmm_weight_grad_fp8(h, out, d_t, d_ts, a_t, a_ts, off, **o), (out,)),
    }


def _overwrite(results):
    for r in results:
        r.fill_(float("nan") if r.is_floating_point() else 0x5A)


def _same(results, want):
    import torch
    return all(torch.equal(r, v) for r, v in zip(results, want))


def _wanted(call, results):
    """The results of a call alone, which is not what they hold before it."""
    import torch
    _overwrite(results)
    call()
    torch.cuda.synchronize()
    want = [r.clone() for r in results]
    assert not any(torch.isnan(r).any() for r in want if r.is_floating_point())
    _overwrite(results)
    torch.cuda.synchronize()
    assert not any(torch.equal(r, v) for r, v in zip(results, want))
    return want


@pytest.mark.parametrize("name", ["route", "route_grad", "rows", "tiles", "cols", "weight_grad"])
def test_the_first_call_of_a_thread_writes(name):
    import torch
    from ragged_matmul_gb300 import binding
    h = binding.gmm_create(5, 0)
    call, results = _calls(h, 5)[name]
    want = _wanted(call, results)
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
    assert _same(results, want)
    binding.gmm_destroy(h)


def test_calls_side_by_side_write_what_each_writes_alone():
    import torch
    from ragged_matmul_gb300 import binding
    h = binding.gmm_create(5, 0)
    calls = _calls(h, 5)
    want = {n: _wanted(*c) for n, c in calls.items()}
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        for _, results in calls.values():
            _overwrite(results)
        torch.cuda.synchronize()
        for _ in range(3):
            for s, (call, _) in zip(streams, calls.values()):
                call(stream=s)
        torch.cuda.synchronize()
        assert all(_same(results, want[n]) for n, (_, results) in calls.items())
    assert binding.gmm_query_status(h) == binding.GMM_OK
    binding.gmm_destroy(h)
