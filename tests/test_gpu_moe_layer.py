"""examples/moe_layer.py: the calls together, against plain references.

serve: the reference repeats the layer in fp32 on the very values that the quantised
operands stand for (dequantised by the library, whose inverse is tested by itself), so what
is left are fp32 sums, bf16 roundings of the intermediate rows and of the result, and rows
of the intermediate quantised from values that differ by a bf16 rounding (2^-8): a value
that crosses a rounding boundary of e2m1 moves by half its step.  A product of hidden values
with errors of at most one e2m1 step each would be off by 2^-2 of the sum's root mean
square; the expected share of crossings (2^-8 over steps of 2^-2 and more: below 2^-6 of the
elements) puts the relative 2-norm below 2^-2 * sqrt(2^-6) = 2^-5.
Experts: bf16 roundings of y, out, d_y, d_rows and d_x, at most five of relative size 2^-8 on
the way to a gradient: relative 2-norms below 5 * 2^-8.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    from ragged_matmul_gb300 import build as gbuild
    gbuild.build()
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,top_k,E", [(1, 2, 4), (37, 3, 5), (530, 4, 16)])
def test_serve(fmt, T, top_k, E):
    import torch
    m = _example()
    g = m.gmm
    h = g.gmm_create(E, 0)
    width, hidden = 160, 288
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x = rnd(T, width).bfloat16()
    router = rnd(width, E)
    up, down = m.Fp4Weights(h, rnd(E, hidden, width) * 0.1, fmt), m.Fp4Weights(h, rnd(E, width, hidden) * 0.1, fmt)
    out = m.serve(h, x, router, up, down, top_k)
    assert g.gmm_query_status(h) == g.GMM_OK

    def values(packed, scales, glob):
        y = torch.empty((packed.shape[0], packed.shape[1] * 2), device="cuda")
        g.gmm_dequantize_fp4(h, y, packed, scales, fmt=fmt, global_scale=glob)
        return y

    def weight(w, e):
        return values(w.packed[e], w.scales[e], None if w.globals is None else w.globals[e:e + 1])

    ids, weights = m.route(x, router, top_k)
    xq = values(*m._quantise(h, x, fmt))
    mid = torch.zeros((T, top_k, hidden), device="cuda")
    for j in range(top_k):
        for t in range(T):
            mid[t, j] = torch.nn.functional.silu(weight_cache(weight, up, int(ids[t, j])) @ xq[t])
    mq = values(*m._quantise(h, mid.reshape(T * top_k, hidden).bfloat16(), fmt)).reshape(T, top_k, hidden)
    want = torch.zeros((T, width), device="cuda")
    for j in range(top_k):
        for t in range(T):
            want[t] += weights[t, j] * (weight_cache(weight, down, int(ids[t, j])) @ mq[t, j])
    assert _rel(out, want) < 2.0 ** -5
    g.gmm_destroy(h)


def weight_cache(weight, w, e):
    cache = w.__dict__.setdefault("_values", {})
    if e not in cache:
        cache[e] = weight(w, e)
    return cache[e]


@pytest.mark.parametrize("T,top_k,E", [(1, 1, 2), (65, 2, 4), (700, 4, 8)])
def test_experts_gradients(T, top_k, E):
    import torch
    m = _example()
    h = m.gmm.gmm_create(E, 0)
    K, N = 96, 136
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, w, G = rnd(T, K).bfloat16(), (rnd(E, N, K) * 0.1).bfloat16(), rnd(T, N).bfloat16()
    ids, weights = m.route(x, rnd(K, E), top_k)
    x1, w1 = x.clone().requires_grad_(), weights.clone().requires_grad_()
    out = m.Experts.apply(x1, w1, ids, w, w.transpose(1, 2).contiguous(), h)
    out.backward(G)
    x2, w2 = x.double().requires_grad_(), weights.double().requires_grad_()
    want = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    for j in range(top_k):
        want = want + w2[:, j:j + 1] * torch.einsum("tk,tnk->tn", x2, w.double()[ids[:, j].long()])
    want.backward(G.double())
    bound = 5 * 2.0 ** -8
    assert _rel(out.detach(), want.detach()) < bound
    assert _rel(x1.grad, x2.grad) < bound
    assert _rel(w1.grad, w2.grad) < bound
    assert m.gmm.gmm_query_status(h) == m.gmm.GMM_OK
    m.gmm.gmm_destroy(h)
