"""examples/moe_layer.py: the router's choice and the expert product in 8 bits together, with all gradients.

Bounds.  An e4m3 value is off by half a step, 2^-4 of it at most, and such errors are independent of one
another and without a mean.  The error of a sum of products of two quantised operands then has an expected
square of at most 2 (2^-4)^2 times the sum of the products' squares, which for independent operands without a
mean is the expected square of the sum itself: relative 2-norms below sqrt(2) 2^-4, plus a few bf16 roundings
of 2^-8.  A gradient that goes through two such products one after the other (the router's, through the rows
of the forward product and their weights) stays below twice that."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BOUND = 2 ** 0.5 * 2.0 ** -4 + 4 * 2.0 ** -8


def _example():
    from ragged_matmul_gb300 import build as gbuild
    gbuild.build()
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def _layer(m, h, x, router, w, top_k, options, bias):
    weights, ids = m.Route.apply(x @ router, top_k, h, options, bias)
    return m.Fp8Experts.apply(x, weights, ids, w, h), weights, ids


def _plain(x, router, w, ids, options):
    """The same layer in 64 bits, the choice given."""
    import torch
    logits = x @ router
    s = logits.sigmoid() if options.get("scoring") == "sigmoid" else logits.softmax(1)
    p = s.gather(1, ids.long())
    p = options.get("scale", 1.0) * p / p.sum(1, keepdim=True)
    out = 0
    for j in range(ids.shape[1]):
        out = out + p[:, j:j + 1] * torch.einsum("tk,tnk->tn", x, w[ids[:, j].long()])
    return out


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,top_k,E,K,N", [(65, 2, 4, 96, 144), (700, 4, 8, 272, 256), (301, 8, 16, 144, 400)])
def test_layer_and_gradients(T, top_k, E, K, N, scoring):
    import torch
    m = _example()
    h = m.gmm.gmm_create(E, 0)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, router, w, G = rnd(T, K).bfloat16(), (rnd(K, E) * K ** -0.5).bfloat16(), (rnd(E, N, K) * 0.1).bfloat16(), rnd(T, N).bfloat16()
    options = dict(scoring=scoring, expert_groups=4, top_groups=2, group_top=1, scale=2.5)
    if top_k > E // 2:
        options = dict(scoring=scoring, scale=2.5)
    bias = 0.01 * rnd(E)
    leaves = [t.clone().requires_grad_() for t in (x, router, w)]
    out, weights, ids = _layer(m, h, *leaves, top_k, options, bias)
    out.backward(G)
    assert m.gmm.gmm_query_status(h) == m.gmm.GMM_OK
    assert int(ids.min()) >= 0
    plain = [t.double().requires_grad_() for t in (x, router, w)]
    want = _plain(*plain, ids, options)
    want.backward(G.double())
    assert _rel(out.detach(), want.detach()) < BOUND
    assert _rel(leaves[0].grad, plain[0].grad) < 2 * BOUND
    assert _rel(leaves[1].grad, plain[1].grad) < 2 * BOUND
    assert _rel(leaves[2].grad, plain[2].grad) < BOUND
    first = [t.grad.clone() for t in leaves]          # the same bits again
    for t in leaves:
        t.grad = None
    _layer(m, h, *leaves, top_k, options, bias)[0].backward(G)
    assert all(torch.equal(a, t.grad) for a, t in zip(first, leaves))
    m.gmm.gmm_destroy(h)


def test_masked_tokens_and_experts():
    """A padded batch: tokens whose logits are all masked get no expert, no output and no gradient, and an
    expert that is masked for everyone gets a gradient of zeros."""
    import torch
    m = _example()
    E, T, K, N, top_k = 6, 90, 64, 80, 2
    h = m.gmm.gmm_create(E, 0)
    torch.manual_seed(1)
    x = torch.randn((T, K), device="cuda").bfloat16().requires_grad_()
    w = (torch.randn((E, N, K), device="cuda") * 0.1).bfloat16().requires_grad_()
    mask = torch.zeros((T, E), device="cuda")
    mask[50:] = -float("inf")
    mask[:, 3] = -float("inf")
    logits = torch.randn((T, E), device="cuda").requires_grad_()
    weights, ids = m.Route.apply(logits + mask, top_k, h, {})
    out = m.Fp8Experts.apply(x, weights, ids, w, h)
    out.sum().backward()
    assert m.gmm.gmm_query_status(h) == m.gmm.GMM_OK
    assert (ids[50:] == -1).all() and not (ids == 3).any()
    assert (out[50:] == 0).all() and (x.grad[50:] == 0).all() and (logits.grad[50:] == 0).all()
    assert (w.grad[3] == 0).all() and (w.grad[0] != 0).any()
    assert all(torch.isfinite(t.grad).all() for t in (x, w, logits))
    m.gmm.gmm_destroy(h)


def test_without_tokens():
    import torch
    m = _example()
    h = m.gmm.gmm_create(3, 0)
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda").requires_grad_()
    w = torch.randn((3, 48, 64), device="cuda").bfloat16().requires_grad_()
    weights, ids = m.Route.apply(torch.zeros((0, 3), device="cuda").requires_grad_(), 2, h, {})
    out = m.Fp8Experts.apply(x, weights, ids, w, h)
    out.sum().backward()
    assert out.shape == (0, 48) and x.grad.shape == (0, 64)
    assert (w.grad == 0).all()
    assert m.gmm.gmm_query_status(h) == m.gmm.GMM_OK
    m.gmm.gmm_destroy(h)


def test_gradients_of_any_strides():
    import torch
    m = _example()
    E, T, K, N = 4, 40, 64, 48
    h = m.gmm.gmm_create(E, 0)
    torch.manual_seed(2)
    x, w = torch.randn((T, K), device="cuda").bfloat16(), torch.randn((E, N, K), device="cuda").bfloat16()
    logits = torch.randn((T, E), device="cuda")
    G = torch.randn((T, N), device="cuda").bfloat16()
    grads = []
    for g in (G, G.t().contiguous().t(), G.repeat(1, 2)[:, :N]):
        leaves = [t.clone().requires_grad_() for t in (x, w, logits)]
        weights, ids = m.Route.apply(leaves[2], 2, h, dict(renormalise=False))
        m.Fp8Experts.apply(leaves[0], weights, ids, leaves[1], h).backward(g)
        grads.append([t.grad for t in leaves])
    for other in grads[1:]:
        assert all(torch.equal(a, b) for a, b in zip(grads[0], other))
    m.gmm.gmm_destroy(h)


def test_a_training_step_in_a_graph():
    """Forward and backward captured once and replayed on other inputs give what eager calls give."""
    import torch
    m = _example()
    E, T, K, N, top_k = 8, 200, 128, 144, 2
    h = m.gmm.gmm_create(E, 0)
    torch.manual_seed(3)
    x, w = torch.randn((T, K), device="cuda").bfloat16(), (torch.randn((E, N, K), device="cuda") * 0.1).bfloat16()
    logits, G = torch.randn((T, E), device="cuda"), torch.randn((T, N), device="cuda").bfloat16()

    def step(x, logits, w):
        weights, ids = m.Route.apply(logits, top_k, h, dict(scoring="sigmoid"), None)
        out = m.Fp8Experts.apply(x, weights, ids, w, h)
        return (out, *torch.autograd.grad(out, (x, logits, w), G))

    static = [t.clone().requires_grad_() for t in (x, logits, w)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step(*static)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(*static)
    with torch.no_grad():
        static[0].copy_(torch.randn((T, K), device="cuda"))
        static[1].copy_(torch.randn((T, E), device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    eager = step(*[t.detach().clone().requires_grad_() for t in static])
    assert all(torch.equal(a, b) for a, b in zip(captured, eager))
    assert m.gmm.gmm_query_status(h) == m.gmm.GMM_OK
    m.gmm.gmm_destroy(h)
