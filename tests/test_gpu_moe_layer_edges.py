"""examples/moe_layer.py on a batch without tokens and under the gradients that autograd really passes."""
import pytest
import torch
from test_gpu_moe_layer import _example

pytestmark = pytest.mark.gpu


def _layer(T, E=4, top_k=2, K=96, N=136, seed=3):
    m = _example()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, w = rnd(T, K).bfloat16(), (rnd(E, N, K) * 0.1).bfloat16()
    ids, weights = m.route(x, rnd(K, E), top_k)
    x, weights = x.requires_grad_(), weights.detach().requires_grad_()
    h = m.gmm.gmm_create(E, 0)
    out = m.Experts.apply(x, weights, ids, w, w.transpose(1, 2).contiguous(), h)
    return m, h, x, weights, out


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_serve_without_tokens(fmt):
    m = _example()
    E, width, hidden = 4, 160, 288
    h = m.gmm.gmm_create(E, 0)
    up = m.Fp4Weights(h, torch.randn((E, hidden, width), device="cuda"), fmt)
    down = m.Fp4Weights(h, torch.randn((E, width, hidden), device="cuda"), fmt)
    x = torch.zeros((0, width), dtype=torch.bfloat16, device="cuda")
    out = m.serve(h, x, torch.randn((width, E), device="cuda"), up, down, 2)
    assert out.shape == (0, width) and m.gmm.gmm_query_status(h) == m.gmm.GMM_OK
    m.gmm.gmm_destroy(h)


def test_training_without_tokens():
    m, h, x, weights, out = _layer(0)
    out.backward(torch.zeros_like(out))
    assert x.grad.shape == x.shape and weights.grad.shape == weights.shape
    assert m.gmm.gmm_query_status(h) == m.gmm.GMM_OK
    m.gmm.gmm_destroy(h)


@pytest.mark.parametrize("kind", ["sum", "transposed", "row", "column"])
def test_gradients_of_any_strides(kind):
    """The gradient that reaches the layer may be expanded (out.sum()), column-major or one row for
    all tokens; it gives what its contiguous copy gives."""
    m, h, x, weights, out = _layer(37)
    T, N = out.shape
    g = torch.randn((N, T), device="cuda").bfloat16()
    grad = {"sum": torch.ones((), device="cuda").bfloat16().expand(T, N), "transposed": g.t(),
            "row": g.t()[:1].contiguous().expand(T, N), "column": g.t()[:, :1].expand(T, N)}[kind]
    assert not grad.is_contiguous()
    want = torch.autograd.grad(out, (x, weights), grad.contiguous(), retain_graph=True)
    got = torch.autograd.grad(out, (x, weights), grad, retain_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    if kind == "sum":
        out.sum().backward()
        assert torch.equal(x.grad, want[0]) and torch.equal(weights.grad, want[1])
    assert m.gmm.gmm_query_status(h) == m.gmm.GMM_OK
    m.gmm.gmm_destroy(h)


def test_second_derivatives_are_refused():
    """The layer's gradients are constants to autograd: a second derivative through them is an error and
    not the part of it that other terms contribute."""
    m, h, x, weights, out = _layer(9)
    g, = torch.autograd.grad(out.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (g.sum() + x.square().sum()).backward()
    m.gmm.gmm_destroy(h)
