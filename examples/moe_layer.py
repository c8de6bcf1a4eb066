"""A mixture-of-experts layer on the library's calls, as a program would use them.

`serve` runs it on microscaled 4-bit weights and activations: the router's choice is
sorted by expert, the tokens are quantised while they are gathered into expert order,
two grouped products run the experts (the first with a fused silu), and the weighted
sum takes the rows back to their tokens.

`Experts` is one bf16 expert product with its gradients for the layer's input and for
the router's weights, for training (the expert weights are frozen).

    python examples/moe_layer.py        # needs the GPU and the built library
"""
from __future__ import annotations

import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from ragged_matmul_gb300 import binding as gmm  # noqa: E402


def route(x, router, top_k):
    """(int32 expert ids, fp32 weights), both [tokens, top_k], from the router matrix [width, E]."""
    top = torch.topk(x.float() @ router.float(), top_k, dim=1)
    return top.indices.to(torch.int32), torch.softmax(top.values, dim=1)


class Fp4Weights:
    """[E, N, K] weights in 4 bits: each expert quantised with a scale of its own (nvfp4)."""

    def __init__(self, h, w, fmt="nvfp4"):
        E, N, K = w.shape
        self.fmt = fmt
        self.packed = torch.empty((E, N, K // 2), dtype=torch.uint8, device=w.device)
        self.scales = torch.empty((E, N, gmm.fp4_scale_pitch(K, fmt)), dtype=torch.uint8, device=w.device)
        self.globals = None
        if fmt == "nvfp4":     # the largest magnitude becomes 6 times the largest block scale, 448
            self.globals = w.abs().amax(dim=(1, 2)).float().clamp(min=1e-20) / (6 * 448)
        for e in range(E):
            gmm.gmm_quantize_fp4(h, self.packed[e], self.scales[e], w[e], fmt=fmt,
                                 global_scale=None if self.globals is None else self.globals[e:e + 1])


def _quantise(h, x, fmt, row_slots=None, top_k=1):
    """(packed, scales, global scale) of x's rows, or of the rows that row_slots picks."""
    rows = x.shape[0] if row_slots is None else row_slots.numel()
    packed = torch.empty((rows, x.shape[1] // 2), dtype=torch.uint8, device=x.device)
    scales = torch.empty((rows, gmm.fp4_scale_pitch(x.shape[1], fmt)), dtype=torch.uint8, device=x.device)
    g = None
    if fmt == "nvfp4":
        top = x.abs().amax() if x.numel() else x.new_zeros(())     # no tokens: no largest one
        g = (top.float().clamp(min=1e-20) / (6 * 448)).reshape(1)
    gmm.gmm_quantize_fp4(h, packed, scales, x, fmt=fmt, row_slots=row_slots, top_k=top_k, global_scale=g)
    return packed, scales, g


def serve(h, x, router, up: Fp4Weights, down: Fp4Weights, top_k):
    """out [tokens, width] = sum over a token's experts of weight * down(silu(up(x)))."""
    T, width = x.shape
    E, hidden = up.packed.shape[:2]
    dev = x.device
    ids, weights = route(x, router, top_k)
    off = torch.empty(E + 1, dtype=torch.int32, device=dev)
    slot_rows = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    row_slots = torch.empty(T * top_k, dtype=torch.int32, device=dev)
    experts = torch.arange(E, dtype=torch.int32, device=dev)
    stats = torch.empty(2, dtype=torch.int32, device=dev)
    gmm.gmm_dispatch(h, off, slot_rows, row_slots, ids)
    a, a_scales, ga = _quantise(h, x, up.fmt, row_slots, top_k)
    mid = torch.zeros((T * top_k, hidden), dtype=torch.bfloat16, device=dev)
    gmm.gmm_run_fp4(h, mid, a, off, up.packed, experts, stats, a_scales, up.scales, fmt=up.fmt, a_global=ga,
                    b_global=up.globals, activation="silu")
    a, a_scales, ga = _quantise(h, mid, down.fmt)
    rows = torch.zeros((T * top_k, width), dtype=torch.bfloat16, device=dev)
    gmm.gmm_run_fp4(h, rows, a, off, down.packed, experts, stats, a_scales, down.scales, fmt=down.fmt, a_global=ga,
                    b_global=down.globals)
    out = torch.empty_like(x)
    gmm.gmm_combine(h, out, rows, slot_rows, weights)
    return out


class Experts(torch.autograd.Function):
    """out[t] = sum_j weights[t, j] * (x[t] @ w[ids[t, j]].T), with the gradients for x and weights.

    w [E, N, K] and w_t [E, K, N] (its transpose, laid out once) are bf16 and frozen; x is bf16."""

    @staticmethod
    def forward(ctx, x, weights, ids, w, w_t, h):
        T, K = x.shape
        k = ids.shape[1]
        E, N, _ = w.shape
        dev = x.device
        off = torch.empty(E + 1, dtype=torch.int32, device=dev)
        slot_rows = torch.empty((T, k), dtype=torch.int32, device=dev)
        row_slots = torch.empty(T * k, dtype=torch.int32, device=dev)
        experts = torch.arange(E, dtype=torch.int32, device=dev)
        stats = torch.empty(2, dtype=torch.int32, device=dev)
        rows = torch.empty((T * k, K), dtype=x.dtype, device=dev)
        gmm.gmm_dispatch(h, off, slot_rows, row_slots, ids, rows=rows, tokens=x)
        y = torch.empty((T * k, N), dtype=x.dtype, device=dev)
        gmm.gmm_run(h, y, rows, off, w, experts, stats)
        out = torch.empty((T, N), dtype=x.dtype, device=dev)
        gmm.gmm_combine(h, out, y, slot_rows, weights)
        ctx.save_for_backward(y, weights, off, slot_rows, experts, stats, w_t)
        ctx.h = h
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        y, weights, off, slot_rows, experts, stats, w_t = ctx.saved_tensors
        h = ctx.h
        if d_out.stride(1) != 1:     # an expanded or transposed gradient (that of out.sum(), for one)
            d_out = d_out.contiguous()
        d_y, d_weights = torch.empty_like(y), torch.empty_like(weights)
        gmm.gmm_combine_grad(h, d_y, d_weights, d_out, y, slot_rows, weights)
        d_rows = torch.empty((y.shape[0], w_t.shape[1]), dtype=y.dtype, device=y.device)
        gmm.gmm_run(h, d_rows, d_y, off, w_t, experts, stats)
        d_x = torch.empty((slot_rows.shape[0], w_t.shape[1]), dtype=y.dtype, device=y.device)
        gmm.gmm_combine(h, d_x, d_rows, slot_rows)     # the gradient of dispatch's copy
        return d_x, d_weights, None, None, None, None


def main():
    torch.manual_seed(0)
    T, width, hidden, E, top_k = 300, 512, 1024, 16, 4
    dev = "cuda"
    h = gmm.gmm_create(E, torch.cuda.current_device())
    x = torch.randn((T, width), device=dev).bfloat16()
    router = torch.randn((width, E), device=dev) * width ** -0.5
    w_up = torch.randn((E, hidden, width), device=dev) * width ** -0.5
    w_down = torch.randn((E, width, hidden), device=dev) * hidden ** -0.5
    ids, weights = route(x, router, top_k)
    want = torch.zeros((T, width), device=dev)
    for j in range(top_k):
        e = ids[:, j].long()
        mid = torch.nn.functional.silu(torch.einsum("tk,tnk->tn", x.float(), w_up[e]))
        want += weights[:, j:j + 1] * torch.einsum("tn,tkn->tk", mid, w_down[e])
    for fmt in ("nvfp4", "mxfp4"):
        out = serve(h, x, router, Fp4Weights(h, w_up, fmt), Fp4Weights(h, w_down, fmt), top_k)
        rel = float((out.float() - want).norm() / want.norm())
        print(f"serve {fmt}: relative difference from the unquantised layer {rel:.3f}")
    w = w_up.bfloat16()
    xt, wt = x.clone().requires_grad_(), weights.clone().requires_grad_()
    out = Experts.apply(xt, wt, ids, w, w.transpose(1, 2).contiguous(), h)
    out.float().square().mean().backward()
    print(f"train: |d_x| {float(xt.grad.float().norm()):.4f}, |d_weights| {float(wt.grad.norm()):.4f}")
    status = gmm.gmm_query_status(h)
    print("status:", gmm.gmm_error_string(status))
    gmm.gmm_destroy(h)
    return 0 if status == gmm.GMM_OK else 1


if __name__ == "__main__":
    sys.exit(main())
