"""Calls whose thread has made no CUDA call of its own, as autograd's worker threads before a backward pass."""
import threading

import pytest

pytestmark = pytest.mark.gpu


def _mods():
    import torch
    from ragged_matmul_gb300 import binding
    from ragged_matmul_gb300 import build as gbuild
    gbuild.build()
    return torch, binding


def _in_new_thread(call):
    got = []

    def run():
        try:
            got.append(call())
        except Exception as err:
            got.append(err)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    return got[0]


@pytest.mark.parametrize("name", ["bf16", "planes", "int4", "dense_int4", "fp8", "fp8_block", "nvfp4", "mxfp4", "sort",
                                  "empty_sort", "combine", "combine_grad", "quantise", "dequantise"])
def test_first_call_of_a_thread(name):
    """Every call, as the first one of its thread, gives what it gives on this one."""
    torch, binding = _mods()
    E, N, K, R = 2, 256, 256, 40
    h = binding.gmm_create(E, 0)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    bf, i32 = torch.bfloat16, dict(dtype=torch.int32, device="cuda")
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    byte = lambda *s: torch.randint(0, 64, s, generator=gen, dtype=torch.uint8, device="cuda")  # noqa: E731
    off, ids, st = torch.tensor([0, 25, R], **i32), torch.arange(E, **i32), torch.zeros(2, **i32)
    c, a, b = torch.zeros((R, N), dtype=bf, device="cuda"), rnd(R, K).to(bf), rnd(E, N, K).to(bf)
    q = torch.randint(-2 ** 31, 2 ** 31 - 1, (E, N, K // 8), generator=gen, **i32)
    qs = rnd(E, N, K // 64).to(bf)
    one = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    slots = torch.randint(0, E, (R // 2, 2), generator=gen, **i32)
    sr = torch.randperm(R, generator=gen, device="cuda").to(torch.int32).reshape(R // 2, 2)
    tok, out, wts = rnd(R // 2, K).to(bf), torch.zeros((R // 2, K), dtype=bf, device="cuda"), rnd(R // 2, 2)
    p = binding.fp4_scale_pitch(K, "nvfp4")
    u8a, u8s = byte(R, K // 2), byte(R, p)
    offs, srs, rss = torch.zeros(E + 1, **i32), torch.zeros((R // 2, 2), **i32), torch.zeros(R, **i32)
    pt = {f: binding.fp4_scale_pitch(K, f) for f in ("nvfp4", "mxfp4")}
    base = {"nvfp4": 0, "mxfp4": 90}
    fp4 = {f: (u8a, byte(E, N, K // 2), byte(R, pt[f]) + base[f], byte(E, N, pt[f]) + base[f]) for f in pt}
    s1, s2, w1, w2 = one(R, 1), one(R, 2), one(E, 2, 1), one(E, 2, 2)
    a8, b8, s3 = byte(R, K), byte(E, N, K), torch.cat([a, a, a])

    def product(f):
        x, w, xs, ws = fp4[f]
        return binding.gmm_run_fp4(h, c, x, off, w, ids, st, xs, ws, fmt=f)
    call, result = {
        "bf16": (lambda: binding.gmm_run(h, c, a, off, b, ids, st), c),
        "planes": (lambda: binding.gmm_run_planes(h, c, s3, off, b, ids, st, (256, 0)), c),
        "int4": (lambda: binding.gmm_run_int4(h, c, a, off, q, qs, ids, st, group_size=64), c),
        "dense_int4": (lambda: binding.gmm_matmul_int4(h, c, a, q[0], qs[0], group_size=64), c),
        "fp8": (lambda: binding.gmm_run_fp8(h, c, a8, off, b8, ids, st, s1, w1), c),
        "fp8_block": (lambda: binding.gmm_run_fp8(h, c, a8, off, b8, ids, st, s2, w2, (1, 128, 128)), c),
        "nvfp4": (lambda: product("nvfp4"), c),
        "mxfp4": (lambda: product("mxfp4"), c),
        "sort": (lambda: binding.gmm_dispatch(h, offs, srs, rss, slots, rows=c, tokens=tok), c),
        "empty_sort": (lambda: binding.gmm_dispatch(h, offs, srs[:0], rss[:0], slots[:0]), offs),
        "combine": (lambda: binding.gmm_combine(h, out, a, sr, wts), out),
        "combine_grad": (lambda: binding.gmm_combine_grad(h, c, wts, tok, a, sr), c),
        "quantise": (lambda: binding.gmm_quantize_fp4(h, u8a, u8s, a), u8a),
        "dequantise": (lambda: binding.gmm_dequantize_fp4(h, c, u8a, u8s), c),
    }[name]
    assert call() == 0
    torch.cuda.synchronize()
    want = result.clone()
    result.fill_(3)
    torch.cuda.synchronize()
    assert _in_new_thread(call) == 0
    torch.cuda.synchronize()
    assert torch.equal(result.view(torch.uint8), want.view(torch.uint8))
    assert binding.gmm_query_status(h) == 0
    binding.gmm_destroy(h)
