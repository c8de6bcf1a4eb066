"""Grouped products of a batch without rows: empty tensors have no address, the groups are the experts."""
import pytest

pytestmark = pytest.mark.gpu
E, N, K = 4, 256, 256


def _mods():
    import torch
    from ragged_matmul_gb300 import binding
    from ragged_matmul_gb300 import build as gbuild
    gbuild.build()
    return torch, binding


def _calls(torch, binding, h, rows=0):
    """name -> call(a_offsets, ids, stats, **kw) with `rows` rows."""
    z = lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    c, a, b = z(rows, N, dtype=bf), z(rows, K, dtype=bf), z(E, N, K, dtype=bf)
    q, s4 = z(E, N, K // 8, dtype=torch.int32), z(E, N, K // 64, dtype=bf)
    f32 = lambda *s: z(*s, dtype=torch.float32)  # noqa: E731
    calls = {
        "bf16": lambda o, i, st, **kw: binding.gmm_run_ex(h, c, a, o, b, i, st, **kw),
        "planes": lambda o, i, st, **kw: binding.gmm_run_planes(h, c, z(3 * rows, K, dtype=bf), o, b, i, st, (256, 0), **kw),
        "int4": lambda o, i, st, **kw: binding.gmm_run_int4_ex(h, c, a, o, q, s4, i, st, group_size=64, **kw),
        "fp8": lambda o, i, st, **kw: binding.gmm_run_fp8(h, c, z(rows, K), o, z(E, N, K), i, st, f32(rows, 1),
                                                          f32(E, 2, 1), **kw),
        "fp8_block": lambda o, i, st, **kw: binding.gmm_run_fp8(h, c, z(rows, K), o, z(E, N, K), i, st, f32(rows, 2),
                                                                f32(E, 2, 2), (1, 128, 128), **kw),
    }
    for fmt in ("nvfp4", "mxfp4"):
        p = binding.fp4_scale_pitch(K, fmt)
        calls[fmt] = lambda o, i, st, fmt=fmt, p=p, **kw: binding.gmm_run_fp4(
            h, c, z(rows, K // 2), o, z(E, N, K // 2), i, st, z(rows, p), z(E, N, p), fmt=fmt, **kw)
    return calls


@pytest.mark.parametrize("name", ["bf16", "planes", "int4", "fp8", "fp8_block", "nvfp4", "mxfp4"])
def test_no_rows(name):
    torch, binding = _mods()
    h = binding.gmm_create(E, 0)
    call = _calls(torch, binding, h)[name]
    i32 = dict(dtype=torch.int32, device="cuda")
    for ids, active, status in (([0, 1, 2, 3], 4, 0), ([0, -1, 3, -1], 2, 0), ([0, 4, 1, 2], 3, binding.GMM_ERR_BAD_INPUT)):
        for epi in ({}, dict(activation="relu", row_scale=torch.zeros(0, device="cuda"))):
            stats = torch.full((4,), -7, **i32)
            call(torch.zeros(E + 1, **i32), torch.tensor(ids, **i32), stats, **epi)
            assert binding.gmm_query_status(h) == status
            assert stats.tolist() == [-7, active, -7, -7]
    stats = torch.full((2,), -7, **i32)     # no groups either
    call(torch.zeros(1, **i32), torch.zeros(0, **i32), stats)
    assert binding.gmm_query_status(h) == 0 and stats[1] == 0
    binding.gmm_destroy(h)


def test_no_rows_takes_no_offsets():
    """Tensors without rows are neither read nor written, whatever the offsets claim."""
    torch, binding = _mods()
    h = binding.gmm_create(E, 0)
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, stats = torch.arange(E, **i32), torch.zeros(2, **i32)
    for name, call in _calls(torch, binding, h).items():
        call(torch.tensor([0, 5, 9, 200, 300], **i32), ids, stats)
        assert binding.gmm_query_status(h) == 0 and stats[1] == E, name
    binding.gmm_destroy(h)


def test_one_missing_pointer_is_an_error():
    torch, binding = _mods()
    lib, h = binding.load_library(), binding.gmm_create(E, 0)
    t = torch.zeros(1 << 16, dtype=torch.int32, device="cuda")
    p, stream = t.data_ptr(), binding.stream_handle(0)
    bad = binding.GMM_ERR_INVALID_ARG
    for c, a in ((None, p), (p, None)):
        assert lib.gmm_run(h.ptr, c, a, p, p, p, p, 1, 64, 64, stream) == bad
        assert lib.gmm_run_int4(h.ptr, c, a, p, p, p, p, p, 1, 64, 64, 64, stream) == bad
        assert lib.gmm_run_fp4(h.ptr, c, a, p, p, p, p, 1, 64, 64, p, p, 0, None, None, None, stream) == bad
        assert lib.gmm_matmul_int4(h.ptr, c, a, p, p, 4, 64, 64, 64, None, stream) == bad
    assert lib.gmm_run(h.ptr, None, None, None, p, p, p, 1, 64, 64, stream) == bad       # offsets all the same
    assert lib.gmm_run_fp4(h.ptr, p, p, p, p, p, p, 1, 64, 64, None, p, 0, None, None, None, stream) == bad
    assert lib.gmm_matmul_int4(h.ptr, None, None, p, p, 4, 64, 64, 64, None, stream) == bad   # its rows are M
    assert binding.gmm_query_status(h) == 0
    binding.gmm_destroy(h)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_chain_without_tokens(fmt):
    """Dispatch, quantise, product, combine and its gradient on no tokens."""
    torch, binding = _mods()
    h = binding.gmm_create(E, 0)
    k, i32 = 2, dict(dtype=torch.int32, device="cuda")
    z = lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    p = binding.fp4_scale_pitch(K, fmt)
    x, off, sr, rs = z(0, K, dtype=torch.bfloat16), torch.full((E + 1,), 9, **i32), torch.zeros((0, k), **i32), torch.zeros(0, **i32)
    binding.gmm_dispatch(h, off, sr, rs, sr)
    a, a_s, stats, rows = z(0, K // 2), z(0, p), torch.zeros(2, **i32), z(0, N, dtype=torch.bfloat16)
    binding.gmm_quantize_fp4(h, a, a_s, x, fmt=fmt, row_slots=rs, top_k=k)
    binding.gmm_dequantize_fp4(h, x, a, a_s, fmt=fmt)
    binding.gmm_run_fp4(h, rows, a, off, z(E, N, K // 2), torch.arange(E, **i32), stats, a_s, z(E, N, p), fmt=fmt)
    out, d_w = z(0, N, dtype=torch.bfloat16), torch.zeros((0, k), device="cuda")
    binding.gmm_combine(h, out, rows, sr, d_w)
    binding.gmm_combine_grad(h, rows, d_w, out, rows, sr, d_w)
    assert binding.gmm_query_status(h) == 0 and (off == 0).all() and stats[1] == E
    binding.gmm_destroy(h)


def test_one_of_two_empty_tensors_has_an_address():
    torch, binding = _mods()
    h = binding.gmm_create(E, 0)
    i32 = dict(dtype=torch.int32, device="cuda")
    base = torch.zeros((8, K), dtype=torch.bfloat16, device="cuda")
    fresh, view = torch.zeros((0, K), dtype=torch.bfloat16, device="cuda"), base[:0]
    w, ids = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda"), torch.arange(E, **i32)
    assert N == K
    for c, a in ((fresh, view), (view, fresh), (view, view)):
        stats = torch.zeros(2, **i32)
        binding.gmm_run(h, c, a, torch.zeros(E + 1, **i32), w, ids, stats)
        assert binding.gmm_query_status(h) == 0 and stats[1] == E
    binding.gmm_destroy(h)
