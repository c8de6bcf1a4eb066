"""Sorting, summing and the gradient at the ends of their ranges."""
import pytest

pytestmark = pytest.mark.gpu


def _mods():
    import torch
    from ragged_matmul_gb300 import binding
    from ragged_matmul_gb300 import build as gbuild
    gbuild.build()
    return torch, binding


@pytest.mark.parametrize("E", [1, 1024, 1025, 4096])
@pytest.mark.parametrize("copy", [False, True])
def test_sort_no_tokens_writes_the_offsets(E, copy):
    """For every number of experts, with and without tokens to copy, by itself and in a graph."""
    torch, binding = _mods()
    h = binding.gmm_create(E, 0)
    off = torch.full((E + 3,), -7, dtype=torch.int32, device="cuda")
    empty = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    kw = dict(rows=empty(0, 16, dtype=torch.bfloat16), tokens=empty(0, 16, dtype=torch.bfloat16)) if copy else {}
    args = (h, off, empty(0, 3), empty(0), empty(0, 3))
    binding.gmm_dispatch(*args, **kw)
    assert binding.gmm_query_status(h) == binding.GMM_OK
    assert (off[: E + 1] == 0).all() and (off[E + 1:] == -7).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.gmm_dispatch(*args, **kw)
    off.fill_(-7)
    graph.replay()
    torch.cuda.synchronize()
    assert (off[: E + 1] == 0).all() and (off[E + 1:] == -7).all()
    binding.gmm_destroy(h)


@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_rows_wider_than_the_column_count_are_refused(dtype):
    """Widths whose column numbers would pass 31 bits are refused before any launch."""
    torch, binding = _mods()
    lib, h = binding.load_library(), binding.gmm_create(2, 0)
    buf = torch.full((64,), 7, dtype=torch.int32, device="cuda")
    p, stream = buf.data_ptr(), binding.stream_handle(0)
    for width in ((1 << 31) - 4095, (1 << 31) - 1):
        assert lib.gmm_dispatch(h.ptr, p, p, p, p, p, p, 0, 1, 1, width, dtype, stream) == binding.GMM_ERR_UNSUPPORTED
        assert lib.gmm_combine(h.ptr, p, width, p, 1, p, None, 1, 1, width, dtype, stream) == binding.GMM_ERR_UNSUPPORTED
        assert lib.gmm_combine_grad(h.ptr, p, p, p, 0, p, 1, p, None, 1, 1, width, dtype, stream) \
            == binding.GMM_ERR_UNSUPPORTED
    assert binding.gmm_query_status(h) == binding.GMM_OK and (buf == 7).all()
    binding.gmm_destroy(h)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,k,E,width", [(3, 4, 2, 24), (40, 6, 3, 33), (1500, 4, 2, 40)])
def test_gradient_through_the_maps_of_repeated_experts(dtype, T, k, E, width):
    """Tokens that name an expert several times: the sort's rows are distinct, as the gradient requires,
    and dispatch, combine and their gradients are those of the layer sum_j w_j x_t.  Whole numbers: exact."""
    torch, binding = _mods()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T + width)
    dt, h = getattr(torch, dtype), binding.gmm_create(E, 0)
    i32 = dict(dtype=torch.int32, device="cuda")
    ids = torch.randint(0, E, (T, k), generator=gen, **i32)
    ids[T // 2] = 0
    ids[::7, 1] = -1
    x = torch.randint(-4, 5, (T, width), generator=gen, device="cuda").to(dt)
    g = torch.randint(-4, 5, (T, width), generator=gen, device="cuda").to(dt)
    w = torch.randint(1, 4, (T, k), generator=gen, device="cuda").float()
    off, sr, rs = torch.empty(E + 1, **i32), torch.empty((T, k), **i32), torch.empty(T * k, **i32)
    rows = torch.zeros((T * k, width), dtype=dt, device="cuda")
    binding.gmm_dispatch(h, off, sr, rs, ids, rows=rows, tokens=x)
    named = sr[sr >= 0]
    assert named.unique().numel() == named.numel() == int((ids >= 0).sum())
    d_rows, d_w, d_x = torch.zeros_like(rows), torch.full_like(w, 9.0), torch.empty_like(x)
    binding.gmm_combine_grad(h, d_rows, d_w, g, rows, sr, w)
    binding.gmm_combine(h, d_x, d_rows, sr)
    live = (ids >= 0).double()
    assert torch.equal(d_w.double(), live * (g.double() * x.double()).sum(1, keepdim=True))
    assert torch.equal(d_x.double(), (live * w.double()).sum(1, keepdim=True) * g.double())
    assert binding.gmm_query_status(h) == binding.GMM_OK
    binding.gmm_destroy(h)
