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
