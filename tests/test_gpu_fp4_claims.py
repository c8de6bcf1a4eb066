"""The 4-bit product's claimed tiles: with at least 8 tiles a CTA pair the pairs draw tiles from the
handle's counter, where group sizes are very uneven from both ends of the tile order.

Tolerance: as for the product's other tests, |error| <= (K / 64 + 6) 2^-22 S before the rounding to
bf16 (2^-8 of the result), S the sum of magnitudes.
"""
import numpy as np
import pytest

import fp4_util as ref

pytestmark = pytest.mark.gpu
TOKENS, COLUMNS = 240, 256        # a tile
EVEN, UNEVEN = [900] * 8, [6000, 1, 5, 900, 0, 240, 241, 33]


def _mods():
    import torch
    from ragged_matmul_gb300 import binding
    from ragged_matmul_gb300 import build as gbuild
    gbuild.build()
    return torch, binding


def _tiles(loads, N):
    return sum(-(-x // TOKENS) for x in loads) * -(-N // COLUMNS)


def _case(torch, rng, loads, N, K, fmt):
    """Operands on the device, the result in 64 bits and its bound."""
    E, R = len(loads), sum(loads)
    a, a_s = ref.random_operand(rng, (R,), K, fmt)
    b, b_s = ref.random_operand(rng, (E, N), K, fmt)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    A, B = dev(ref.values(a, a_s, fmt)), dev(ref.values(b, b_s, fmt))
    off = np.concatenate([[0], np.cumsum(loads)])
    want = torch.cat([A[off[e]:off[e + 1]] @ B[e].t() for e in range(E)])
    S = torch.cat([A[off[e]:off[e + 1]].abs() @ B[e].abs().t() for e in range(E)])
    bound = 2.0 ** -8 * want.abs() + (K / 64 + 6) * 2.0 ** -22 * S
    return [dev(x) for x in (a, a_s, b, b_s, off.astype(np.int32))], want, bound


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("loads,N", [(EVEN, 8192), (UNEVEN, 8192), (UNEVEN, 8200)])
def test_claimed_tiles(fmt, loads, N):
    torch, binding = _mods()
    K, E, R = 64, len(loads), sum(loads)
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    assert _tiles(loads, N) >= 8 * pairs, "too few tiles to be claimed"
    blocks = [-(-x // TOKENS) for x in loads if x]
    assert (max(blocks) >= 4 * min(blocks)) == (loads is UNEVEN)      # from both ends
    if N % 256:
        assert _tiles(loads, N) % 2 == 1                              # the ends meet in the middle of a round
    (a, a_s, b, b_s, off), want, bound = _case(torch, np.random.default_rng([N, E, R]), loads, N, K, fmt)
    h = binding.gmm_create(E, 0)
    ids, stats = torch.arange(E, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    w16 = torch.randn((E, 8192, K), device="cuda").bfloat16()
    x16 = torch.randn((R, K), device="cuda").bfloat16()
    off_list = off.tolist()
    want16 = torch.cat([x16[off_list[e]:off_list[e + 1]].double() @ w16[e].double().t() for e in range(E)])
    for _ in range(3):
        c = torch.full((R, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        binding.gmm_run_fp4(h, c, a, off, b, ids, stats, a_s, b_s, fmt=fmt)
        assert binding.gmm_query_status(h) == 0 and stats[1] == E
        assert ((c.double() - want).abs() <= bound).all()
        # The counter's both halves are zero again: another product of the handle counts on it.
        y = torch.full((R, 8192), float("nan"), dtype=torch.bfloat16, device="cuda")
        binding.gmm_run(h, y, x16, off, w16, ids, stats)
        assert binding.gmm_query_status(h) == 0
        assert float((y.double() - want16).abs().max()) <= float(want16.abs().max()) * 2.0 ** -7
    binding.gmm_destroy(h)
