"""Buffers whose byte offsets pass 32 bits, and calls whose blocks pass 31: a few rows are
looked at, where the low 32 bits of an offset alone would point elsewhere."""
import numpy as np
import pytest

import fp4_util as ref

pytestmark = [pytest.mark.gpu, pytest.mark.slow]


def _mods():
    import torch
    from ragged_matmul_gb300 import binding
    from ragged_matmul_gb300 import build as gbuild
    gbuild.build()
    return torch, binding


def test_quantise_past_31_bits_of_blocks():
    torch, binding = _mods()
    h = binding.gmm_create(1, 0)
    rows, K = (1 << 30) + 5, 32
    x = torch.tensor([[6.0] + [0.5 * (i % 4) for i in range(31)]], device="cuda")
    packed = torch.zeros((rows, 16), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((rows, 16), dtype=torch.uint8, device="cuda")
    binding.gmm_quantize_fp4(h, packed, scales, x.expand(rows, K))
    xd = x.double().cpu().numpy()
    want = ref.pack(ref.codes(xd, np.ones_like(xd)))
    for r in (0, 1, (1 << 28) + 3, (1 << 30) - 200, (1 << 30) - 1, 1 << 30, rows - 1):
        s = scales[r].cpu().numpy()
        a = np.abs(xd.reshape(1, 2, 16)).max(-1)
        assert np.array_equal(s[:2], ref.scale_codes(a, "nvfp4")[0]) and (s[2:] == 0).all(), r
        d = np.repeat(ref.SCALES["nvfp4"][s[:2].astype(int)], 16)[None]
        assert np.array_equal(packed[r].cpu().numpy(), ref.pack(ref.codes(xd, d))[0]), r
    assert want.shape == (1, 16)
    tail = slice(rows - 4, rows)
    y = torch.zeros((4, K), device="cuda")
    binding.gmm_dequantize_fp4(h, y, packed[tail], scales[tail])
    assert np.array_equal(y.double().cpu().numpy(), ref.values(packed[tail].cpu().numpy(), scales[tail].cpu().numpy(), "nvfp4"))
    binding.gmm_destroy(h)


def test_rows_past_32_bits():
    torch, binding = _mods()
    E, T, width = 3, 300_001, 8192
    h = binding.gmm_create(E, 0)
    i32 = dict(dtype=torch.int32, device="cuda")
    ids = torch.randint(0, E, (T, 1), **i32)
    tokens = torch.arange(T, device="cuda").remainder(251).to(torch.bfloat16)[:, None].expand(T, width).contiguous()
    off, sr, rs = torch.zeros(E + 1, **i32), torch.zeros((T, 1), **i32), torch.zeros(T, **i32)
    rows = torch.zeros((T, width), dtype=torch.bfloat16, device="cuda")
    binding.gmm_dispatch(h, off, sr, rs, ids, rows=rows, tokens=tokens)
    assert torch.equal(rows[:, 0], tokens[rs.long(), 0]) and torch.equal(rows[:, -1], tokens[rs.long(), -1])
    out = torch.zeros_like(tokens)
    binding.gmm_combine(h, out, rows, sr)
    assert torch.equal(out, tokens)
    out.zero_()
    d_w = torch.zeros((T, 1), device="cuda")
    binding.gmm_combine_grad(h, out, d_w, tokens, rows, sr)
    assert torch.equal(out, rows)
    assert torch.equal(d_w[:, 0].double(), tokens[:, 0].double() ** 2 * width)   # exact: below 2^24 times a power of two
    binding.gmm_destroy(h)


def test_product_past_32_bits():
    torch, binding = _mods()
    R, N, K = 160_003, 32768, 64
    h = binding.gmm_create(1, 0)
    rng = np.random.default_rng(2)
    b, b_s = ref.random_operand(rng, (1, N), K, "nvfp4")
    a, a_s = ref.random_operand(rng, (257,), K, "nvfp4")
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    pick = torch.arange(R, device="cuda").remainder(257)
    c = torch.zeros((R, N), dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    binding.gmm_run_fp4(h, c, dev(a)[pick], dev(np.array([0, R], np.int32)), dev(b), dev(np.array([0], np.int32)), st,
                        dev(a_s)[pick], dev(b_s))
    assert binding.gmm_query_status(h) == binding.GMM_OK
    C, S, _ = ref.product(a, a_s, [0, 257], b, b_s, [0], "nvfp4")
    for r0 in (0, 65536, 131072 - 100, 131072, R - 257):    # 2^32 bytes of C are 65536 rows, 2^32 elements 131072
        got = c[r0:r0 + 257].double().cpu().numpy()
        want, s = np.roll(C, -(r0 % 257), 0), np.roll(S, -(r0 % 257), 0)
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (K / 64 + 6) * 2.0 ** -22 * s).all(), r0
    binding.gmm_destroy(h)
