"""The router's calls take no device memory of their own: no variant's stack makes the driver reserve more."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch
from ragged_matmul_gb300 import binding


def free():
    torch.cuda.synchronize()
    return torch.cuda.mem_get_info()[0]


keep = []
for E in (64, 256, 1024, 1500, 4096):
    h = binding.gmm_create(E, 0)
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        for T in (3, 2600 if E <= 256 else 5):
            x, b = torch.randn((T, E), device="cuda").to(dtype), torch.zeros(E, device="cuda")
            ids, w = torch.zeros((T, 8), dtype=torch.int32, device="cuda"), torch.zeros((T, 8), device="cuda")
            d = torch.zeros_like(x)
            keep.append((h, x, b, ids, w, d))
            before = free()
            binding.gmm_route(h, ids, w, x)
            binding.gmm_route(h, ids, w, x, bias=b)
            binding.gmm_route(h, ids, w, x, bias=b, expert_groups=4, top_groups=2, group_top=2)
            binding.gmm_route_grad(h, d, w, ids, x)
            binding.gmm_route_grad(h, d, w, ids, x, renormalise=False)
            taken = (before - free()) / 2 ** 20
            assert taken < 32, f"{E} experts, {dtype}, {T} tokens: {taken:.0f} MB"
print("fine")
"""


def test_first_calls_take_no_device_memory():
    """In a process of its own, where nothing has reserved the memory before."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]
