"""Packed attention and append where a wait, a bound or a rounding is at its edge
(tolerances as in test_gpu_packed unless a test derives its own)."""
import numpy as np
import pytest
import torch

import test_gpu_packed as P
from test_gpu_packed import H  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hkv", [1, 3])
@pytest.mark.parametrize("n", [129, 300, 640, 1500])
def test_float32_one_head_per_kv_head_d64(H, n, Hkv):  # noqa: F811
    """A row tile is 128 tokens, two key tiles of 64: row tile 1 has two key tiles more, and goes on
    for two products when row tile 0 has ended."""
    g = torch.Generator(device="cuda").manual_seed(n + Hkv)
    new = [n, 128, 256, 64]
    T = sum(new)
    q, k, v = (P.rand(g, T, Hkv, 64) for _ in range(3))
    out, lse, st = P.run_prefill(H, q, k, v, new, torch.float32)
    assert st == (0, 0)
    P.check_prefill(q, k, v, new, out, lse)
    lens = [n + 700, 128, 256 + 64, 64 + 1]
    K, V, table = P.pages(g, lens, 48, Hkv, 64)
    for _ in range(3):
        out, lse, st = P.run_chunk(H, q, K, V, table, new, lens, Hkv, torch.float32)
        assert st == (0, 0)
    P.check_chunk(q, K, V, table, new, lens, out, lse, Hkv)
