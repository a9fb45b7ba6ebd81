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


def test_items_of_one_key_tile_with_a_part_of_a_second_row_tile(H):  # noqa: F811
    """bf16, d 128: many prompts of 33 to 63 tokens (row tiles are 32), whose whole first row tiles leave
    through the ring right behind one another."""
    g = torch.Generator(device="cuda").manual_seed(3)
    new = [33 + (7 * i) % 31 for i in range(900)]
    Hkv, T = 8, sum(new)
    q, k, v = P.rand(g, T, 4 * Hkv, 128), P.rand(g, T, Hkv, 128), P.rand(g, T, Hkv, 128)
    at = np.concatenate([[0], np.cumsum(new)])
    ref = P.reference(q, lambda s: k[at[s]:at[s + 1]], lambda s: v[at[s]:at[s + 1]], new, new)
    for _ in range(3):
        out, lse, st = P.run_prefill(H, q, k, v, new)
        assert st == (0, 0)
        P.check_rows(out.flatten(0, 1), lse.flatten(), ref, True, "prompts")
