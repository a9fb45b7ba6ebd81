"""Capped scores of long sequences, in items of two row tiles and of one, against the float64 oracle. (Prompts of 8,192
tokens or more have a kernel of their own for bf16 results of head dim 128.)"""
import numpy as np
import pytest
import torch

import test_gpu_score_opts as S
from oracle import serving_oracle as SO
from test_gpu_score_opts import H  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

OPTIONS = {"cap": dict(cap=50.0), "cap-window": dict(cap=50.0, window=600), "cap-prefix": dict(cap=30.0, prefix=[700], first=[130])}


@pytest.mark.parametrize("large", [False, True], ids=["ordinary", "some-large"])
@pytest.mark.parametrize("G", [1, 3, 8])
@pytest.mark.parametrize("name", OPTIONS)
def test_prompt(H, name, G, large):  # noqa: F811
    """`large`: some keys' scores lie beyond half of the cap, so parts of a tile leave its short path."""
    g = torch.Generator(device="cuda").manual_seed(81)
    n, d = 2100, 128
    q, k, v = S.rand(g, n, G, d, scale=3.0), S.rand(g, n, 1, d), S.rand(g, n, 1, d)
    if large:
        k[torch.randperm(n, generator=g, device="cuda")[:60]] *= 6
    o = S.Opts(**OPTIONS[name])
    out, lse = S.prefill(H, q, k, v, [n], o)
    S.check_prefill(q, k, v, [n], o, out, lse, heads=[G - 1])
    again = S.prefill(H, q, k, v, [n], o)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("large", [False, True], ids=["ordinary", "some-large"])
@pytest.mark.parametrize("cap,window", [(50.0, 0), (50.0, 500), (20.0, 0)])
def test_chunk_over_a_wide_table(H, cap, window, large, order):  # noqa: F811
    """Chunks of many tokens and of one, long and short contexts, in a table with room for 4,096 keys a sequence."""
    g = torch.Generator(device="cuda").manual_seed(82)
    new, lens, Hq, Hkv, d, ps = [300, 1, 70, 1, 5], [1500, 2500, 400, 90, 1300], 8, 2, 128, 64
    o = S.Opts(cap=cap, window=window)
    K, V, table = S.pages(g, new, lens, ps, Hkv, d, order, o)
    if large:
        K[torch.rand(K.shape[:3], generator=g, device="cuda") < 0.03] *= 6
    wide = torch.full((len(new), 64), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = S.rand(g, sum(new), Hq, d, scale=3.0)
    out, lse = S.chunk(H, q, K, V, wide, new, lens, Hkv, o)
    S.check_chunk(q, K, V, wide, new, lens, o, out, lse, heads=[0, 7])


LONG = {"cap": dict(cap=50.0), "cap-window": dict(cap=50.0, window=3000), "cap-first": dict(cap=30.0, first=[1000, 5])}


@pytest.mark.parametrize("large", [False, True], ids=["ordinary", "some-large"])
@pytest.mark.parametrize("G", [1, 3, 8])
@pytest.mark.parametrize("name", LONG)
def test_long_prompts(H, name, G, large):  # noqa: F811
    """Two prompts of 8,192 tokens on average; rows at the ends of tiles and anywhere."""
    g = torch.Generator(device="cuda").manual_seed(83)
    new, d = [8300, 8090], 128
    q, k, v = S.rand(g, sum(new), G, d, scale=3.0), S.rand(g, sum(new), 1, d), S.rand(g, sum(new), 1, d)
    if large:
        k[torch.randperm(sum(new), generator=g, device="cuda")[:300]] *= 6
    o = S.Opts(**LONG[name])
    out, lse = S.prefill(H, q, k, v, new, o)
    a = 0
    for s, n in enumerate(new):
        kh, vh = (x[a:a + n, 0].double().cpu().numpy() for x in (k, v))
        opts = o.of(s, 0)
        for i in {0, 1, 127, 128, 129, 255, 256, 1000, 4000, 4095, 4096, n - 1, *np.random.default_rng(s).integers(0, n, 30).tolist()}:
            ref = SO.attention(q[a + i:a + i + 1, G - 1].double().cpu().numpy(), kh[:i + 1], vh[:i + 1], **opts)
            S.check_rows(out[a + i:a + i + 1, G - 1], lse[a + i:a + i + 1, G - 1], ref, f"seq {s} row {i}")
        a += n
    again = S.prefill(H, q, k, v, new, o)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
