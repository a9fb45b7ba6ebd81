"""Host-side checks of prefill and chunk with score options (no device is touched), and the oracle
of their tests against closed forms."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import packed_oracle as PO
from oracle import serving_oracle as SO


@pytest.fixture(scope="module")
def ha():
    from long_context_sparse_score_gb300 import _build
    _build.build()
    from long_context_sparse_score_gb300 import hashattn
    return hashattn


def _calls(ha, opts, chunk=True, **kw):
    t = ha.HATokens()
    t.n_seq, t.total, t.h_q, t.h_kv, t.d = 3, 40, 8, 2, 128
    t.dtype = t.out_dtype = ha.HA_BF16
    t.q_st, t.q_sh, t.k_st, t.k_sh, t.v_st, t.v_sh = 1024, 128, 256, 128, 256, 128
    c = ha.HACache()
    c.dtype, c.n_pages, c.page_size, c.max_pages, c.table_st = ha.HA_BF16, 10, 16, 4, 4
    c.k_sp, c.k_sh, c.k_sn = 16 * 256, 128, 256
    c.v_sp, c.v_sh, c.v_sn = 16 * 256, 128, 256
    for k, v in kw.items():
        if k != "ws":
            setattr(t, k, v)
    L, o = ha.lib(), opts and ctypes.byref(opts)
    return (L.hash_attn_prefill_ex(ctypes.byref(t), o, 512, 512, 512, 512, 512, 512, 1024, kw.get("ws", 0), None),
            chunk and L.hash_attn_chunk_ex(ctypes.byref(t), ctypes.byref(c), o, 512, 512, 512, 512, 512, 512, 512, 512, 1024, kw.get("ws", 0), None))


BAD = [dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=2.0 ** -61), dict(scale=2.0 ** 61), dict(softcap=-50.0),
       dict(softcap=math.nan), dict(softcap=math.inf), dict(softcap=2.0 ** 61), dict(softcap=2.0 ** -61), dict(scale=2.0 ** 40, softcap=2.0 ** -40),
       dict(scale=2.0 ** -40, softcap=2.0 ** 40), dict(window=-1)]


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_options_outside_their_ranges(ha, bad):
    assert _calls(ha, ha.score_opts(**bad)) == (ha.HA_ERR_INVALID_ARG,) * 2
    assert "opts" in ha.last_error()


def test_refusals_as_without_options(ha):
    o = ha.score_opts(softcap=50.0, window=7)
    o.reserved = 1
    assert _calls(ha, o) == (ha.HA_ERR_INVALID_ARG,) * 2
    for o in (None, ha.score_opts(), ha.score_opts(scale=0.5, softcap=50.0, window=1 << 30, slopes=512, prefix=512, first=512)):
        assert _calls(ha, o) == (ha.HA_ERR_WORKSPACE,) * 2              # all else is right: the workspace is too small
        assert _calls(ha, o, dtype=ha.HA_F32) == (ha.HA_ERR_UNSUPPORTED,) * 2
        assert _calls(ha, o, d=96) == (ha.HA_ERR_UNSUPPORTED,) * 2
        assert _calls(ha, o, q_st=1025) == (ha.HA_ERR_INVALID_ARG,) * 2
        assert _calls(ha, o, total=0) == (ha.HA_OK,) * 2


def test_a_prompt_that_sees_itself_both_ways_counts_all_of_its_tiles(ha):
    """Twice the work of a causal one: refused from there on, not wrapped around (one without a prefix
    is not refused here, and not made: it would be launched)."""
    assert _calls(ha, ha.score_opts(prefix=512), chunk=False, n_seq=1, h_q=32, h_kv=8, ws=1 << 40, total=1 << 21)[0] == ha.HA_ERR_UNSUPPORTED
    assert "too much" in ha.last_error()


def test_binding_compares_options_with_the_tokens(ha, monkeypatch):
    monkeypatch.setattr(ha, "_device", lambda: 0)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    ints = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    q, k, v, K, V, table = bf(5, 4, 64), bf(5, 2, 64), bf(5, 2, 64), bf(3, 2, 16, 64), bf(3, 2, 16, 64), ints(2, 4)
    tok, cache = ha.make_tokens(q, k, v, 2, out_dtype=torch.bfloat16), ha.make_cache(K, V, table)
    ws = torch.zeros(64, dtype=torch.uint8)

    def both(match, **kw):
        o = ha.score_opts(**kw)
        for call in (lambda: ha.hash_attn_prefill_ex(tok, o, q, k, v, ints(3), bf(5, 4, 64), torch.zeros(5, 4), workspace=ws, stream=0),
                     lambda: ha.hash_attn_chunk_ex(tok, cache, o, q, K, V, table, ints(3), ints(2), bf(5, 4, 64), torch.zeros(5, 4), workspace=ws,
                                                   stream=0)):
            with pytest.raises(ValueError, match=match):
                call()

    both("current CUDA device", softcap=50.0)
    both("current CUDA device", slopes=torch.zeros(4), prefix=ints(2), first=ints(2))
    for bad in (torch.zeros(3), torch.zeros(4).double(), torch.zeros(8)[::2]):
        both("slopes must be contiguous", slopes=bad)
    for name in ("prefix", "first"):
        for bad in (ints(1), ints(2).long(), ints(4)[::2]):
            both(f"{name} must be contiguous int32", **{name: bad})
    o = ha.score_opts(first=ints(2))
    assert o.tensors is not None and ha.score_opts(softcap=3.0).tensors is None  # and they are kept
    with pytest.raises(ValueError, match="descriptor was made for"):
        ha.hash_attn_prefill_ex(tok, o, bf(4, 4, 64), k, v, ints(3), bf(5, 4, 64), torch.zeros(5, 4), workspace=ws, stream=0)


# ---------------------------------------------------------------- the oracle

def rows(seed, nq, nk, d):
    g = np.random.default_rng(seed)
    return g.standard_normal((nq, d)), g.standard_normal((nk, d)), g.standard_normal((nk, d))


def test_without_options_it_is_causal_attention():
    q, K, V = rows(1, 7, 30, 16)
    ref, got = PO.causal_attention(q, K, V), SO.attention(q, K, V)
    assert np.allclose(got[0], ref[0], rtol=0, atol=1e-13) and np.allclose(got[1], ref[1], rtol=0, atol=1e-13)


def test_a_window_of_one_returns_the_own_value():
    q, K, V = rows(2, 5, 9, 8)
    out, lse = SO.attention(q, K, V, window=1, cap=2.0, slope=3.0)[:2]
    z = (q * K[4:]).sum(1) / math.sqrt(8)
    assert np.allclose(out, V[4:]) and np.allclose(lse, 2 * np.tanh(z / 2))


def test_equal_scores_leave_the_bias():
    """Keys of zeros: weights e^{-slope distance}, a geometric series; both ways with a prefix."""
    _, _, V = rows(3, 1, 6, 4)
    z = np.zeros((6, 4))
    s = 0.7
    out, lse = SO.attention(z, z, V, slope=s)[:2]
    w = np.exp(-s * np.arange(6)[::-1])
    assert np.allclose(out[5], w @ V / w.sum()) and math.isclose(lse[5], math.log((1 - math.exp(-6 * s)) / (1 - math.exp(-s))))
    both = SO.attention(z, z, V, slope=s, prefix=6)[0]
    w = np.exp(-s * np.abs(np.arange(6) - 2))
    assert np.allclose(both[2], w @ V / w.sum())


def test_rows_that_see_nothing_and_first_keys():
    q, K, V = rows(4, 4, 6, 8)
    out, lse = SO.attention(q, K, V, first=4)[:2]
    assert np.all(out[:2] == 0) and np.all(np.isneginf(lse[:2]))   # positions 2 and 3
    assert np.allclose(out[2], V[4])
    again = SO.attention(q[2:], K[4:], V[4:])
    assert np.allclose(out[2:], again[0]) and np.allclose(lse[2:], again[1])
    assert np.allclose(SO.attention(q, K, V, first=4, prefix=5)[0][:3], V[4])  # the prefix shows key 4 to all
