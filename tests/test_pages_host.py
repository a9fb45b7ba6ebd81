"""Host-side checks of the page plan and of the append with several axes (no device is touched),
and the oracle of their tests against plans worked out by hand."""
import ctypes

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


def _paging(ha, **kw):
    p = ha.HAPaging()
    p.n_seq, p.total, p.n_pages, p.page_size, p.max_pages, p.table_st = 3, 40, 10, 16, 4, 4
    for k, v in kw.items():
        setattr(p, k, v)
    return p


NAMES = ["new_lens", "seq_lens", "seq_lens_out", "cu", "table", "slots", "free_pages", "n_free", "n_free_out", "dev_flags"]


def _plan(ha, p, **kw):
    a = [kw.get(n, 512) for n in NAMES]
    return ha.lib().hash_attn_plan_pages(p and ctypes.byref(p), *a, None)


BAD_PAGING = [("n_seq", 0), ("n_seq", (1 << 20) + 1), ("total", -1), ("total", (1 << 24) + 1), ("n_pages", 0), ("page_size", 0),
              ("max_pages", 0), ("max_pages", 1 << 27), ("reserved", 1), ("table_st", 3)]


@pytest.mark.parametrize("field,value", BAD_PAGING)
def test_plan_refusals(ha, field, value):
    assert _plan(ha, _paging(ha, **{field: value})) == ha.HA_ERR_INVALID_ARG
    assert ha.last_error() != ""


def test_plan_refuses_what_is_missing(ha):
    assert _plan(ha, None) == ha.HA_ERR_INVALID_ARG
    for n in NAMES:
        if n not in ("slots", "dev_flags"):
            assert _plan(ha, _paging(ha), **{n: None}) == ha.HA_ERR_INVALID_ARG, n
    assert _plan(ha, _paging(ha, n_pages=1 << 27)) == ha.HA_ERR_UNSUPPORTED  # slots past 2^31


def _axes_args(ha, **kw):
    t = ha.HATokens()
    t.n_seq, t.total, t.h_q, t.h_kv, t.d = 3, 40, 8, 2, 128
    t.dtype = t.out_dtype = ha.HA_BF16
    t.q_st, t.q_sh, t.k_st, t.k_sh, t.v_st, t.v_sh = 1024, 128, 256, 128, 256, 128
    c = ha.HACache()
    c.dtype, c.n_pages, c.page_size, c.max_pages, c.table_st = ha.HA_BF16, 10, 16, 4, 4
    c.k_sp, c.k_sh, c.k_sn = 16 * 256, 128, 256
    c.v_sp, c.v_sh, c.v_sn = 16 * 256, 128, 256
    r = ha.HARopeAxes()
    r.inv_freq, r.rot_dim, r.n_axes = 512, 64, 3
    for i in range(32):
        r.axis[i] = i % 3
    for k, v in kw.items():
        if k.startswith("axis"):
            r.axis[int(k[4:])] = v
        else:
            setattr(r, k, v)
    return t, c, r


def _append_axes(ha, t, c, r, positions=512, pos_st=40):
    return ha.lib().hash_attn_append_axes(ctypes.byref(t), ctypes.byref(c), r and ctypes.byref(r), positions, pos_st, 512, 512, 512, None,
                                          512, 512, 512, 512, 512, 512, None, None, None)


BAD_AXES = [dict(inv_freq=None), dict(rot_dim=8), dict(rot_dim=24), dict(rot_dim=144), dict(interleaved=2), dict(n_axes=0), dict(n_axes=9),
            dict(reserved=1), dict(axis0=3), dict(axis31=200), dict(n_axes=2)]


@pytest.mark.parametrize("bad", BAD_AXES, ids=str)
def test_append_axes_refusals(ha, bad):
    assert _append_axes(ha, *_axes_args(ha, **bad)) == ha.HA_ERR_INVALID_ARG
    assert ha.last_error() != ""


def test_append_axes_refuses_positions_it_cannot_read(ha):
    t, c, r = _axes_args(ha)
    assert _append_axes(ha, t, c, None) == ha.HA_ERR_INVALID_ARG
    assert _append_axes(ha, t, c, r, positions=None) == ha.HA_ERR_INVALID_ARG
    assert _append_axes(ha, t, c, r, pos_st=39) == ha.HA_ERR_INVALID_ARG
    t.total = 0  # nothing to do: what is not read may be missing
    assert _append_axes(ha, t, c, r, positions=None) == ha.HA_OK
    t.total = 40
    t.dtype = 9
    assert _append_axes(ha, t, c, r) == ha.HA_ERR_UNSUPPORTED


# ---------------------------------------------------------------- the binding

def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


REACHED = "current CUDA device"  # a host tensor that got this far is refused for its device


def test_plan_binding_compares_tensors_with_the_paging(ha, monkeypatch):
    monkeypatch.setattr(ha, "_device", lambda: 0)
    table = ints(3, 4)
    p = ha.make_paging(table, 10, 16, 40)
    assert (p.n_seq, p.max_pages, p.table_st, p.n_pages, p.page_size, p.total) == (3, 4, 4, 10, 16, 40)
    good = dict(new=ints(3), had=ints(3), out=ints(3), cu=ints(4), table=table, free=ints(10), n_free=ints(1), n_out=ints(1), slots=ints(40),
                flags=None)

    def call(**kw):
        a = {**good, **kw}
        ha.hash_attn_plan_pages(p, a["new"], a["had"], a["out"], a["cu"], a["table"], a["free"], a["n_free"], a["n_out"], slots=a["slots"],
                                dev_flags=a["flags"], stream=0)

    for kw in ({}, dict(slots=None), dict(flags=ints(1)), dict(table=ints(5, 4))):
        with pytest.raises(ValueError, match=REACHED):
            call(**kw)
    for name, n in (("new", 2), ("had", 2), ("out", 2), ("cu", 3), ("free", 9), ("n_free", 0), ("n_out", 0), ("slots", 39), ("flags", 0)):
        with pytest.raises(ValueError, match="must be contiguous int32"):
            call(**{name: ints(n)})
        with pytest.raises(ValueError, match="must be contiguous int32"):
            call(**{name: torch.zeros(64, dtype=torch.int64)})
    for bad in (ints(2, 4), ints(3, 3), ints(3, 8)[:, :4], ints(4, 3).t(), torch.zeros(3, 4, dtype=torch.int64)):
        with pytest.raises(ValueError, match="page_table"):
            call(table=bad)
    with pytest.raises(ValueError, match="page_table"):
        ha.make_paging(torch.zeros(3, 4), 10, 16, 40)


def test_axes_binding(ha, monkeypatch):
    monkeypatch.setattr(ha, "_device", lambda: 0)
    f = torch.ones(16)
    r = ha.rope_axes(f, [0, 1, 2] * 5 + [4], interleaved=True)
    assert (r.rot_dim, r.n_axes, r.interleaved, list(r.axis)[:17]) == (32, 5, 1, [0, 1, 2] * 5 + [4, 0])
    for bad in ([0] * 15, [0] * 15 + [8], [0] * 15 + [-1], []):
        with pytest.raises(ValueError, match="axis must give"):
            ha.rope_axes(f, bad)
    with pytest.raises(ValueError, match="inv_freq"):
        ha.rope_axes(f.double(), [0] * 16)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    q, k, v, K, V, table = bf(5, 4, 64), bf(5, 2, 64), bf(5, 2, 64), bf(3, 2, 16, 64), bf(3, 2, 16, 64), ints(2, 4)
    tok, cache = ha.make_tokens(q, k, v, 2), ha.make_cache(K, V, table)

    def call(pos, **kw):
        ha.hash_attn_append_axes(tok, cache, kw.get("q", q), k, v, table, ints(3), ints(2), pos, bf(5, 4, 64), K, V, rope=r, stream=0)

    for pos in (ints(5, 5), ints(6, 5), ints(5, 9)[:, :5]):
        with pytest.raises(ValueError, match=REACHED):
            call(pos)
    for pos in (ints(4, 5), ints(5, 6), ints(5, 5).t()[:, :4], torch.zeros(5, 5, dtype=torch.int64), ints(1, 5).expand(5, 5), ints(5, 5).t()):
        with pytest.raises(ValueError, match="positions must be"):
            call(pos)
    with pytest.raises(ValueError, match="descriptor was made for"):
        call(ints(5, 5), q=bf(5, 3, 64))


# ---------------------------------------------------------------- the oracle

def test_plan_by_hand():
    """Pages of 4 tokens: one sequence fills its page and begins another, one ends, one begins."""
    r = SO.plan_pages([2, -1, 5, 0], [3, 6, 0, 4], [[7, -1], [2, 5], [-1, -1], [1, -1]], [9, 8, 0, 0, 0, 0, 0, 0, 0, 0], 2, 10, 4, 8)
    # 2 and 5 come back on top of 9, 8; then 5 is taken by the first, 2 and 8 by the third
    assert r["free"][:4] == [9, 8, 2, 5] and r["n_free"] == 1
    assert r["table"] == [[7, 5], [2, 5], [2, 8], [1, -1]] and r["lens"] == [5, 0, 5, 4] and r["cu"] == [0, 2, 2, 7, 7]
    assert r["slots"] == [7 * 4 + 3, 5 * 4, 2 * 4, 9, 10, 11, 8 * 4, -1] and r["flags"] == 0


def test_plan_by_hand_short_of_pages():
    r = SO.plan_pages([1, 5, 1, 1], [4, 0, 8, 1], [[0, -1, -1], [-1] * 3, [1, 2, -1], [3, -1, -1]], [4, 5], 2, 6, 4, 8)
    assert r["lens"] == [5, -1, -9, 2]          # one page for the first; the second needs two, the third is behind it
    assert r["n_free"] == 1 and r["flags"] == SO.PAGES and r["table"][0] == [0, 5, -1] and r["table"][1] == [-1] * 3
    assert r["slots"] == [20] + [-1] * 6 + [13] and r["cu"] == [0, 1, 6, 7, 8]


def test_rotation_by_one_axis_is_the_plain_rotation():
    g = np.random.default_rng(1)
    x, w = g.standard_normal((3, 64)), 10.0 ** -np.arange(16)
    for inter in (False, True):
        a = SO.rotate_axes(x, [5, 77], [1] * 16, w, inter)
        assert np.allclose(a, PO.rotate(x, 77, w, inter), rtol=0, atol=1e-12)
