"""Host-side checks of the packed-token entry points (no device is touched), and the
float64 oracle of their tests against closed forms."""
import ctypes
import math

import numpy as np
import pytest

from oracle import hashattn_oracle as O
from oracle import packed_oracle as PO


@pytest.fixture(scope="module")
def ha():
    from long_context_sparse_score_gb300 import _build
    _build.build()
    from long_context_sparse_score_gb300 import hashattn
    return hashattn


def _tokens(ha, **kw):
    t = ha.HATokens()
    t.n_seq, t.total, t.h_q, t.h_kv, t.d = 3, 40, 8, 2, 128
    t.dtype = t.out_dtype = ha.HA_BF16
    t.q_st, t.q_sh, t.k_st, t.k_sh, t.v_st, t.v_sh = 1024, 128, 256, 128, 256, 128
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _cache(ha, **kw):
    c = ha.HACache()
    c.dtype, c.n_pages, c.page_size, c.max_pages, c.table_st = ha.HA_BF16, 10, 16, 4, 4
    c.k_sp, c.k_sh, c.k_sn = 16 * 256, 128, 256
    c.v_sp, c.v_sh, c.v_sn = 16 * 256, 128, 256
    c.ks_sp, c.ks_sh = 32, 16
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _prefill(ha, t, *, q=512, K=512, V=512, cu=512, out=512, lse=512, ws=1024, ws_bytes=1 << 40):
    return ha.lib().hash_attn_prefill(t and ctypes.byref(t), q, K, V, cu, out, lse, ws, ws_bytes, None)


def _chunk(ha, t, c, *, q=512, K=512, V=512, table=512, cu=512, lens=512, out=512, lse=512, ws=1024, ws_bytes=1 << 40):
    return ha.lib().hash_attn_chunk(ctypes.byref(t), c and ctypes.byref(c), q, K, V, table, cu, lens, out, lse, ws, ws_bytes, None)


def _append(ha, t, c, r=None, *, q=512, k=512, v=512, W=None, table=512, cu=512, lens=512, q_out=512, K=512, V=512, sig=None):
    return ha.lib().hash_attn_append(ctypes.byref(t), c and ctypes.byref(c), r and ctypes.byref(r), q, k, v, W, table, cu, lens,
                                     q_out, K, V, sig, None, None)


BAD_TOKENS = [("n_seq", 0, -1), ("n_seq", (1 << 20) + 1, -1), ("total", -1, -1), ("total", (1 << 24) + 1, -1), ("h_q", 7, -1),
              ("h_kv", 0, -1), ("h_q", 0, -1), ("d", 96, -2), ("d", 256, -2), ("dtype", 7, -2), ("reserved", 1, -1)]


@pytest.mark.parametrize("field,value,status", BAD_TOKENS)
def test_bad_tokens_are_refused_everywhere(ha, field, value, status):
    t, c = _tokens(ha, **{field: value}), _cache(ha)
    n = ctypes.c_size_t(0)
    assert ha.lib().hash_attn_packed_workspace_size(ctypes.byref(t), ctypes.byref(n)) == status
    assert _prefill(ha, t) == status and _chunk(ha, t, c) == status and _append(ha, t, c) == status
    assert ha.last_error() != ""


def test_prefill_and_chunk_refusals(ha):
    t, c = _tokens(ha), _cache(ha)
    for call in (lambda **kw: _prefill(ha, kw.pop("t", t), **kw), lambda **kw: _chunk(ha, kw.pop("t", t), c, **kw)):
        for name in ("q", "K", "V", "cu", "out", "lse"):
            assert call(**{name: None}) == ha.HA_ERR_INVALID_ARG, name
        for name in ("q", "K", "V", "out"):
            assert call(**{name: 520}) == ha.HA_ERR_INVALID_ARG, name              # 8 bytes off
        assert call(t=_tokens(ha, dtype=ha.HA_F32)) == ha.HA_ERR_UNSUPPORTED
        assert call(t=_tokens(ha, out_dtype=5)) == ha.HA_ERR_UNSUPPORTED
        assert call(t=_tokens(ha, h_q=258)) == ha.HA_ERR_UNSUPPORTED               # 129 heads per KV head
        assert call(t=_tokens(ha, q_st=1025)) == ha.HA_ERR_INVALID_ARG             # rows off 16 bytes
        assert call(t=_tokens(ha, q_sh=0)) == ha.HA_ERR_INVALID_ARG
        assert call(t=_tokens(ha, q_st=-1024)) == ha.HA_ERR_INVALID_ARG
        assert call(ws=None) == ha.HA_ERR_WORKSPACE
        assert call(ws=1024 + 16) == ha.HA_ERR_WORKSPACE
        assert call(ws_bytes=4096) == ha.HA_ERR_WORKSPACE
    # more tiles than the kernel counts (a prompt of 16 M tokens; 2^20 sequences of 2^30 keys)
    big = _tokens(ha, n_seq=1, total=1 << 24)
    assert _prefill(ha, big) == ha.HA_ERR_UNSUPPORTED and "too much" in ha.last_error()
    many = _cache(ha, page_size=1 << 10, max_pages=1 << 20, table_st=1 << 20)
    assert _chunk(ha, _tokens(ha, n_seq=1 << 20, total=1 << 20), many) == ha.HA_ERR_UNSUPPORTED and "too much" in ha.last_error()
    assert _prefill(ha, None) == ha.HA_ERR_INVALID_ARG
    assert _prefill(ha, _tokens(ha, k_sh=100)) == ha.HA_ERR_INVALID_ARG
    assert _prefill(ha, _tokens(ha, total=0)) == ha.HA_OK                           # nothing to do
    assert _chunk(ha, t, None) == ha.HA_ERR_INVALID_ARG
    assert _chunk(ha, t, c, table=None) == ha.HA_ERR_INVALID_ARG
    assert _chunk(ha, t, c, lens=None) == ha.HA_ERR_INVALID_ARG
    assert _chunk(ha, t, _cache(ha, page_size=24)) == ha.HA_ERR_UNSUPPORTED
    assert _chunk(ha, t, _cache(ha, dtype=ha.HA_F32)) == ha.HA_ERR_UNSUPPORTED
    for bad in (dict(n_pages=0), dict(page_size=0), dict(max_pages=0), dict(max_pages=1 << 27), dict(table_st=3),
                dict(k_sn=64), dict(v_sp=4097), dict(k_sh=0)):
        assert _chunk(ha, t, _cache(ha, **bad)) == ha.HA_ERR_INVALID_ARG, bad


def test_append_refusals(ha):
    t, c = _tokens(ha), _cache(ha)
    for name in ("k", "v", "table", "cu", "lens", "K", "V"):
        assert _append(ha, t, c, **{name: None}) == ha.HA_ERR_INVALID_ARG, name
    for name in ("q", "k", "v", "q_out", "K", "V"):
        assert _append(ha, t, c, **{name: 520}) == ha.HA_ERR_INVALID_ARG, name
    assert _append(ha, t, None) == ha.HA_ERR_INVALID_ARG
    assert _append(ha, t, c, q=None) == ha.HA_ERR_INVALID_ARG                       # q_out without q
    assert _append(ha, t, c, q_out=None) == ha.HA_ERR_INVALID_ARG
    assert _append(ha, _tokens(ha, q_st=2048), c) == ha.HA_ERR_INVALID_ARG          # in place, not contiguous
    assert _append(ha, t, c, W=512) == ha.HA_ERR_INVALID_ARG                        # codes without a pool
    assert _append(ha, t, c, sig=512) == ha.HA_ERR_INVALID_ARG
    assert _append(ha, t, _cache(ha, ks_sh=15), W=512, sig=512) == ha.HA_ERR_INVALID_ARG
    assert _append(ha, t, _cache(ha, dtype=9)) == ha.HA_ERR_UNSUPPORTED
    good = ha.HARope(512, 128, 0)
    for bad in (ha.HARope(None, 128, 0), ha.HARope(512, 0, 0), ha.HARope(512, 24, 0), ha.HARope(512, 144, 0), ha.HARope(512, 64, 2)):
        assert _append(ha, t, c, bad) == ha.HA_ERR_INVALID_ARG
    assert _append(ha, _tokens(ha, total=0), c, good) == ha.HA_OK                   # nothing to do
    assert _append(ha, _tokens(ha, k_st=255), c, good) == ha.HA_ERR_INVALID_ARG


def test_workspace_size_is_fixed_by_the_heads_not_the_context(ha):
    one = ha.hash_attn_packed_workspace_size(_tokens(ha, n_seq=1, total=1))
    big = ha.hash_attn_packed_workspace_size(_tokens(ha, total=1 << 24))
    assert one < 22 * 2 ** 20 < big < 64 * 2 ** 20 and big == ha.hash_attn_packed_workspace_size(_tokens(ha, total=100))


def test_binding_checks_shapes(ha):
    import torch
    q, k = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    t = ha.make_tokens(q, k, k, 2)
    assert (t.total, t.h_q, t.h_kv, t.d, t.q_st, t.k_sh, t.out_dtype) == (5, 4, 2, 64, 256, 64, ha.HA_F32)
    with pytest.raises(ValueError):
        ha.make_tokens(q, k, k[:4], 2)
    with pytest.raises(ValueError):
        ha.make_tokens(q, k.float(), k.float(), 2)
    with pytest.raises(ValueError):
        ha.make_tokens(q, k.transpose(1, 2).contiguous().transpose(1, 2), k, 2)      # dims not contiguous
    with pytest.raises(ValueError):
        ha.make_tokens(q, k, k, 2, out_dtype=torch.float16)
    pool, table = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 4, dtype=torch.int32)
    c = ha.make_cache(pool, pool, table)
    assert (c.n_pages, c.page_size, c.max_pages, c.table_st, c.k_sp, c.k_sh, c.k_sn) == (3, 16, 4, 4, 2048, 1024, 64)
    with pytest.raises(ValueError):
        ha.make_cache(pool, pool[:2], table)
    with pytest.raises(ValueError):
        ha.make_cache(pool, pool, table.long())


def test_binding_refuses_tensors_elsewhere(ha, monkeypatch):
    """A host tensor (or one of another device) never reaches a kernel."""
    import torch
    monkeypatch.setattr(ha, "_device", lambda: 0)
    q, k = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    pool, table = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 4, dtype=torch.int32)
    t, c, i, f = ha.make_tokens(q, k, k, 2), ha.make_cache(pool, pool, table), torch.zeros(3, dtype=torch.int32), torch.zeros(5, 4)
    out = torch.zeros(5, 4, 64)
    for call in (lambda: ha.hash_attn_append(t, c, q, k, k, table, i, i, q, pool, pool, stream=0),
                 lambda: ha.hash_attn_prefill(t, q, k, k, i, out, f, workspace=f, stream=0),
                 lambda: ha.hash_attn_chunk(t, c, q, pool, pool, table, i, i, out, f, workspace=f, stream=0)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()


def test_binding_refuses_outputs_that_do_not_fit(ha):
    """Wrong size, type or strides of what a call writes (or of its bounds) would go past the end."""
    import torch
    q, k = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    pool, table = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 4, dtype=torch.int32)
    t, c = ha.make_tokens(q, k, k, 2), ha.make_cache(pool, pool, table)
    cu, lens, out, lse = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(5, 4, 64), torch.zeros(5, 4)

    def prefill(cu=cu, out=out, lse=lse):
        ha.hash_attn_prefill(t, q, k, k, cu, out, lse, workspace=lse, stream=0)

    def chunk(cu=cu, lens=lens, out=out, lse=lse):
        ha.hash_attn_chunk(t, c, q, pool, pool, table, cu, lens, out, lse, workspace=lse, stream=0)

    def append(cu=cu, lens=lens, q_out=q, W=None):
        ha.hash_attn_append(t, c, q, k, k, table, cu, lens, q_out, pool, pool, W=W, stream=0)

    bad_out = [out[:4], out.bfloat16(), torch.zeros(5, 4, 128)[..., :64]]
    for call, bad in [(prefill, dict(out=bad_out, lse=[lse[1:], lse.half()], cu=[cu[:2], cu.long()])),
                      (chunk, dict(out=bad_out, lse=[lse[1:]], cu=[cu[:2]], lens=[lens[:1], lens.long()])),
                      (append, dict(q_out=[q[:4], q.float()], cu=[cu[:2]], lens=[lens.long()], W=[torch.zeros(2, 32, 32)]))]:
        for name, values in bad.items():
            for v in values:
                with pytest.raises(ValueError, match="must be contiguous"):
                    call(**{name: v})
    table = table[:1]  # two sequences
    for call in (chunk, append):
        with pytest.raises(ValueError, match="a row for each"):
            call()


# ---------------------------------------------------------------- the oracle

def test_oracle_rotation():
    rng = np.random.default_rng(1)
    w = 10000.0 ** (-np.arange(4) / 4)
    x, y = rng.standard_normal((2, 12)), rng.standard_normal((2, 12))
    for inter in (False, True):
        assert np.allclose(PO.rotate(x, 0, w, inter), x)
        r = PO.rotate(x, 17, w, inter)
        assert np.allclose((r[:, :8] ** 2).sum(-1), (x[:, :8] ** 2).sum(-1)) and np.array_equal(r[:, 8:], x[:, 8:])
        # products of rotated rows depend on the positions' difference alone
        dots = [(PO.rotate(x, p + 5, w, inter) * PO.rotate(y, p, w, inter)).sum() for p in (0, 3, 1000)]
        assert np.allclose(dots, dots[0])
    # a quarter turn of the first pair
    e = np.zeros(4)
    e[0] = 1.0
    assert np.allclose(PO.rotate(e, 1, [math.pi / 2, 0.0]), [0, 0, 1, 0])
    assert np.allclose(PO.rotate(e, 1, [math.pi / 2, 0.0], True), [0, 1, 0, 0])


def test_oracle_causal_attention():
    rng = np.random.default_rng(2)
    q, K, V = rng.standard_normal((5, 8)), rng.standard_normal((9, 8)), rng.standard_normal((9, 8))
    out, lse, mag, _ = PO.causal_attention(q, K, V)
    for i in range(5):
        ro, rl = O.attend(q[i], K, V, np.arange(9 - 5 + i + 1))
        assert np.allclose(out[i], ro) and np.isclose(lse[i], rl) and np.all(mag[i] >= np.abs(out[i]) - 1e-12)
    out, lse, _, _ = PO.causal_attention(q, K[:2], V[:2])
    assert np.all(out[:3] == 0) and np.all(np.isneginf(lse[:3])) and np.allclose(out[3], V[0])
