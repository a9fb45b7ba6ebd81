"""The binding of the packed-token calls takes tensors as their descriptors tell of them: what was
made for another pool, table or batch is refused before anything is enqueued (no device is touched)."""
import pytest
import torch

T, N, HQ, HKV, D, PS, PAGES = 5, 2, 4, 2, 64, 16, 3


@pytest.fixture(scope="module")
def ha():
    from long_context_sparse_score_gb300 import _build
    _build.build()
    from long_context_sparse_score_gb300 import hashattn
    return hashattn


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


class Calls:
    """The three calls with arguments that fit, one of them replaced at a time."""

    def __init__(self, ha):
        self.ha = ha
        self.q, self.k, self.v = bf(T, HQ, D), bf(T, HKV, D), bf(T, HKV, D)
        self.K, self.V, self.sig = bf(PAGES, HKV, PS, D), bf(PAGES, HKV, PS, D), ints(PAGES, HKV, PS)
        self.table, self.cu, self.lens = ints(N, 4), ints(N + 1), ints(N)
        self.out, self.lse, self.ws = torch.zeros(T, HQ, D), torch.zeros(T, HQ), torch.zeros(64, dtype=torch.uint8)
        self.W = torch.zeros(HKV, 32, D)
        self.tokens, self.cache = ha.make_tokens(self.q, self.k, self.v, N), ha.make_cache(self.K, self.V, self.table, self.sig)

    def append(self, **kw):
        a = {x: kw.get(x, getattr(self, x)) for x in ("q", "k", "v", "table", "cu", "lens", "K", "V", "W", "sig")}
        self.ha.hash_attn_append(kw.get("tokens", self.tokens), kw.get("cache", self.cache), a["q"], a["k"], a["v"], a["table"],
                                 a["cu"], a["lens"], kw.get("q_out", bf(T, HQ, D)), a["K"], a["V"], W=a["W"], k_sig=a["sig"],
                                 rope=kw.get("rope"), dev_flags=kw.get("dev_flags"), stream=0)

    def prefill(self, **kw):
        self.ha.hash_attn_prefill(self.tokens, kw.get("q", self.q), kw.get("k", self.k), kw.get("v", self.v), kw.get("cu", self.cu),
                                  kw.get("out", self.out), kw.get("lse", self.lse), workspace=self.ws, stream=0)

    def chunk(self, **kw):
        a = {x: kw.get(x, getattr(self, x)) for x in ("q", "K", "V", "table", "cu", "lens", "out", "lse")}
        self.ha.hash_attn_chunk(self.tokens, self.cache, *a.values(), workspace=self.ws, stream=0)


@pytest.fixture()
def calls(ha, monkeypatch):
    monkeypatch.setattr(ha, "_device", lambda: 0)  # a host tensor that got this far is refused for its device
    return Calls(ha)


REACHED = "current CUDA device"


def test_arguments_that_fit_reach_the_device_check(calls):
    for call in (calls.append, calls.prefill, calls.chunk):
        with pytest.raises(ValueError, match=REACHED):
            call()
    with pytest.raises(ValueError, match=REACHED):
        calls.append(W=None, sig=None)


ROWS = {
    "fewer rows": lambda h: bf(T - 1, h, D), "fewer heads": lambda h: bf(T, h - 1, D), "another type": lambda h: bf(T, h, D).half(),
    "float32": lambda h: torch.zeros(T, h, D), "another head dim": lambda h: bf(T, h, 2 * D),
    "rows apart": lambda h: bf(T, 2 * h, D)[:, :h], "heads first": lambda h: bf(h, T, D).transpose(0, 1),
}
POOLS = {
    "fewer pages": lambda: bf(PAGES - 1, HKV, PS, D), "fewer heads": lambda: bf(PAGES, HKV - 1, PS, D),
    "smaller pages": lambda: bf(PAGES, HKV, PS // 2, D), "another head dim": lambda: bf(PAGES, HKV, PS, D // 2),
    "another type": lambda: bf(PAGES, HKV, PS, D).half(), "float32": lambda: torch.zeros(PAGES, HKV, PS, D),
    "tokens before heads": lambda: bf(PAGES, PS, HKV, D).permute(0, 2, 1, 3), "flat": lambda: bf(PAGES * HKV * PS * D),
}


@pytest.mark.parametrize("name", ROWS)
def test_rows_that_differ_from_the_tokens(calls, name):
    for which, h in (("q", HQ), ("k", HKV), ("v", HKV)):
        bad = {which: ROWS[name](h)}
        for call in (calls.append, calls.prefill) + ((calls.chunk,) if which == "q" else ()):
            with pytest.raises(ValueError, match="descriptor was made for"):
                call(**bad)


@pytest.mark.parametrize("name", POOLS)
def test_pools_that_differ_from_the_cache(calls, name):
    for which in ("K", "V"):
        for call in (calls.append, calls.chunk):
            with pytest.raises(ValueError, match="descriptor was made for"):
                call(**{which: POOLS[name]()})
    with pytest.raises(ValueError, match="descriptor was made for"):  # the pool is whole, the cache was made for a larger one
        calls.append(cache=calls.ha.make_cache(bf(PAGES + 1, HKV, PS, D), bf(PAGES + 1, HKV, PS, D), calls.table, ints(PAGES + 1, HKV, PS)))


def test_pools_that_differ_from_the_heads_of_the_tokens(calls):
    tokens = calls.ha.make_tokens(bf(T, 4, D), bf(T, 4, D), bf(T, 4, D), N)
    with pytest.raises(ValueError, match="descriptor was made for"):
        calls.append(tokens=tokens, q=bf(T, 4, D), k=bf(T, 4, D), v=bf(T, 4, D), W=None, sig=None)


def test_code_pools_tables_and_bounds(calls):
    for sig in (ints(PAGES - 1, HKV, PS), ints(PAGES, HKV, PS).short(), torch.zeros(PAGES, HKV, PS), ints(PAGES, HKV, 2 * PS)[..., :PS]):
        with pytest.raises(ValueError):
            calls.append(sig=sig)
    for W in (torch.zeros(HKV, 32, D).half(), torch.zeros(HKV, 32, D - 1), ints(HKV, 32, D)):
        with pytest.raises(ValueError, match="W must be contiguous"):
            calls.append(W=W)
    for flags in (torch.zeros(1), torch.zeros(1, dtype=torch.int64), ints(0)):
        with pytest.raises(ValueError, match="dev_flags"):
            calls.append(dev_flags=flags)
    tables = [ints(N, 3), torch.zeros(N, 4), ints(N, 4).long(), ints(N, 8)[:, :4], ints(4, N).t(), ints(N, 8)[:, ::2]]
    for call in (calls.append, calls.chunk):
        for table in tables:
            with pytest.raises(ValueError, match="page_table"):
                call(table=table)
        with pytest.raises(ValueError, match="a row for each"):
            call(table=ints(N - 1, 4))
        for bad in (torch.zeros(N + 1), ints(N), ints(N + 1).long(), ints(2 * N + 2)[::2]):
            with pytest.raises(ValueError, match="cu must be"):
                call(cu=bad)
        with pytest.raises(ValueError, match="seq_lens must be"):
            call(lens=torch.zeros(N))
    for call in (calls.prefill, calls.chunk):
        for lse in (ints(T, HQ), torch.zeros(T, HQ).double(), torch.zeros(T, HQ + 1)):
            with pytest.raises(ValueError, match="lse must be"):
                call(lse=lse)
        with pytest.raises(ValueError, match="out must be"):
            call(out=torch.zeros(T, HQ, D, dtype=torch.int32))
    with pytest.raises(ValueError):
        calls.ha.make_cache(calls.K, calls.V, torch.zeros(N, 4))


def test_what_a_call_does_not_look_at_may_differ(calls, ha):
    """Wider tables of the same stride, more bounds than sequences, strides of extents of one, raw addresses."""
    wide = ints(N, 8)
    cache = ha.make_cache(calls.K, calls.V, wide[:, :4], calls.sig)
    with pytest.raises(ValueError, match=REACHED):
        calls.append(cache=cache, table=wide, cu=ints(9), lens=ints(9), dev_flags=ints(3))
    one = ha.make_tokens(bf(1, 1, D), bf(1, 1, D), bf(1, 1, D), 1)
    pool = bf(1, 1, PS, D)
    cache = ha.make_cache(pool, pool, ints(1, 1))
    apart = bf(1, 1, 9 * D)[..., :D]
    with pytest.raises(ValueError, match=REACHED):
        ha.hash_attn_append(one, cache, apart, apart, apart, ints(1, 1), ints(2), ints(1), bf(1, 1, D), bf(1, 7, PS, D)[:, :1],
                            bf(1, 7, PS, D)[:, :1], stream=0)
    with pytest.raises(ValueError, match=REACHED):
        calls.append(q=None, q_out=None, k=4096, K=4096, table=4096, cu=4096)


def test_rope_takes_contiguous_float32_on_the_calls_device(calls, ha):
    f = torch.ones(D // 2)
    for bad in (f.double(), f.bfloat16(), f.half(), f.int(), torch.ones(D)[::2]):
        with pytest.raises(ValueError, match="inv_freq"):
            ha.rope(bad)
    r = ha.rope(f)
    assert r.rot_dim == D and r.inv_freq == f.data_ptr()
    addr = 4096
    with pytest.raises(ValueError, match=REACHED):  # everything else is a raw address
        calls.append(q=addr, k=addr, v=addr, table=addr, cu=addr, lens=addr, K=addr, V=addr, W=None, sig=None, q_out=addr, rope=r)
    at = ha.rope(torch.ones(D // 2)).tensor  # the struct keeps its tensor
    assert at.numel() == D // 2


def test_a_call_without_rows_does_nothing(ha, monkeypatch):
    """total = 0: empty tensors have no address, and nothing is asked of rows that are not there."""
    import ctypes
    monkeypatch.setattr(ha, "_device", lambda: -1)  # host tensors count as here: no kernel is started
    q, k = bf(0, HQ, D), bf(0, HKV, D)
    assert q.data_ptr() == 0
    pool, table, cu, lens = bf(PAGES, HKV, PS, D), ints(N, 4), ints(N + 1), ints(N)
    room = torch.zeros(1 << 12, dtype=torch.uint8)  # too small for a call with rows
    for out_dtype in (torch.bfloat16, torch.float32):
        tokens, cache = ha.make_tokens(q, k, k, N, out_dtype=out_dtype), ha.make_cache(pool, pool, table)
        out, lse = torch.zeros(0, HQ, D, dtype=out_dtype), torch.zeros(0, HQ)
        ha.hash_attn_append(tokens, cache, q, k, k, table, cu, lens, bf(0, HQ, D), pool, pool, stream=0)
        ha.hash_attn_append(tokens, cache, None, k, k, table, cu, lens, None, pool, pool, stream=0)
        ha.hash_attn_prefill(tokens, q, k, k, cu, out, lse, workspace=room, stream=0)
        ha.hash_attn_chunk(tokens, cache, q, pool, pool, table, cu, lens, out, lse, workspace=room, stream=0)
    L, t, c = ha.lib(), ctypes.byref(tokens), ctypes.byref(cache)
    assert L.hash_attn_prefill(t, None, None, None, 512, None, None, None, 0, None) == ha.HA_OK
    assert L.hash_attn_chunk(t, c, None, 512, 512, 512, 512, 512, None, None, None, 0, None) == ha.HA_OK
    assert L.hash_attn_append(t, c, None, None, None, None, None, 512, 512, 512, None, 512, 512, None, None, None) == ha.HA_OK
    # what is not rows is looked at all the same
    assert L.hash_attn_prefill(t, None, None, None, None, None, None, None, 0, None) == ha.HA_ERR_INVALID_ARG
    assert L.hash_attn_chunk(t, c, None, None, 512, 512, 512, 512, None, None, None, 0, None) == ha.HA_ERR_INVALID_ARG
    assert L.hash_attn_append(t, c, None, None, None, None, None, None, 512, 512, None, 512, 512, None, None, None) == ha.HA_ERR_INVALID_ARG


def test_workspace_of_the_largest_total_group_and_head_dim_serves_all(ha):
    """More heads alone are not more workspace: a group of four takes twice that of one, for the same total."""
    def size(total, h_q, h_kv, d):
        t = ha.HATokens()
        t.n_seq, t.total, t.h_q, t.h_kv, t.d, t.dtype = 1, total, h_q, h_kv, d, ha.HA_BF16
        return ha.hash_attn_packed_workspace_size(t)
    assert size(100, 8, 2, 128) > size(100, 32, 32, 128)
    totals, groups = [0, 1, 2, 9, 10, 32, 33, 64, 128, 129, 5000, 1 << 24], [1, 2, 3, 4, 8, 12, 16, 64, 128]
    for d in (64, 128):
        for G in groups:
            for h_kv in (1, 8):
                sizes = [size(t, G * h_kv, h_kv, d) for t in totals]
                assert sizes == sorted(sizes) and sizes == [size(t, G, 1, d) for t in totals]
                assert all(a >= b for a, b in zip(sizes, [size(t, 1, 1, 64) for t in totals]))
        for t in totals:
            sizes = [size(t, G, 1, d) for G in groups]
            assert sizes == sorted(sizes)
