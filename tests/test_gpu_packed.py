"""Prompts and chunks of new tokens: hash_attn_append, hash_attn_prefill and
hash_attn_chunk against the float64 oracle.

Tolerances, from the arithmetic (u = half a step: 2^-8 for bf16, 2^-24 for float32):

* out in bf16: each weight is rounded to bf16 once (u relative), so the weighted sum
  moves by at most u sum_j p_j |v_j| = u mag; the result is rounded once (u |out|).
* scores and weights in float32: a score sums d exact products (at most d steps of
  2 u zmax, if the adder truncates), its exponent is formed with one rounding of at
  most 2 u log2(e) |z - max| + u and 2^-22 for the exponential; l and O sum n terms
  (at most 2 u each). Together at most E = 2^-23 (d zmax + 4 zmax + n + 16) relative
  per weight, twice (numerator and denominator): 2 E mag.
* lse: E + 2^-22 (1 + |lse|).
"""
import math

import numpy as np
import pytest
import torch

from oracle import packed_oracle as PO

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module")
def H():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from long_context_sparse_score_gb300 import _build
    _build.build()
    from long_context_sparse_score_gb300 import hashattn
    hashattn.lib()
    return hashattn


def rand(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def cumulative(new):
    return torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")


def check_rows(got_out, got_lse, ref, bf16, what):
    out, lse, mag, zmax, n = ref
    d = out.shape[1]
    E = 2.0 ** -23 * (d * zmax + 4 * zmax + n + 16)
    tol = 2 * E[:, None] * mag + 1e-30
    if bf16:
        tol = tol + 2.0 ** -8 * mag * (1 + 2 * E[:, None]) + 2.0 ** -8 * np.abs(out) * (1 + 2.0 ** -7)
    got = got_out.double().cpu().numpy()
    err = np.abs(got - out)
    assert np.all(err <= tol), f"{what}: out off by {np.nanmax(err):.3g}, worst ratio {np.nanmax(err / tol):.3g}"
    gl = got_lse.double().cpu().numpy()
    none = np.isneginf(lse)
    assert np.array_equal(np.isneginf(gl), none), f"{what}: rows without keys"
    fin = ~none
    lt = E[fin] + 2.0 ** -22 * (1 + np.abs(lse[fin]))
    assert np.all(np.abs(gl[fin] - lse[fin]) <= lt), f"{what}: lse off by {np.abs(gl[fin] - lse[fin]).max():.3g}"


def run_chunk(H, q, K, V, table, new, lens, Hkv, out_dtype=torch.bfloat16, ws=None, cu=None, lens_t=None):
    T = q.shape[0]
    tok = H.make_tokens(q, None, None, len(new), h_kv=Hkv, out_dtype=out_dtype)
    cache = H.make_cache(K, V, table)
    if ws is None:
        ws = torch.full((H.hash_attn_packed_workspace_size(tok),), 0xFF, dtype=torch.uint8, device="cuda")
        H.hash_attn_workspace_init(ws[:256])
    out = torch.full((T, q.shape[1], q.shape[2]), NAN, dtype=out_dtype, device="cuda")
    lse = torch.full((T, q.shape[1]), NAN, device="cuda")
    cu = cumulative(new) if cu is None else cu
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda") if lens_t is None else lens_t
    H.hash_attn_chunk(tok, cache, q, K, V, table, cu, lens_t, out, lse, workspace=ws)
    return out, lse, H.hash_attn_device_status(ws)


def run_prefill(H, q, k, v, new, out_dtype=torch.bfloat16, ws=None, cu=None):
    tok = H.make_tokens(q, k, v, len(new), out_dtype=out_dtype)
    if ws is None:
        ws = torch.full((H.hash_attn_packed_workspace_size(tok),), 0xFF, dtype=torch.uint8, device="cuda")
        H.hash_attn_workspace_init(ws[:256])
    out = torch.full(tuple(q.shape), NAN, dtype=out_dtype, device="cuda")
    lse = torch.full(tuple(q.shape[:2]), NAN, device="cuda")
    H.hash_attn_prefill(tok, q, k, v, cumulative(new) if cu is None else cu, out, lse, workspace=ws)
    return out, lse, H.hash_attn_device_status(ws)


def pages(g, seqs, ps, Hkv, d, order="token", extra=2, dirty=True):
    """Random pool, a table that scatters its pages; rows behind the sequences are NaN."""
    need = [(n + ps - 1) // ps for n in seqs]
    n_pages = sum(need) + extra
    shape = (n_pages, ps, Hkv, d) if order == "token" else (n_pages, Hkv, ps, d)
    K, V = rand(g, *shape), rand(g, *shape)
    if order == "token":
        K, V = K.permute(0, 2, 1, 3), V.permute(0, 2, 1, 3)
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(seqs), max(1, max(need))), -5, dtype=torch.int32, device="cuda")  # unused entries are bad
    own = torch.zeros(n_pages, ps, dtype=torch.bool, device="cuda")
    at = 0
    for s, n in enumerate(seqs):
        table[s, :need[s]] = perm[at:at + need[s]]
        for i in range(need[s]):
            own[perm[at + i], :min(ps, n - i * ps)] = True
        at += need[s]
    if dirty:
        bad = ~own[:, None, :, None].expand(K.shape)
        K[bad] = NAN
        V[bad] = float("inf")
    return K, V, table


def check_chunk(q, K, V, table, new, lens, out, lse, Hkv, what="", heads=None):
    G = q.shape[1] // Hkv
    qh, tb = q.double().cpu().numpy(), table.cpu().numpy()
    a = 0
    for s, (nq, nk) in enumerate(zip(new, lens)):
        for g in range(Hkv):
            if heads is not None and g not in heads:
                continue
            Kh = PO.page_rows(K[:, g].double().cpu().numpy(), tb[s], nk)
            Vh = PO.page_rows(V[:, g].double().cpu().numpy(), tb[s], nk)
            for h in range(g * G, (g + 1) * G):
                ref = (*PO.causal_attention(qh[a:a + nq, h], Kh, Vh), nk)
                if nq:
                    check_rows(out[a:a + nq, h], lse[a:a + nq, h], ref, out.dtype == torch.bfloat16, f"{what} seq {s} head {h}")
        a += nq


def check_prefill(q, k, v, new, out, lse, what="", heads=None):
    Hkv = k.shape[1]
    G = q.shape[1] // Hkv
    qh, kh, vh = (x.double().cpu().numpy() for x in (q, k, v))
    a = 0
    for s, n in enumerate(new):
        for h in range(q.shape[1]) if heads is None else heads:
            if n:
                ref = (*PO.causal_attention(qh[a:a + n, h], kh[a:a + n, h // G], vh[a:a + n, h // G]), n)
                check_rows(out[a:a + n, h], lse[a:a + n, h], ref, out.dtype == torch.bfloat16, f"{what} seq {s} head {h}")
        a += n


# ---------------------------------------------------------------- prefill

PREFILL = [
    # name, lengths, Hq, Hkv, d
    ("one-token", [1], 1, 1, 128),
    ("tile-edges", [127, 128, 129, 255, 256, 257], 2, 1, 64),
    ("g4", [5, 0, 300, 64, 1], 8, 2, 128),
    ("g3-odd-tile", [200, 85, 43], 6, 2, 128),
    ("g7", [19, 150], 7, 1, 64),
    ("g16", [100, 31], 16, 1, 128),
    ("g128", [9, 2], 128, 1, 64),
    ("long", [700], 2, 2, 128),
]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", PREFILL, ids=[c[0] for c in PREFILL])
def test_prefill(H, case, out_dtype):
    _, new, Hq, Hkv, d = case
    g = torch.Generator(device="cuda").manual_seed(11)
    T = sum(new)
    q, k, v = rand(g, T, Hq, d), rand(g, T, Hkv, d), rand(g, T, Hkv, d)
    out, lse, st = run_prefill(H, q, k, v, new, out_dtype)
    assert st == (0, 0)
    check_prefill(q, k, v, new, out, lse)


def test_prefill_strided_inputs_and_rows_behind(H):
    """q, k, v as views of one fused projection; rows that no sequence owns stay as they
    were, and NaN in them or in other sequences reaches nobody."""
    g = torch.Generator(device="cuda").manual_seed(12)
    new, Hq, Hkv, d = [70, 33], 4, 2, 64
    T = sum(new) + 9
    qkv = rand(g, T, Hq + 2 * Hkv, d)
    qkv[sum(new):] = NAN
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    out, lse, st = run_prefill(H, q, k, v, new)
    assert st == (0, 0)
    check_prefill(q, k, v, new, out, lse)
    assert torch.isnan(out[sum(new):]).all() and torch.isnan(lse[sum(new):]).all()
    qkv[:70] = NAN  # the first sequence is no number: the second does not see it
    out2, lse2, _ = run_prefill(H, q, k, v, new)
    assert torch.equal(out2[70:103], out[70:103]) and torch.equal(lse2[70:103], lse[70:103])
    assert torch.isnan(out2[:70]).all()


@pytest.mark.parametrize("scale", [30.0, 1000.0])
def test_prefill_large_scores(H, scale):
    """Scores far apart: the running maximum grows again and again (O is rescaled)."""
    g = torch.Generator(device="cuda").manual_seed(13)
    T, d = 640, 128
    q, k, v = rand(g, T, 2, d), rand(g, T, 1, d), rand(g, T, 1, d)
    k = (k.float() * torch.linspace(0.01, scale, T, device="cuda")[:, None, None]).bfloat16()
    out, lse, st = run_prefill(H, q, k, v, [T], torch.float32)
    assert st == (0, 0)
    check_prefill(q, k, v, [T], out, lse)


def test_prefill_bad_bounds_are_flagged(H):
    g = torch.Generator(device="cuda").manual_seed(14)
    q, k, v = rand(g, 60, 2, 64), rand(g, 60, 1, 64), rand(g, 60, 1, 64)
    cu = torch.tensor([0, 20, 10, 61, 60, 60], dtype=torch.int32, device="cuda")  # only [0, 20) is in order
    out, lse, st = run_prefill(H, q, k, v, [20, 0, 0, 0, 0], cu=cu)
    assert st == (H.HA_ERR_DEVICE, H.HA_DEVERR_SEQLEN)
    check_prefill(q[:20], k[:20], v[:20], [20], out[:20], lse[:20])
    assert torch.isnan(out[20:]).all()


# ---------------------------------------------------------------- chunk

CHUNK = [
    # name, new, lens, Hq, Hkv, d, page, order
    ("decode-1", [1], [1], 4, 1, 128, 16, "token"),
    ("decode-ragged", [1] * 6, [1, 15, 16, 129, 400, 1000], 8, 2, 128, 16, "token"),
    ("decode-g8", [1] * 3, [700, 64, 65], 16, 2, 64, 32, "head"),
    ("decode-g1", [1, 1], [300, 40], 3, 3, 128, 48, "head"),
    ("chunk", [40, 7, 130], [300, 7, 900], 4, 2, 128, 64, "token"),
    ("chunk-80", [100, 3], [333, 500], 6, 2, 64, 80, "head"),
    ("mixed", [1, 60, 1, 0, 33], [200, 500, 3, 77, 33], 8, 1, 64, 128, "token"),
    ("rows-without-keys", [50, 4, 9], [20, 0, 9], 4, 2, 128, 16, "token"),
    ("parity-items-split", [3], [2000], 4, 1, 128, 256, "head"),
    ("two-tiles-split", [96], [1500], 4, 1, 128, 16, "head"),
    ("g128", [2, 1], [150, 70], 128, 1, 128, 16, "token"),
]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CHUNK, ids=[c[0] for c in CHUNK])
def test_chunk(H, case, out_dtype):
    """Rows of the pages behind the sequences hold NaN and infinities, unused table entries are bad."""
    _, new, lens, Hq, Hkv, d, ps, order = case
    g = torch.Generator(device="cuda").manual_seed(21)
    K, V, table = pages(g, lens, ps, Hkv, d, order)
    q = rand(g, sum(new), Hq, d)
    out, lse, st = run_chunk(H, q, K, V, table, new, lens, Hkv, out_dtype)
    assert st == (0, 0), hex(st[1])
    check_chunk(q, K, V, table, new, lens, out, lse, Hkv)
    again = run_chunk(H, q, K, V, table, new, lens, Hkv, out_dtype)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)  # the split's order is fixed


@pytest.mark.parametrize("layout", ["kv-by-token", "kv-by-page", "padded-heads", "one-head"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_chunk_pools_of_other_strides(H, layout, out_dtype):
    """K and V as views of one pool, or of rows that lie apart."""
    g = torch.Generator(device="cuda").manual_seed(27)
    new, lens, Hkv, d, ps, pages_ = [1, 70, 3], [300, 200, 77], 2, 128, 32, 24
    if layout == "kv-by-token":
        pool = rand(g, pages_, ps, 2, Hkv, d)
        K, V = pool[:, :, 0].permute(0, 2, 1, 3), pool[:, :, 1].permute(0, 2, 1, 3)
    elif layout == "kv-by-page":
        pool = rand(g, pages_, 2, Hkv, ps, d)
        K, V = pool[:, 0], pool[:, 1]
    elif layout == "padded-heads":
        K, V = rand(g, pages_, Hkv, ps, d + 8)[..., :d], rand(g, pages_, Hkv, ps + 4, d)[:, :, :ps]
    else:
        Hkv = 1
        K, V = rand(g, pages_, 2, ps, d)[:, :1], rand(g, pages_, 2, ps, d)[:, 1:]
    table = torch.randperm(pages_, generator=g, device="cuda").to(torch.int32)[:24].view(3, 8).repeat(1, 2)
    table[:, 8:] = table[:, :2].repeat(1, 4)  # pages may be read by several sequences and twice by one
    q = rand(g, sum(new), 4, d)
    out, lse, st = run_chunk(H, q, K, V, table, new, lens, Hkv, out_dtype)
    assert st == (0, 0)
    check_chunk(q, K, V, table, new, lens, out, lse, Hkv)


def test_chunk_contiguous_cache_of_any_length(H):
    """One page per sequence: the cache [batch, h_kv, n_cap, d] of the decode step, n_cap odd."""
    g = torch.Generator(device="cuda").manual_seed(22)
    B, Hq, Hkv, d, cap = 3, 8, 2, 128, 613
    K, V = rand(g, B, Hkv, cap, d), rand(g, B, Hkv, cap, d)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
    lens, new = [613, 100, 257], [2, 1, 5]
    q = rand(g, sum(new), Hq, d)
    out, lse, st = run_chunk(H, q, K, V, table, new, lens, Hkv)
    assert st == (0, 0)
    check_chunk(q, K, V, table, new, lens, out, lse, Hkv)


def test_chunk_agrees_with_dense_decode(H):
    """One new token per sequence is the decode step's dense path."""
    g = torch.Generator(device="cuda").manual_seed(23)
    B, Hq, Hkv, d, cap = 4, 16, 4, 128, 2048
    K, V, q = rand(g, B, Hkv, cap, d), rand(g, B, Hkv, cap, d), rand(g, B, Hq, d)
    lens = [2048, 1, 777, 1500]
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    shape = H.make_shape(q, K, V)
    ws = torch.empty(H.hash_attn_workspace_size(shape, cap, 0, 0), dtype=torch.uint8, device="cuda")
    H.hash_attn_workspace_init(ws)
    ro, rl = torch.empty(B, Hq, d, device="cuda"), torch.empty(B, Hq, device="cuda")
    H.hash_attn_decode(shape, q, None, None, K, V, lt, None, cap, 0, 0, ro, rl, workspace=ws)
    assert H.hash_attn_device_status(ws)[0] == 0
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
    out, lse, st = run_chunk(H, q, K, V, table, [1] * B, lens, Hkv, torch.float32)
    assert st == (0, 0)
    check_chunk(q, K, V, table, [1] * B, lens, out, lse, Hkv)
    # the decode step's own parity tolerance
    assert torch.all((out - ro).abs() <= 2e-3 * (1 + ro.abs())) and torch.all((lse - rl).abs() <= 1e-4 * (1 + rl.abs()))


def test_chunk_device_errors(H):
    """Bad lengths count as empty, bad bounds are skipped, a bad page is one of zeros."""
    g = torch.Generator(device="cuda").manual_seed(24)
    lens, Hkv, d, ps = [64, 64, 64], 1, 64, 16
    K, V, table = pages(g, lens, ps, Hkv, d)
    q = rand(g, 3, 2, d)
    bad = torch.tensor([64, 65, -1], dtype=torch.int32, device="cuda")
    out, lse, st = run_chunk(H, q, K, V, table, [1, 1, 1], lens, Hkv, lens_t=bad)
    assert st == (H.HA_ERR_DEVICE, H.HA_DEVERR_SEQLEN)
    check_chunk(q[:1], K, V, table, [1], [64], out[:1], lse[:1], Hkv)
    assert torch.all(out[1:] == 0) and torch.all(torch.isneginf(lse[1:]))
    cu = torch.tensor([0, 1, 9, 3], dtype=torch.int32, device="cuda")
    out, lse, st = run_chunk(H, q, K, V, table, [1, 1, 1], lens, Hkv, cu=cu)
    assert st == (H.HA_ERR_DEVICE, H.HA_DEVERR_SEQLEN)
    check_chunk(q[:1], K, V, table, [1], [64], out[:1], lse[:1], Hkv)
    assert torch.isnan(out[1:]).all()
    zeros = table.clone()
    zeros[1, 2] = K.shape[0]
    zeros[2, 0] = -1
    out, lse, st = run_chunk(H, q, K, V, zeros, [1, 1, 1], lens, Hkv)
    assert st == (H.HA_ERR_DEVICE, H.HA_DEVERR_INDEX)
    K2, V2 = torch.cat([K, torch.zeros_like(K[:1])]), torch.cat([V, torch.zeros_like(V[:1])])
    zeros[1, 2] = zeros[2, 0] = K.shape[0]
    check_chunk(q, K2, V2, zeros, [1, 1, 1], lens, out, lse, Hkv)


def test_workspace_serves_calls_in_turn(H):
    """One workspace, calls of several shapes back to back with nothing between them."""
    g = torch.Generator(device="cuda").manual_seed(25)
    ws = None
    runs = []
    for new, lens, Hq, Hkv, d in [([200, 3], [900, 3], 8, 2, 128), ([1, 1], [3000, 50], 8, 1, 128), ([7], [1999], 4, 4, 64)]:
        K, V, table = pages(g, lens, 32, Hkv, d)
        q = rand(g, sum(new), Hq, d)
        tok = H.make_tokens(q, None, None, len(new), h_kv=Hkv)
        size = H.hash_attn_packed_workspace_size(tok)
        if ws is None or ws.numel() < size:
            ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        runs.append((tok, H.make_cache(K, V, table), q, K, V, table, cumulative(new),
                     torch.tensor(lens, dtype=torch.int32, device="cuda"), new, lens, Hkv))
    outs = [(torch.empty(r[2].shape, device="cuda"), torch.empty(r[2].shape[:2], device="cuda")) for r in runs for _ in range(2)]
    for i, (o, l) in enumerate(outs):
        tok, cache, q, K, V, table, cu, lt = runs[i // 2][:8]
        H.hash_attn_chunk(tok, cache, q, K, V, table, cu, lt, o, l, workspace=ws)
    assert H.hash_attn_device_status(ws) == (0, 0)
    for i, (o, l) in enumerate(outs):
        _, _, q, K, V, table, _, _, new, lens, Hkv = runs[i // 2]
        check_chunk(q, K, V, table, new, lens, o, l, Hkv, f"call {i}")


def test_large_pool_offsets(H):
    """Rows more than 2^31 elements into the pool."""
    g = torch.Generator(device="cuda").manual_seed(26)
    Hkv, d, ps = 8, 128, 64
    n_pages = (1 << 31) // (Hkv * d * ps) + 40
    K = torch.zeros(n_pages, ps, Hkv, d, dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)
    V = torch.zeros_like(K)
    table = torch.tensor([[n_pages - 1, 3, n_pages - 2]], dtype=torch.int32, device="cuda")
    k, v, q = rand(g, 130, Hkv, d), rand(g, 130, Hkv, d), rand(g, 130, Hkv, d)
    tok = H.make_tokens(q, k, v, 1, out_dtype=torch.float32)
    cache = H.make_cache(K, V, table)
    cu, lt = cumulative([130]), torch.tensor([130], dtype=torch.int32, device="cuda")
    H.hash_attn_append(tok, cache, None, k, v, table, cu, lt, None, K, V)
    assert torch.equal(K[n_pages - 1].permute(1, 0, 2), k[:64]) and torch.equal(V[n_pages - 2, :, :2].permute(1, 0, 2), v[128:])
    out, lse, st = run_chunk(H, q, K, V, table, [130], [130], Hkv, torch.float32)
    assert st == (0, 0)
    check_prefill(q, k, v, [130], out, lse, heads=[0, 7])


def reference(q, keys, values, new, lens):
    """Float64 on the GPU: out, lse, and what check_rows measures errors by, over all rows."""
    T, Hq, d = q.shape
    out, mag = torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda"), torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    zmax = torch.zeros(T, Hq, dtype=torch.float64, device="cuda")
    a = 0
    for s, (nq, nk) in enumerate(zip(new, lens)):
        if nq and nk:
            K, V = keys(s).double(), values(s).double()  # [nk, Hkv, d]
            x = q[a:a + nq].double().view(nq, K.shape[1], -1, d)
            z = torch.einsum("ihgd,jhd->ihgj", x, K) / math.sqrt(d)
            sees = torch.arange(nk, device="cuda") <= nk - nq + torch.arange(nq, device="cuda")[:, None]
            z.masked_fill_(~sees[:, None, None], -math.inf)
            l = torch.logsumexp(z, -1)
            w = torch.exp(z - l.clamp(min=-1e300)[..., None])
            out[a:a + nq] = torch.einsum("ihgj,jhd->ihgd", w, V).reshape(nq, Hq, d)
            mag[a:a + nq] = torch.einsum("ihgj,jhd->ihgd", w, V.abs()).reshape(nq, Hq, d)
            lse[a:a + nq] = l.reshape(nq, Hq)
            zmax[a:a + nq] = (torch.einsum("ihgd,jhd->ihgj", x.abs(), K.abs()).amax(-1) / math.sqrt(d)).reshape(nq, Hq)
        a += nq
    flat = lambda t: t.reshape(-1, *t.shape[2:]).cpu().numpy()  # noqa: E731
    return flat(out), flat(lse), flat(mag), flat(zmax), max(lens)


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(H, seed):
    """Seeded shapes over the whole range: heads, groups, dims, lengths, pages, both output types."""
    import random
    r = random.Random(1000 + seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    Hkv, G, d = r.choice([1, 2, 3, 5, 8]), r.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 33, 64]), r.choice([64, 128])
    n = r.choice([1, 2, 5, 17, 40])
    most = r.choice([1, 4, 60, 400])
    new = [r.randint(0, most) for _ in range(n)]
    new[0] = max(1, new[0])
    out_dtype = r.choice([torch.bfloat16, torch.float32])
    q = rand(g, sum(new), Hkv * G, d)
    if seed % 3 == 0:
        k, v = rand(g, sum(new), Hkv, d), rand(g, sum(new), Hkv, d)
        out, lse, st = run_prefill(H, q, k, v, new, out_dtype)
        at = np.concatenate([[0], np.cumsum(new)])
        ref = reference(q, lambda s: k[at[s]:at[s + 1]], lambda s: v[at[s]:at[s + 1]], new, new)
    else:
        lens = [max(0, a + r.randint(-3, r.choice([5, 900, 5000]))) for a in new]
        K, V, table = pages(g, lens, ps := r.choice([16, 32, 48, 112, 256]), Hkv, d, r.choice(["token", "head"]))
        out, lse, st = run_chunk(H, q, K, V, table, new, lens, Hkv, out_dtype)

        def rows(X, s):
            j = torch.arange(lens[s], device="cuda")
            return X[table[s].long()[j // ps], :, j % ps]
        ref = reference(q, lambda s: rows(K, s), lambda s: rows(V, s), new, lens)
    assert st == (0, 0)
    check_rows(out.flatten(0, 1), lse.flatten(), ref, out_dtype == torch.bfloat16, f"seed {seed}")


@pytest.mark.parametrize("n", [33, 700, 2500])
def test_many_sequences(H, n):
    """More sequences than a warp, or than CTAs; some of them empty."""
    g = torch.Generator(device="cuda").manual_seed(28)
    rng = np.random.default_rng(n)
    Hq, Hkv, d, ps = 4, 2, 64, 16
    new = [int(x) for x in rng.choice([0, 1, 1, 1, 2], n)]
    lens = [a + int(x) for a, x in zip(new, rng.integers(0, 60, n))]
    K, V, table = pages(g, lens, ps, Hkv, d)
    q = rand(g, sum(new), Hq, d)
    out, lse, st = run_chunk(H, q, K, V, table, new, lens, Hkv)
    assert st == (0, 0)

    def rows(X, s):
        j = torch.arange(lens[s], device="cuda")
        return X[table[s].long()[j // ps], :, j % ps]
    ref = reference(q, lambda s: rows(K, s), lambda s: rows(V, s), new, lens)
    check_rows(out.flatten(0, 1), lse.flatten(), ref, True, f"{n} sequences")


def test_two_streams_with_their_own_workspaces(H):
    """Two calls at once."""
    g = torch.Generator(device="cuda").manual_seed(29)
    lens, new, Hkv, d = [3000, 2000], [1, 90], 2, 128
    K, V, table = pages(g, lens, 64, Hkv, d)
    q = rand(g, sum(new), 8, d)
    want = run_chunk(H, q, K, V, table, new, lens, Hkv)[:2]
    tok, cache = H.make_tokens(q, None, None, 2, h_kv=Hkv, out_dtype=torch.bfloat16), H.make_cache(K, V, table)
    cu, lt = cumulative(new), torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            ws = torch.zeros(H.hash_attn_packed_workspace_size(tok), dtype=torch.uint8, device="cuda")
            outs = [(torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")) for _ in range(5)]
            got.append((outs, ws))
    for i in range(5):
        for st, (outs, ws) in zip(streams, got):
            H.hash_attn_chunk(tok, cache, q, K, V, table, cu, lt, *outs[i], workspace=ws, stream=st)
    torch.cuda.synchronize()
    for outs, _ in got:
        for o, l in outs:
            assert torch.equal(o, want[0]) and torch.equal(l, want[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_a_row_tile_without_keys_beside_one_with(H, d, out_dtype):
    """The first 44 of 64 tokens see no key (a row tile is 32 of them), then a sequence of whole tiles."""
    g = torch.Generator(device="cuda").manual_seed(31)
    new, lens, Hkv = [64, 128], [20, 150], 2
    K, V, table = pages(g, lens, 16, Hkv, d)
    q = rand(g, sum(new), 4 * Hkv, d)
    out, lse, st = run_chunk(H, q, K, V, table, new, lens, Hkv, out_dtype)
    assert st == (0, 0)
    check_chunk(q, K, V, table, new, lens, out, lse, Hkv)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_output_on_any_16_bytes_keeps_its_neighbours(H, d, out_dtype):
    """`out` 16 bytes off a 32-byte boundary: the same bits, and nothing written around it."""
    g = torch.Generator(device="cuda").manual_seed(32)
    new, Hq = [300, 33, 64], 6
    q, k, v = (rand(g, sum(new), h, d) for h in (Hq, 2, 2))
    want, want_lse, _ = run_prefill(H, q, k, v, new, out_dtype)
    pad = 16 // want.element_size()
    room = torch.full((want.numel() + 2 * pad,), 7.0, dtype=out_dtype, device="cuda")
    out, lse = room[pad:-pad].view(want.shape), torch.empty_like(want_lse)
    tok = H.make_tokens(q, k, v, len(new), out_dtype=out_dtype)
    ws = torch.zeros(H.hash_attn_packed_workspace_size(tok), dtype=torch.uint8, device="cuda")
    H.hash_attn_prefill(tok, q, k, v, cumulative(new), out, lse, workspace=ws)
    assert H.hash_attn_device_status(ws) == (0, 0)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert bool((room[:pad] == 7).all()) and bool((room[-pad:] == 7).all())


def test_captured_graphs_share_a_workspace(H):
    """A prompt and a mixed batch captured into a graph each, replayed in turn with new inputs."""
    g = torch.Generator(device="cuda").manual_seed(33)
    Hkv, d, new, lens, prompts = 2, 128, [1, 80, 0, 200], [700, 80, 0, 2500], [500, 40]
    K, V, table = pages(g, lens, 32, Hkv, d)
    q, cu, lt = rand(g, sum(new), 8, d), cumulative(new), torch.tensor(lens, dtype=torch.int32, device="cuda")
    pq, pk, pv, pcu = rand(g, sum(prompts), 8, d), rand(g, sum(prompts), Hkv, d), rand(g, sum(prompts), Hkv, d), cumulative(prompts)
    t0, t1 = H.make_tokens(q, None, None, len(new), h_kv=Hkv, out_dtype=q.dtype), H.make_tokens(pq, pk, pv, 2, out_dtype=q.dtype)
    cache = H.make_cache(K, V, table)
    ws = torch.zeros(max(map(H.hash_attn_packed_workspace_size, (t0, t1))), dtype=torch.uint8, device="cuda")
    out, lse, pout, plse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"), torch.empty_like(pq), torch.empty(pq.shape[:2], device="cuda")

    def chunk():
        H.hash_attn_chunk(t0, cache, q, K, V, table, cu, lt, out, lse, workspace=ws, stream=torch.cuda.current_stream())

    def prompt():
        H.hash_attn_prefill(t1, pq, pk, pv, pcu, pout, plse, workspace=ws, stream=torch.cuda.current_stream())

    chunk(), prompt()
    torch.cuda.synchronize()
    graphs = []
    for call in (chunk, prompt):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
            call()
    for seed in (1, 2):
        q.copy_(rand(g.manual_seed(seed), *q.shape))
        pk.copy_(rand(g, *pk.shape))
        want = run_chunk(H, q, K, V, table, new, lens, Hkv)
        want_p = run_prefill(H, pq, pk, pv, prompts)
        for x in (out, lse, pout, plse):
            x.fill_(NAN)
        for _ in range(3):
            for gr in graphs:
                gr.replay()
        assert H.hash_attn_device_status(ws) == (0, 0)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(pout, want_p[0]) and torch.equal(plse, want_p[1])


@pytest.mark.parametrize("n", [8, 1100])
def test_bounds_that_go_back_and_forth(H, n):
    """Every other sequence covers all rows: more work than the call can have, and than 32 bits count."""
    g = torch.Generator(device="cuda").manual_seed(30)
    total = 65536 if n > 8 else 300
    q, k = rand(g, total, 128, 64), rand(g, total, 8, 64)
    cu = torch.tensor([0, total] * (n // 2) + [0], dtype=torch.int32, device="cuda")
    tok = H.make_tokens(q, k, k, n, out_dtype=torch.bfloat16)
    out, lse = torch.full_like(q, 7.0), torch.full((total, 128), 7.0, device="cuda")
    ws = torch.zeros(H.hash_attn_packed_workspace_size(tok), dtype=torch.uint8, device="cuda")
    H.hash_attn_prefill(tok, q, k, k, cu, out, lse, workspace=ws, stream=torch.cuda.current_stream())
    assert H.hash_attn_device_status(ws, torch.cuda.current_stream()) == (H.HA_ERR_DEVICE, H.HA_DEVERR_SEQLEN)
    assert bool((out == 7).all()) and bool((lse == 7).all())


# ---------------------------------------------------------------- append

def inv_freq(rot, base=500000.0):
    return torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], device="cuda")


def run_append(H, q, k, v, table, new, lens, q_out, K, V, rope=None, cu=None, lens_t=None, W=None, k_sig=None, flags=None):
    tok = H.make_tokens(k if q is None else q, k, v, len(new))
    H.hash_attn_append(tok, H.make_cache(K, V, table, k_sig), q, k, v, table, cumulative(new) if cu is None else cu,
                       torch.tensor(lens, dtype=torch.int32, device="cuda") if lens_t is None else lens_t, q_out, K, V,
                       rope=rope, W=W, k_sig=k_sig, dev_flags=flags)


def close_rotated(got, ref, x, dtype, what):
    """A rotated value a c - b s in float32: the angle is off by 2^-24 turns at most (2^-31
    half turns and one rounding of the product's 2^-25), cos and sin by 2 steps: at most
    2^-21 |pair|; then one rounding to dtype."""
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    tol = 2.0 ** -21 * np.abs(x) + u * np.abs(ref) * 1.01 + 1e-30
    err = np.abs(got - ref)
    assert np.all(err <= tol), f"{what}: off by {err.max():.3g}, worst ratio {(err / tol).max():.3g}"


APPEND = [
    # name, new, lens, Hq, Hkv, d, page, order, rot, interleaved, dtype, cache dtype
    ("decode", [1, 1, 1], [1, 17, 1000000], 8, 2, 128, 16, "token", 128, False, torch.bfloat16, torch.bfloat16),
    ("prompts", [40, 0, 130], [40, 9, 300], 6, 2, 64, 48, "head", 64, False, torch.bfloat16, torch.bfloat16),
    ("interleaved-f32", [33, 5], [33, 70], 4, 1, 64, 7, "token", 64, True, torch.float32, torch.float32),
    ("partial", [20], [500], 2, 2, 128, 64, "token", 32, False, torch.float32, torch.bfloat16),
    ("partial-interleaved", [20], [90], 2, 1, 128, 128, "head", 96, True, torch.bfloat16, torch.float32),
    ("smallest-rotation", [9], [9], 1, 1, 64, 5, "head", 16, False, torch.float32, torch.float32),
]


@pytest.mark.parametrize("case", APPEND, ids=[c[0] for c in APPEND])
def test_append(H, case):
    _, new, lens, Hq, Hkv, d, ps, order, rot, inter, dt, cdt = case
    g = torch.Generator(device="cuda").manual_seed(31)
    T, n = sum(new), len(new)
    q, k, v = rand(g, T, Hq, d, dtype=dt), rand(g, T, Hkv, d, dtype=dt), rand(g, T, Hkv, d, dtype=dt)
    first = [(b - a) // ps for a, b in zip(new, lens)]
    need = [(b + ps - 1) // ps for b in lens]
    n_pages = sum(b - a for a, b in zip(first, need)) + 3
    shape = (n_pages, ps, Hkv, d) if order == "token" else (n_pages, Hkv, ps, d)
    K, V = rand(g, *shape, dtype=cdt), rand(g, *shape, dtype=cdt)
    if order == "token":
        K, V = K.permute(0, 2, 1, 3), V.permute(0, 2, 1, 3)
    table = torch.full((n, max(need)), -9, dtype=torch.int32, device="cuda")
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    at = 0
    for s in range(n):
        table[s, first[s]:need[s]] = perm[at:at + need[s] - first[s]]
        at += need[s] - first[s]
    K0, V0 = K.clone(), V.clone()
    w = inv_freq(rot)
    rope = H.rope(w, inter)
    q_out = torch.full((T, Hq, d), NAN, dtype=dt, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    run_append(H, q, k, v, table, new, lens, q_out, K, V, rope, flags=flags)
    torch.cuda.synchronize()
    assert int(flags) == 0
    wh, tb = w.double().cpu().numpy(), table.cpu().numpy()
    qh, kh, vh = (x.double().cpu().numpy() for x in (q, k, v))
    touched = torch.zeros(n_pages, ps, dtype=torch.bool, device="cuda")
    t = 0
    pair = lambda x: np.sqrt(2) * np.abs(x).max()  # noqa: E731
    for s in range(n):
        for i in range(new[s]):
            pos = lens[s] - new[s] + i
            pg, row = tb[s, pos // ps], pos % ps
            touched[pg, row] = True
            close_rotated(q_out[t].double().cpu().numpy(), PO.rotate(qh[t], pos, wh, inter), pair(qh[t]), dt, f"q {s} {i}")
            close_rotated(K[pg, :, row].double().cpu().numpy(), PO.rotate(kh[t], pos, wh, inter), pair(kh[t]), cdt, f"k {s} {i}")
            assert torch.equal(V[pg, :, row], v[t].to(cdt))
            assert torch.equal(q_out[t, :, rot:], q[t, :, rot:]) and torch.equal(K[pg, :, row, rot:], k[t, :, rot:].to(cdt))
            t += 1
    keep = ~touched[:, None, :, None].expand(K.shape)
    assert torch.equal(K[keep], K0[keep]) and torch.equal(V[keep], V0[keep])
    # in place, and without queries
    q2 = q.clone()
    run_append(H, q2, k, v, table, new, lens, q2, K, V, rope)
    assert torch.equal(q2, q_out)
    K1, V1 = K0.clone(), V0.clone()
    run_append(H, None, k, v, table, new, lens, None, K1, V1, rope)
    assert torch.equal(K1, K) and torch.equal(V1, V)


@pytest.mark.parametrize("n,most", [(40, 3), (700, 2), (5000, 1)])
def test_append_to_many_sequences(H, n, most):
    """Sequences without new tokens among the others; every token at its place, nothing flagged."""
    g = torch.Generator(device="cuda").manual_seed(34)
    rng = np.random.default_rng(n)
    new = [int(x) for x in rng.integers(0, most + 1, n)]
    lens = [a + int(x) for a, x in zip(new, rng.integers(0, 70, n))]
    Hkv, d, ps = 2, 64, 16
    K, V, table = pages(g, lens, ps, Hkv, d, dirty=False)
    k, v = rand(g, sum(new), Hkv, d), rand(g, sum(new), Hkv, d)
    tok, flags = H.make_tokens(k, k, v, n), torch.zeros(1, dtype=torch.int32, device="cuda")
    before = K.clone()
    H.hash_attn_append(tok, H.make_cache(K, V, table), None, k, v, table, cumulative(new),
                       torch.tensor(lens, dtype=torch.int32, device="cuda"), None, K, V, dev_flags=flags)
    assert int(flags) == 0
    seq = torch.tensor([s for s, a in enumerate(new) for _ in range(a)], device="cuda")
    pos = torch.tensor([l - a + i for a, l in zip(new, lens) for i in range(a)], device="cuda")
    page, row = table[seq, pos // ps].long(), pos % ps
    assert torch.equal(K[page, :, row], k) and torch.equal(V[page, :, row], v)
    before[page, :, row] = k
    assert torch.equal(K, before)


def test_append_far_positions(H):
    """Every position keeps its angle to 2^-21, up to the longest cache (2^30 tokens)."""
    d, ps = 64, 1 << 10
    x = torch.zeros(1, 1, d, device="cuda")
    x[..., : d // 2] = 1.0
    K, V = torch.zeros(1, 1, ps, d, device="cuda"), torch.zeros(1, 1, ps, d, device="cuda")
    table = torch.zeros(1, 1 << 20, dtype=torch.int32, device="cuda")
    w = torch.cat([inv_freq(d)[:16], torch.tensor([1.0, 0.3333333, 3.0, 1e-9, 1e-30, 0.0, -0.7, 65504.0], device="cuda"),
                   inv_freq(d)[24:]])
    for pos in [0, 1, 12345, 1 << 20, (1 << 24) + 1, (1 << 30) - 1]:
        q_out = torch.empty(1, 1, d, device="cuda")
        run_append(H, x, x, x, table, [1], [pos + 1], q_out, K, V, H.rope(w))
        ref = PO.rotate(x[0, 0].cpu().numpy(), pos, w.double().cpu().numpy())
        # inv_freq * pos is exact in 64 bits, its cosine to 2^-52 of an angle below 2^46
        err = np.abs(q_out[0, 0].double().cpu().numpy() - ref)
        assert err.max() <= 2.0 ** -21 + 2.0 ** -24 + 2.0 ** (math.log2(65504.0 * (pos + 1)) - 53), (pos, err.max())


def test_append_codes_equal_encode_keys(H):
    """The codes written with the keys are those of hash_attn_encode_keys on the stored keys."""
    g = torch.Generator(device="cuda").manual_seed(33)
    for d, cdt in ((128, torch.bfloat16), (64, torch.float32)):
        B, Hkv, cap = 3, 2, 200
        new, lens = [150, 1, 90], [150, 40, 200]
        T = sum(new)
        k, v = rand(g, T, Hkv, d), rand(g, T, Hkv, d)
        K, V = torch.zeros(B, Hkv, cap, d, dtype=cdt, device="cuda"), torch.zeros(B, Hkv, cap, d, dtype=cdt, device="cuda")
        W = torch.randn(Hkv, 32, d, generator=g, device="cuda")
        table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
        sig = torch.full((B, Hkv, cap), 0x55, dtype=torch.int32, device="cuda")
        run_append(H, None, k, v, table, new, lens, None, K, V, H.rope(inv_freq(d)), W=W, k_sig=sig)
        ref = torch.full((B, Hkv, cap), 0x55, dtype=torch.int32, device="cuda")
        shape = H.make_shape(torch.zeros(B, Hkv, d, dtype=torch.bfloat16, device="cuda"), K, V, ref)
        for i in range(max(new)):
            pos = torch.tensor([b - a + i if i < a else -1 for a, b in zip(new, lens)], dtype=torch.int32, device="cuda")
            H.hash_attn_encode_keys(shape, K, W, pos, ref)
        assert torch.equal(sig, ref)


def test_append_device_errors_skip_and_flag(H):
    g = torch.Generator(device="cuda").manual_seed(34)
    Hkv, d, ps = 2, 64, 16
    new = [4, 3, 2, 5]
    k, v, q = rand(g, 14, Hkv, d), rand(g, 14, Hkv, d), rand(g, 14, 4, d)
    K, V = torch.zeros(6, Hkv, ps, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(6, Hkv, ps, d, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, 1], [2, 6], [3, 4], [5, 5]], dtype=torch.int32, device="cuda")
    sig = torch.zeros(6, Hkv, ps, dtype=torch.int32, device="cuda")
    W = torch.randn(Hkv, 32, d, generator=g, device="cuda")

    def call(lens, cu=None):
        K.zero_(), V.zero_(), sig.zero_()
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        q_out = torch.full((14, 4, d), NAN, dtype=torch.bfloat16, device="cuda")
        run_append(H, q, k, v, table, new, lens, q_out, K, V, None, W=W, k_sig=sig, flags=flags, cu=cu)
        return int(flags), q_out, (V != 0).any(-1).any(1), (sig != 0).any(1)

    # a page outside the pool: its keys and values are skipped, its queries are not
    fl, qo, wrote, coded = call([4, 18, 2, 5])
    assert fl == H.HA_DEVERR_INDEX and torch.equal(qo, q)
    want = torch.zeros(6, ps, dtype=torch.bool)
    want[0, :4] = want[3, :2] = want[5, :5] = True
    want[2, 15] = True
    assert torch.equal(wrote.cpu(), want) and torch.equal(coded.cpu(), want)
    # lengths outside the table, and new tokens that start before the sequence
    fl, qo, wrote, _ = call([33, 3, -1, 3])
    assert fl == H.HA_DEVERR_SEQLEN | H.HA_DEVERR_INDEX
    want.zero_()
    want[2, :3] = want[5, :3] = True
    assert torch.equal(wrote.cpu(), want)
    assert torch.isnan(qo[:4]).all() and torch.equal(qo[4:7], q[4:7]) and torch.isnan(qo[7:11]).all() and torch.equal(qo[11:], q[11:])
    # bounds that fall, and rows behind the last sequence
    fl, qo, wrote, _ = call([4, 3, 2, 5], cu=torch.tensor([0, 4, 2, 5, 9], dtype=torch.int32, device="cuda"))
    assert fl & H.HA_DEVERR_SEQLEN and torch.isnan(qo[9:]).all()


# ---------------------------------------------------------------- together

def test_prompt_then_chunks_then_decode(H):
    """As a serving loop runs them: prompts are attended over and appended with their codes,
    a second chunk follows, then single tokens by the chunk call and by the sparse decode
    step on the same cache; all captured once into a graph and replayed as well."""
    g = torch.Generator(device="cuda").manual_seed(41)
    B, Hq, Hkv, d, cap = 2, 8, 2, 128, 512
    W = torch.randn(Hkv, 32, d, generator=g, device="cuda")
    K, V = torch.zeros(B, Hkv, cap, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, Hkv, cap, d, dtype=torch.bfloat16, device="cuda")
    sig = torch.zeros(B, Hkv, cap, dtype=torch.int32, device="cuda")
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
    rope = H.rope(w := inv_freq(d))
    steps = [[200, 131], [60, 3], [1, 1]]
    data, done = [], [0, 0]
    for new in steps:
        done = [a + b for a, b in zip(done, new)]
        T = sum(new)
        q, k, v = rand(g, T, Hq, d), rand(g, T, Hkv, d), rand(g, T, Hkv, d)
        data.append((H.make_tokens(q, k, v, B, out_dtype=torch.float32), q, k, v, cumulative(new),
                     torch.tensor(done, dtype=torch.int32, device="cuda"), torch.empty_like(q),
                     torch.empty(T, Hq, d, device="cuda"), torch.empty(T, Hq, device="cuda")))
    cache = H.make_cache(K, V, table, sig)
    ws = torch.zeros(max(H.hash_attn_packed_workspace_size(x[0]) for x in data), dtype=torch.uint8, device="cuda")
    shape = H.make_shape(data[2][1], K, V, sig)
    m = 48
    wd = torch.empty(H.hash_attn_workspace_size(shape, m, 4, 8), dtype=torch.uint8, device="cuda")
    H.hash_attn_workspace_init(wd)
    q_sig = torch.empty(B, Hq, dtype=torch.int32, device="cuda")
    so, sl = torch.empty(B, Hq, d, device="cuda"), torch.empty(B, Hq, device="cuda")
    first = torch.empty_like(data[0][7]), torch.empty_like(data[0][8])

    def loop():
        for i, (tok, q, k, v, cu, lt, qr, out, lse) in enumerate(data):
            H.hash_attn_append(tok, cache, q, k, v, table, cu, lt, qr, K, V, rope=rope, W=W, k_sig=sig)
            H.hash_attn_chunk(tok, cache, qr, K, V, table, cu, lt, out, lse, workspace=ws)
        qr, lt = data[2][6], data[2][5]
        H.hash_attn_encode_queries(shape, qr, W, q_sig)
        H.hash_attn_decode(shape, qr, q_sig, sig, K, V, lt, None, m, 4, 8, so, sl, workspace=wd)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        loop()
        assert H.hash_attn_device_status(ws)[0] == 0 and H.hash_attn_device_status(wd)[0] == 0
    torch.cuda.current_stream().wait_stream(side)
    eager = [x.clone() for e in data for x in (e[7], e[8])] + [so.clone(), sl.clone(), K.clone(), sig.clone()]
    # against the oracle: the rotated queries over the cache as it stood at each step
    for (tok, q, k, v, cu, lt, qr, out, lse), new in zip(data, steps):
        check_chunk(qr, K, V, table, new, lt.tolist(), out, lse, Hkv)
    # whole prompts: prefill over the rotated rows says the same as the chunk over the cache
    kr = torch.cat([K[0, :, :200], K[1, :, :131]], 1).permute(1, 0, 2).contiguous()
    vr = torch.cat([V[0, :, :200], V[1, :, :131]], 1).permute(1, 0, 2).contiguous()
    H.hash_attn_prefill(H.make_tokens(data[0][6], kr, vr, B, out_dtype=torch.float32), data[0][6], kr, vr, data[0][4], *first,
                        workspace=ws)
    check_prefill(data[0][6], kr, vr, steps[0], *first)
    # the sparse step against the oracle's selection on these codes
    from oracle import hashattn_oracle as O
    for b, h in [(0, 0), (1, 5)]:
        n = int(data[2][5][b])
        idx, _, ro, rl = O.decode_head(data[2][6][b, h].float().cpu().numpy(), int(q_sig[b, h]) & 0xFFFFFFFF,
                                       sig[b, h // 4].cpu().numpy().astype(np.int64) & 0xFFFFFFFF, K[b, h // 4].float().cpu().numpy(),
                                       V[b, h // 4].float().cpu().numpy(), n, m, 4, 8)
        assert np.all(np.abs(so[b, h].cpu().numpy() - ro) <= 2e-3 * (1 + np.abs(ro)))
    # captured and replayed on new storage contents
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop()
    K.zero_(), sig.zero_()
    for e in data:
        e[7].fill_(NAN)
    so.fill_(NAN)
    graph.replay()
    torch.cuda.synchronize()
    assert H.hash_attn_device_status(ws)[0] == 0
    for a, b in zip(eager, [x for e in data for x in (e[7], e[8])] + [so, sl, K, sig]):
        assert torch.equal(a, b)
