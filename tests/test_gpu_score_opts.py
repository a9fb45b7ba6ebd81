"""hash_attn_prefill_ex and hash_attn_chunk_ex (capped, biased and masked scores) against the float64
oracle.

Tolerances: the float32 part comes from the oracle (oracle/serving_oracle.py, attention). A bf16 result
adds the rounding of each weight (2^-8 of sum_j p_j |v_j|) and its own (2^-8 of the value)."""
import random

import numpy as np
import pytest
import torch

from oracle import packed_oracle as PO
from oracle import serving_oracle as SO

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


def rand(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def sums(new):
    return ints(np.concatenate([[0], np.cumsum(new)]).tolist())


def check_rows(out, lse, ref, what):
    want, wl, tol, tol_lse, mag = ref
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (mag + tol) + 2.0 ** -8 * (np.abs(want) + tol + 2.0 ** -8 * mag)
    got = out.double().cpu().numpy()
    err = np.abs(got - want)
    assert np.all(err <= tol + 1e-30), f"{what}: out off by {np.nanmax(err):.3g}, worst ratio {np.nanmax(err / (tol + 1e-30)):.3g}"
    gl, none = lse.double().cpu().numpy(), np.isneginf(wl)
    assert np.array_equal(np.isneginf(gl), none), f"{what}: rows without keys"
    off = np.abs(gl[~none] - wl[~none])
    assert np.all(off <= tol_lse[~none]), f"{what}: lse off by {off.max():.3g} of {tol_lse[~none].min():.3g}"


class Opts:
    """Options on the host, a list of first and prefix for the sequences, slopes for the heads."""

    def __init__(self, cap=0.0, window=0, slopes=None, prefix=None, first=None, scale=None):
        self.cap, self.window, self.slopes, self.prefix, self.first, self.scale = cap, window, slopes, prefix, first, scale

    def made(self, H):
        f = None if self.slopes is None else torch.tensor(self.slopes, dtype=torch.float32, device="cuda")
        return H.score_opts(scale=self.scale or 0.0, softcap=self.cap, window=self.window, slopes=f,
                            prefix=None if self.prefix is None else ints(self.prefix), first=None if self.first is None else ints(self.first))

    def of(self, s, h):
        return dict(scale=self.scale, cap=self.cap, window=self.window, slope=0.0 if self.slopes is None else float(np.float32(self.slopes[h])),
                    prefix=0 if self.prefix is None else self.prefix[s], first=0 if self.first is None else self.first[s])


def workspace(H, tok):
    ws = torch.full((H.hash_attn_packed_workspace_size(tok),), 0xFF, dtype=torch.uint8, device="cuda")
    H.hash_attn_workspace_init(ws[:256])
    return ws


def prefill(H, q, k, v, new, opts, out_dtype=torch.bfloat16, ws=None):
    tok = H.make_tokens(q, k, v, len(new), out_dtype=out_dtype)
    ws = workspace(H, tok) if ws is None else ws
    out, lse = torch.full(tuple(q.shape), NAN, dtype=out_dtype, device="cuda"), torch.full(tuple(q.shape[:2]), NAN, device="cuda")
    H.hash_attn_prefill_ex(tok, opts if opts is None or not isinstance(opts, Opts) else opts.made(H), q, k, v, sums(new), out, lse, workspace=ws)
    assert H.hash_attn_device_status(ws) == (0, 0)
    return out, lse


def chunk(H, q, K, V, table, new, lens, Hkv, opts, out_dtype=torch.bfloat16, status=(0, 0), ws=None):
    tok, cache = H.make_tokens(q, None, None, len(new), h_kv=Hkv, out_dtype=out_dtype), H.make_cache(K, V, table)
    ws = workspace(H, tok) if ws is None else ws
    out, lse = torch.full(tuple(q.shape), NAN, dtype=out_dtype, device="cuda"), torch.full(tuple(q.shape[:2]), NAN, device="cuda")
    H.hash_attn_chunk_ex(tok, cache, opts if opts is None or not isinstance(opts, Opts) else opts.made(H), q, K, V, table, sums(new), ints(lens),
                         out, lse, workspace=ws)
    assert H.hash_attn_device_status(ws) == status
    return out, lse


def seen_keys(opts, s, nq, nk):
    """The keys that a token of the sequence sees, as a set of flags."""
    o, seen = opts.of(s, 0), np.zeros(nk, dtype=bool)
    for pos in range(nk - nq, nk):
        seen[max(0, o["first"], pos - o["window"] + 1 if o["window"] else 0):max(0, min(nk, max(pos + 1, o["prefix"])))] = True
    return seen


def pages(g, new, lens, ps, Hkv, d, order, opts):
    """Random pool and a table that scatters its pages. What no token sees holds NaN and infinities; entries of pages
    without a key that is seen are bad."""
    need = [-(-n // ps) for n in lens]
    n_pages = sum(need) + 2
    shape = (n_pages, ps, Hkv, d) if order == "token" else (n_pages, Hkv, ps, d)
    K, V = rand(g, *shape), rand(g, *shape)
    if order == "token":
        K, V = K.permute(0, 2, 1, 3), V.permute(0, 2, 1, 3)
    perm = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), max(1, max(need))), -5, dtype=torch.int32, device="cuda")
    own, at = torch.zeros(n_pages, ps, dtype=torch.bool, device="cuda"), 0
    for s, n in enumerate(lens):
        seen = torch.zeros(need[s] * ps, dtype=torch.bool)
        seen[:n] = torch.from_numpy(seen_keys(opts, s, new[s], n))
        for i in range(need[s]):
            mine = seen[i * ps:(i + 1) * ps]
            if mine.any():
                table[s, i] = perm[at + i]
                own[perm[at + i]] = mine.cuda()
        at += need[s]
    bad = ~own[:, None, :, None].expand(K.shape)
    K[bad] = NAN
    V[bad] = float("inf")
    return K, V, table


def check_prefill(q, k, v, new, opts, out, lse, what="", heads=None):
    G, a = q.shape[1] // k.shape[1], 0
    qh, kh, vh = (x.double().cpu().numpy() for x in (q, k, v))
    for s, n in enumerate(new):
        for h in range(q.shape[1]) if heads is None else heads:
            if n:
                ref = SO.attention(qh[a:a + n, h], kh[a:a + n, h // G], vh[a:a + n, h // G], **opts.of(s, h))
                check_rows(out[a:a + n, h], lse[a:a + n, h], ref, f"{what} seq {s} head {h}")
        a += n


def check_chunk(q, K, V, table, new, lens, opts, out, lse, what="", heads=None):
    Hkv = K.shape[1]
    G, a = q.shape[1] // Hkv, 0
    qh, tb = q.double().cpu().numpy(), table.cpu().numpy().clip(0, K.shape[0] - 1)  # a bad entry's keys are not seen
    for s, (nq, nk) in enumerate(zip(new, lens)):
        for h in range(q.shape[1]) if heads is None else heads:
            if nq:
                Kh = PO.page_rows(K[:, h // G].double().cpu().numpy(), tb[s], nk)
                Vh = PO.page_rows(V[:, h // G].double().cpu().numpy(), tb[s], nk)
                ref = SO.attention(qh[a:a + nq, h], Kh, Vh, **opts.of(s, h))
                check_rows(out[a:a + nq, h], lse[a:a + nq, h], ref, f"{what} seq {s} head {h}")
        a += nq


def alibi(n):
    return [2.0 ** (-8.0 * (h + 1) / n) for h in range(n)]


# ---------------------------------------------------------------- prompts

OPTIONS = {
    # cap, window, bias, prefix and first as shares of the length
    "none": {}, "cap-50": dict(cap=50.0), "cap-30": dict(cap=30.0), "cap-2": dict(cap=2.0), "cap-1000": dict(cap=1000.0), "bias": dict(bias=1),
    "bias-cap": dict(bias=1, cap=20.0), "bias-against": dict(bias=-1, cap=10.0), "window-1": dict(window=1), "window-70": dict(window=70),
    "window-128": dict(window=128, cap=50.0), "prefix": dict(prefix=0.4), "both-ways": dict(prefix=1.0, cap=50.0),
    "both-ways-bias": dict(prefix=1.0, bias=1), "prefix-window": dict(prefix=0.5, window=33, bias=1), "first": dict(first=0.3),
    "first-window": dict(first=0.2, window=100, cap=30.0), "first-prefix": dict(first=0.5, prefix=0.7, bias=1), "first-all": dict(first=1.0),
    "scale": dict(scale=0.37), "scale-cap-bias": dict(scale=0.5, cap=5.0, bias=1),
}


def options(name, lens, Hq):
    o = dict(OPTIONS[name])
    share = lambda x: None if x is None else [round(x * n) for n in lens]  # noqa: E731
    b = o.pop("bias", 0)
    return Opts(prefix=share(o.pop("prefix", None)), first=share(o.pop("first", None)), slopes=[b * x for x in alibi(Hq)] if b else None, **o)


PREFILL = [
    ("tile-edges", [127, 1, 129, 0, 257], 2, 1, 64),
    ("g3", [200, 43], 6, 2, 128),
    ("g16", [100, 31], 16, 1, 128),
    ("long", [700], 2, 2, 128),
    ("long-64", [650], 1, 1, 64),
]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", OPTIONS)
@pytest.mark.parametrize("case", PREFILL, ids=[c[0] for c in PREFILL])
def test_prefill(H, case, name, out_dtype):
    _, new, Hq, Hkv, d = case
    g = torch.Generator(device="cuda").manual_seed(31)
    T = sum(new)
    q, k, v = rand(g, T, Hq, d, scale=3.0), rand(g, T, Hkv, d), rand(g, T, Hkv, d)
    opts = options(name, new, Hq)
    out, lse = prefill(H, q, k, v, new, opts, out_dtype)
    check_prefill(q, k, v, new, opts, out, lse, heads=sorted({0, Hq // 2, Hq - 1}))
    again = prefill(H, q, k, v, new, opts, out_dtype)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_options_that_change_nothing(H, d, out_dtype):
    """No options, a window over all keys, a first and a prefix of 0: the bits of hash_attn_prefill."""
    g = torch.Generator(device="cuda").manual_seed(32)
    new, Hq, Hkv = [300, 64, 0, 5], 4, 2
    T = sum(new)
    q, k, v = rand(g, T, Hq, d), rand(g, T, Hkv, d), rand(g, T, Hkv, d)
    want = prefill(H, q, k, v, new, None, out_dtype)
    tok = H.make_tokens(q, k, v, len(new), out_dtype=out_dtype)
    ws, out, lse = workspace(H, tok), torch.full_like(want[0], NAN), torch.full_like(want[1], NAN)
    H.hash_attn_prefill(tok, q, k, v, sums(new), out, lse, workspace=ws)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for o in (Opts(), Opts(window=T), Opts(window=(1 << 31) - 1, first=[-7, 0, 0, 0], prefix=[0, -1, 0, 1])):
        got = prefill(H, q, k, v, new, o, out_dtype)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cap", [1.0, 30.0, 50.0, 200.0])
@pytest.mark.parametrize("sign", [1, -1, 0])
def test_scores_far_beyond_the_cap(H, cap, sign, out_dtype):
    """All scores in the hundreds, of one sign (so every weight is e^cap, or e^-cap, or nearly) or of either, and infinite products."""
    g = torch.Generator(device="cuda").manual_seed(33)
    n, d = 300, 128
    q, k, v = rand(g, n, 2, d), rand(g, n, 1, d), rand(g, n, 1, d)
    if sign:
        q, k = q.abs(), k.abs() * sign
    k = k * 100
    q[7] = 3.0e38  # products of infinity and its like
    k[3] = sign * 3.0e38 if sign else k[3]
    opts = Opts(cap=cap)
    out, lse = prefill(H, q, k, v, [n], opts, out_dtype)
    rows = [i for i in range(n) if i != 7]
    qh, kh, vh = (x.double().cpu().numpy() for x in (q, k, v))
    for h in range(2):
        ref = SO.attention(qh[:, h], kh[:, 0], vh[:, 0], cap=cap)
        # the scores' own error does not matter where the cap is flat; it is bounded by the cap's range
        E = 2.0 ** -20 * cap + 2.0 ** -23 * (n + 16) + 2.0 ** -19
        if sign:
            check_rows(out[rows, h], lse[rows, h], (ref[0][rows], ref[1][rows], 2 * E * ref[4][rows], np.full(len(rows), E + 2.0 ** -22 * (1 + 3 * cap)),
                                                    ref[4][rows]), f"head {h}")
        else:
            keep = [i for i in rows]
            check_rows(out[keep, h], lse[keep, h], tuple(x[keep] for x in ref), f"head {h}")
    if sign:  # row 7's products are infinite
        assert torch.isfinite(out[7]).all() and torch.isfinite(lse[7]).all()


def test_bias_that_leaves_only_far_keys(H):
    """A first key behind the row's position, seen through the prefix: all weights are far away, none is lost."""
    g = torch.Generator(device="cuda").manual_seed(34)
    n, d = 900, 64
    q, k, v = rand(g, n, 2, d), rand(g, n, 1, d), rand(g, n, 1, d)
    opts = Opts(slopes=[2.0, 0.5], first=[800], prefix=[850], cap=30.0)
    for dt in (torch.bfloat16, torch.float32):
        out, lse = prefill(H, q, k, v, [n], opts, dt)
        check_prefill(q, k, v, [n], opts, out, lse)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [16, 32, 48, 64, 96])
def test_a_reference_that_moves_within_a_tile(H, at, d, out_dtype):
    """Scores 0 to the first 16 (32, 64) keys, then about 2^39.8 times their weight at key at - 1 and 2^40.6
    times at key `at`, with values of 1 and -1: the reference moves between the two, and the first one's
    weight keeps its precision."""
    g = torch.Generator(device="cuda").manual_seed(at)
    n, Hq = 160, 4
    q, k = torch.zeros(n, Hq, d, device="cuda"), torch.zeros(n, 1, d, device="cuda")
    q[..., 0], q[..., 1] = 1.0, torch.rand(n, Hq, generator=g, device="cuda")
    k[at - 1, 0, :2], k[at, 0, :2] = torch.tensor([27.5, 0.1]), torch.tensor([28.0, 0.2])
    q, k, v = q.bfloat16(), k.bfloat16(), rand(g, n, 1, d)
    v[at - 1], v[at] = 1.0, -1.0
    opts = Opts(scale=1.0, slopes=[0.0] * Hq)
    out, lse = prefill(H, q, k, v, [n], opts, out_dtype)
    check_prefill(q, k, v, [n], opts, out, lse, f"at {at}")


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cap", [30.0, 50.0])
def test_weights_over_the_whole_range_of_the_cap(H, cap, out_dtype):
    """The first keys' scores saturate at -cap, the last ones' at +cap (or the other way round), with large values: from
    the smallest weights to the largest, none is lost and no sum overflows."""
    g = torch.Generator(device="cuda").manual_seed(35)
    n, d = 400, 128
    q, v = rand(g, n, 1, d).abs() + 1, rand(g, n, 1, d, scale=2.0 ** 17)
    k = torch.full((n, 1, d), 500.0, device="cuda").bfloat16()
    k[:200] = -500.0
    for keys in (k, k.flip(0)):
        out, lse = prefill(H, q, keys, v, [n], Opts(cap=cap), out_dtype)
        qh, kh, vh = (x.double().cpu().numpy()[:, 0] for x in (q, keys, v))
        ref = SO.attention(qh, kh, vh, cap=cap)
        E = 2.0 ** -20 * cap + 2.0 ** -23 * (n + 16) + 2.0 ** -19  # (the cap is flat: the scores' own error does not matter)
        check_rows(out[:, 0], lse[:, 0], (ref[0], ref[1], 2 * E * ref[4], np.full(n, E + 2.0 ** -22 * (1 + 3 * cap)), ref[4]), f"cap {cap}")


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cap,scale", [(1e-3, None), (1e6, None), (2.0 ** 60, None), (2.0 ** -30, 2.0 ** -40), (2.0 ** 40, 2.0 ** -20), (3.0, 2.0 ** -30), (60.0, 1.0)])
def test_caps_and_scales_of_any_size(H, cap, scale, out_dtype):
    g = torch.Generator(device="cuda").manual_seed(36)
    n, d = 200, 64
    q, k, v = rand(g, n, 2, d), rand(g, n, 1, d), rand(g, n, 1, d)
    opts = Opts(cap=cap, scale=scale)
    out, lse = prefill(H, q, k, v, [n], opts, out_dtype)
    qh, kh, vh = (x.double().cpu().numpy() for x in (q, k, v))
    for h in range(2):
        ref = SO.attention(qh[:, h], kh[:, 0], vh[:, 0], **opts.of(0, h))
        if cap > 1e5:  # a score's share of the cap's error goes by the score, not by the cap: 2^-20 of its magnitude
            plain = SO.attention(qh[:, h], kh[:, 0], vh[:, 0], scale=scale)
            z = (np.abs(qh[:, h]) @ np.abs(kh[:, 0]).T).max(1) * (scale or d ** -0.5)
            tol = plain[2] + 2.0 ** -19 * z[:, None] * plain[4]
            ref = (ref[0], ref[1], tol, plain[3] + 2.0 ** -20 * z, ref[4])
        check_rows(out[:, h], lse[:, h], ref, f"cap {cap} head {h}")


# ---------------------------------------------------------------- chunks

CHUNK = [
    ("decode", [1] * 6, [1, 15, 16, 129, 400, 1000], 8, 2, 128, 16, "token"),
    ("decode-64", [1] * 3, [700, 64, 65], 16, 2, 64, 32, "head"),
    ("chunk", [40, 7, 130], [300, 7, 900], 4, 2, 128, 64, "token"),
    ("chunk-48", [100, 3], [333, 500], 6, 2, 64, 48, "head"),
    ("mixed", [1, 60, 1, 0, 33], [200, 500, 3, 77, 33], 8, 1, 64, 128, "token"),
    ("rows-without-keys", [50, 4, 9], [20, 0, 9], 4, 2, 128, 16, "token"),
    ("split", [3], [2000], 4, 1, 128, 256, "head"),
    ("g128", [2, 1], [150, 70], 128, 1, 128, 16, "token"),
]
SOME = ["none", "cap-50", "cap-2", "bias-cap", "window-70", "window-128", "prefix", "both-ways-bias", "prefix-window", "first", "first-window",
        "first-prefix", "first-all"]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", SOME)
@pytest.mark.parametrize("case", CHUNK, ids=[c[0] for c in CHUNK])
def test_chunk(H, case, name, out_dtype):
    """What no token sees (before a window or the first key, behind the end) holds NaN and infinities; table entries
    of pages that hold nothing else are bad."""
    _, new, lens, Hq, Hkv, d, ps, order = case
    g = torch.Generator(device="cuda").manual_seed(41)
    opts = options(name, lens, Hq)
    K, V, table = pages(g, new, lens, ps, Hkv, d, order, opts)
    q = rand(g, sum(new), Hq, d, scale=3.0)
    out, lse = chunk(H, q, K, V, table, new, lens, Hkv, opts, out_dtype)
    check_chunk(q, K, V, table, new, lens, opts, out, lse, heads=sorted({0, Hq // 2, Hq - 1}))
    again = chunk(H, q, K, V, table, new, lens, Hkv, opts, out_dtype)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_chunk_options_that_change_nothing(H):
    g = torch.Generator(device="cuda").manual_seed(42)
    new, lens, Hkv = [1, 70, 3], [900, 200, 77], 2
    K, V, table = pages(g, new, lens, 16, Hkv, 128, "token", Opts())
    q = rand(g, sum(new), 8, 128)
    for dt in (torch.bfloat16, torch.float32):
        want = chunk(H, q, K, V, table, new, lens, Hkv, None, dt)
        for o in (Opts(), Opts(window=901), Opts(first=[0, -3, 0], prefix=[0, 0, 1])):
            got = chunk(H, q, K, V, table, new, lens, Hkv, o, dt)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_bad_pages_that_are_seen_are_flagged(H):
    """A bad entry of a page that a window reaches counts as zeros and is flagged; one before it is neither."""
    g = torch.Generator(device="cuda").manual_seed(43)
    opts = Opts(window=40, cap=50.0)
    K, V, table = pages(g, [1], [100], 16, 1, 64, "token", opts)  # keys 60 to 99: pages 3 to 6
    q = rand(g, 1, 2, 64)
    assert (table[0, :3] == -5).all() and (table[0, 3:] >= 0).all()
    chunk(H, q, K, V, table, [1], [100], 1, opts)
    for entry in (-1, K.shape[0], 1 << 30):
        t = table.clone()
        t[0, 4] = entry
        out, lse = chunk(H, q, K, V, t, [1], [100], 1, opts, status=(H.HA_ERR_DEVICE, H.HA_DEVERR_INDEX))
        K2, V2 = torch.cat([K, torch.zeros_like(K[:1])]), torch.cat([V, torch.zeros_like(V[:1])])
        t[0, 4] = K.shape[0]
        check_chunk(q, K2, V2, t, [1], [100], opts, out, lse)


def test_device_errors(H):
    """Bad and stopped lengths count as empty of keys, bad bounds are skipped, whatever the options say."""
    g = torch.Generator(device="cuda").manual_seed(49)
    lens, d = [64, 64, 64], 64
    K, V, table = pages(g, [1, 1, 1], lens, 16, 1, d, "token", Opts())
    q = rand(g, 3, 2, d)
    for o in (Opts(window=5, prefix=[64, 64, 64]), Opts(cap=50.0, first=[3, 60, 70]), Opts(cap=50.0, slopes=[0.1, 0.2], prefix=[9, 9, 9])):
        out, lse = chunk(H, q, K, V, table, [1, 1, 1], [64, 65, -65], 1, o, status=(H.HA_ERR_DEVICE, H.HA_DEVERR_SEQLEN))
        check_chunk(q[:1], K, V, table, [1], [64], o, out[:1], lse[:1])
        assert torch.all(out[1:] == 0) and torch.all(torch.isneginf(lse[1:]))
        tok, cache = H.make_tokens(q, None, None, 3, h_kv=1, out_dtype=torch.bfloat16), H.make_cache(K, V, table)
        ws, out, lse = workspace(H, tok), torch.full_like(q, NAN), torch.full((3, 2), NAN, device="cuda")
        H.hash_attn_chunk_ex(tok, cache, o.made(H), q, K, V, table, ints([0, 1, 9, 3]), ints(lens), out, lse, workspace=ws)
        assert H.hash_attn_device_status(ws) == (H.HA_ERR_DEVICE, H.HA_DEVERR_SEQLEN)
        check_chunk(q[:1], K, V, table, [1], [64], o, out[:1], lse[:1])
        assert torch.isnan(out[1:]).all()


def test_documents_of_one_sequence(H):
    """Three documents in one sequence's pages, new tokens of the last two: sequences that share a row of the table."""
    g = torch.Generator(device="cuda").manual_seed(44)
    docs, Hq, Hkv, d, ps = [100, 90, 77], 4, 2, 128, 16
    n = sum(docs)
    k, v = rand(g, n, Hkv, d), rand(g, n, Hkv, d)
    q = rand(g, docs[1] + docs[2], Hq, d)
    pool = torch.zeros(20, ps, Hkv, d, dtype=torch.bfloat16, device="cuda")
    row = torch.randperm(20, generator=g, device="cuda").int()[:17]
    V = pool.clone()
    pool[row.long()] = torch.cat([k, k[:272 - n]]).view(17, ps, Hkv, d)
    V[row.long()] = torch.cat([v, v[:272 - n]]).view(17, ps, Hkv, d)
    table = row.expand(2, 17).contiguous()
    out, lse = chunk(H, q, pool.permute(0, 2, 1, 3), V.permute(0, 2, 1, 3), table, docs[1:], [190, 267], Hkv, Opts(first=[100, 190]), torch.float32)
    want = prefill(H, q, k[100:], v[100:], docs[1:], Opts(), torch.float32)
    # the same sums over tiles that begin elsewhere: both within the tolerance of the definition
    check_prefill(q, k[100:], v[100:], docs[1:], Opts(), out, lse)
    check_prefill(q, k[100:], v[100:], docs[1:], Opts(), *want)


def test_rows_behind_and_other_sequences(H):
    g = torch.Generator(device="cuda").manual_seed(45)
    new, Hq, Hkv, d = [70, 33], 4, 2, 64
    qkv = rand(g, sum(new) + 9, Hq + 2 * Hkv, d)
    qkv[:70] = NAN
    qkv[103:] = NAN
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    opts = Opts(cap=50.0, slopes=alibi(Hq), prefix=[70, 20], window=25, first=[0, 3])
    out, lse = prefill(H, q, k, v, new, opts)
    assert torch.isnan(out[103:]).all() and torch.isnan(lse[103:]).all() and torch.isnan(out[:70]).all()
    check_rows(out[70:103, 1], lse[70:103, 1], SO.attention(*(x[70:103, i].double().cpu().numpy() for x, i in ((q, 1), (k, 0), (v, 0))), **opts.of(1, 1)), "")


def test_a_number_that_is_none_reaches_its_own_row(H):
    """NaN in a query, or in a key that is seen, makes NaN of the rows that see it, and of no other."""
    g = torch.Generator(device="cuda").manual_seed(46)
    n, d = 300, 128
    for cap, window in ((50.0, 60), (1.0, 60), (0.0, 60)):
        q, k, v = rand(g, n, 2, d), rand(g, n, 1, d), rand(g, n, 1, d)
        opts = Opts(cap=cap, window=window)
        clean = prefill(H, q, k, v, [n], opts)
        q[5, 1] = NAN
        k[100] = NAN
        out, lse = prefill(H, q, k, v, [n], opts)
        hit = torch.zeros(n, 2, dtype=torch.bool, device="cuda")
        hit[5, 1] = True
        hit[100:160] = True
        assert torch.equal(torch.isnan(lse), hit) and torch.isnan(out[hit]).all()
        check = ~hit
        assert torch.equal(out[check], clean[0][check]) and torch.equal(lse[check], clean[1][check])


def test_graph_and_changed_options(H):
    """A captured call reads first, prefix, lengths and the options' arrays when it runs; two graphs share a workspace."""
    g = torch.Generator(device="cuda").manual_seed(47)
    lens, Hq, Hkv, d = [900, 300], 8, 2, 128
    o1, o2 = Opts(cap=50.0, first=[10, 20], slopes=alibi(Hq)), Opts(window=100, prefix=[40, 290])
    new = [1, 40]
    K, V, table = pages(g, new, lens, 16, Hkv, d, "token", Opts())
    q = rand(g, sum(new), Hq, d)
    tok, cache = H.make_tokens(q, None, None, 2, h_kv=Hkv, out_dtype=torch.bfloat16), H.make_cache(K, V, table)
    ws, cu, lt = workspace(H, tok), sums(new), ints(lens)
    res = []
    for o in (o1, o2):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        made = o.made(H)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            H.hash_attn_chunk_ex(tok, cache, made, q, K, V, table, cu, lt, out, lse, workspace=ws)
        res.append((o, made, graph, out, lse))
    for _ in range(3):
        for o, made, graph, out, lse in res:
            graph.replay()
    for o, made, graph, out, lse in res:
        check_chunk(q, K, V, table, new, lens, o, out, lse, heads=[0, 5])
    o, made, graph, out, lse = res[0]
    made.tensors[2].copy_(ints([500, 0]))
    made.tensors[0].mul_(0.5)
    o.first, o.slopes = [500, 0], [x / 2 for x in o.slopes]
    graph.replay()
    check_chunk(q, K, V, table, new, lens, o, out, lse, heads=[0, 5])


def test_two_streams(H):
    g = torch.Generator(device="cuda").manual_seed(48)
    n, d = 1500, 128
    q, k, v = rand(g, n, 4, d), rand(g, n, 2, d), rand(g, n, 2, d)
    opts = [Opts(cap=50.0), Opts(window=200, slopes=alibi(4))]
    want = [prefill(H, q, k, v, [n], o) for o in opts]
    tok = H.make_tokens(q, k, v, 1, out_dtype=torch.bfloat16)
    ws, made, cu = [workspace(H, tok) for _ in opts], [o.made(H) for o in opts], sums([n])
    outs = [(torch.empty_like(q), torch.empty(n, 4, device="cuda")) for _ in opts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                H.hash_attn_prefill_ex(tok, made[i], q, k, v, cu, *outs[i], workspace=ws[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, o in zip(want, outs) for a, b in zip(w, o))


def random_case(seed):
    r = random.Random(seed)
    Hkv, G, d = r.choice([1, 2, 3]), r.choice([1, 2, 3, 4, 5, 7, 8, 16, 20]), r.choice([64, 128])
    n = r.randint(1, 6)
    new = [r.choice([0, 1, 1, r.randint(2, 40), r.randint(2, 300)]) for _ in range(n)]
    if sum(new) == 0:
        new[0] = 1
    lens = [m + r.choice([0, r.randint(0, 900), r.randint(-m, 0)]) for m in new]
    at = lambda: [r.choice([0, t, r.randint(0, t)]) for t in lens]  # noqa: E731
    opts = Opts(cap=r.choice([0, 0, 0.5, 30, 50, 300]), window=r.choice([0, 0, 1, r.randint(1, 200), r.randint(1, 1000)]),
                slopes=r.choice([None, [r.uniform(-0.05, 1) for _ in range(Hkv * G)]]), prefix=r.choice([None, at()]), first=r.choice([None, at()]),
                scale=r.choice([None, None, 0.3]))
    return new, lens, Hkv * G, Hkv, d, r.choice([16, 16, 48, 64, 128, 256]), r.choice(["token", "head"]), opts, r.choice([torch.bfloat16, torch.float32])


@pytest.mark.parametrize("seed", range(60))
def test_random_chunks(H, seed):
    new, lens, Hq, Hkv, d, ps, order, opts, dt = random_case(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    K, V, table = pages(g, new, lens, ps, Hkv, d, order, opts)
    q = rand(g, sum(new), Hq, d, scale=2.0)
    out, lse = chunk(H, q, K, V, table, new, lens, Hkv, opts, dt)
    check_chunk(q, K, V, table, new, lens, opts, out, lse, str(vars(opts)), heads=sorted({0, Hq - 1}))


# ---------------------------------------------------------------- a serving run

def test_serving_run(H):
    """Plan, append with three axes, attention with a cap, a window and a prefix, step after step: against attention
    over each sequence's whole history. Sequences end and their pages go to others."""
    g = torch.Generator(device="cuda").manual_seed(51)
    n, Hq, Hkv, d, ps, n_pages, cols, room = 3, 4, 2, 64, 16, 24, 8, 120
    pool = [torch.full((n_pages, ps, Hkv, d), NAN, dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3) for _ in range(2)]
    table, free, n_free = torch.full((n, cols), -1, dtype=torch.int32, device="cuda"), torch.arange(n_pages, device="cuda").int(), ints([n_pages])
    lens, cu, flags, prefix = ints([0] * n), ints([0] * (n + 1)), ints([0]), ints([0] * n)
    paging = H.make_paging(table, n_pages, ps, room)
    inv = torch.tensor([100.0 ** (-i / 32) for i in range(32)], device="cuda")
    axis = [0, 1, 2, 0] * 8
    rope = H.rope_axes(inv, axis)
    o = dict(cap=30.0, window=50)
    history = [None] * n
    pre = [0] * n
    r = random.Random(9)
    for step, new in enumerate([[40, 7, 0], [1, 1, 60], [1, -1, 1], [25, 33, 1], [-1, 1, -1], [50, 1, 2], [1, 1, 1]]):
        T = sum(max(m, 0) for m in new)
        qkv = rand(g, room, Hq + 2 * Hkv, d)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        pos = torch.randint(0, 300, (3, room), generator=g, device="cuda").int()
        H.hash_attn_plan_pages(paging, ints(new), lens, lens, cu, table, free, n_free, n_free, dev_flags=flags)
        for s, m in enumerate(new):
            if m < 0:
                history[s] = None
            elif m > 0 and history[s] is None:
                pre[s] = r.randint(0, m)
        prefix.copy_(ints(pre))
        q_out = torch.zeros(room, Hq, d, dtype=torch.bfloat16, device="cuda")
        tok, cache = H.make_tokens(q, k, v, n, out_dtype=torch.float32), H.make_cache(*pool, table)
        H.hash_attn_append_axes(tok, cache, q, k, v, table, cu, lens, pos, q_out, *pool, rope=rope, dev_flags=flags)
        rot = H.make_tokens(q_out, None, None, n, h_kv=Hkv, out_dtype=torch.float32)
        ws = workspace(H, rot)
        out, lse = torch.full((room, Hq, d), NAN, device="cuda"), torch.full((room, Hq), NAN, device="cuda")
        H.hash_attn_chunk_ex(rot, cache, H.score_opts(softcap=o["cap"], window=o["window"], prefix=prefix), q_out, *pool, table, cu, lens, out, lse,
                             workspace=ws)
        assert H.hash_attn_device_status(ws) == (0, 0) and flags.item() == 0
        ph, a = pos.cpu().numpy(), 0
        for s, m in enumerate(new):
            if m <= 0:
                continue
            kk = np.stack([SO.rotate_axes(k[t].double().cpu().numpy(), ph[:, t], axis, inv.double().cpu().numpy()) for t in range(a, a + m)])
            vv = v[a:a + m].double().cpu().numpy()
            history[s] = (kk, vv) if history[s] is None else tuple(np.concatenate(x) for x in zip(history[s], (kk, vv)))
            row = table[s].tolist()
            for h in range(Hq):
                Kc, Vc = (PO.page_rows(x[:, h // 2].double().cpu().numpy(), row, len(history[s][0])) for x in pool)
                assert np.array_equal(Vc, history[s][1][:, h // 2])
                assert np.all(np.abs(Kc - history[s][0][:, h // 2]) <= 2.0 ** -8 * np.abs(Kc) + 1e-5)  # rotated, then rounded to bf16
                ref = SO.attention(q_out[a:a + m, h].double().cpu().numpy(), Kc, Vc, prefix=pre[s], **o)
                check_rows(out[a:a + m, h], lse[a:a + m, h], ref, f"step {step} seq {s} head {h}")
            a += m
        assert torch.isnan(out[T:]).all()
    assert lens.tolist() == [51, 36, 3] and n_free.item() == n_pages - 4 - 3 - 1


def test_a_captured_serving_step(H):
    """Plan, append and attention captured once: replays with other lengths, one of which ends a sequence and one of which
    runs out of pages (that sequence is stopped: out = 0, lse = -inf, and it goes on when its length is written again)."""
    g = torch.Generator(device="cuda").manual_seed(52)
    n, Hq, Hkv, d, ps, n_pages, room = 3, 8, 2, 128, 16, 6, 40
    pool = [torch.zeros(n_pages, ps, Hkv, d, dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3) for _ in range(2)]
    table, free, n_free = torch.full((n, 4), -1, dtype=torch.int32, device="cuda"), torch.arange(n_pages, device="cuda").int(), ints([n_pages])
    lens, cu, new, flags = ints([0] * n), ints([0] * (n + 1)), ints([1] * n), ints([0])
    q, k, v = rand(g, room, Hq, d), rand(g, room, Hkv, d), rand(g, room, Hkv, d)
    q_out, out, lse = torch.zeros_like(q), torch.full((room, Hq, d), NAN, device="cuda"), torch.full((room, Hq), NAN, device="cuda")
    pos, slots = torch.zeros(2, room, dtype=torch.int32, device="cuda"), torch.zeros(room, dtype=torch.int32, device="cuda")
    paging, rope = H.make_paging(table, n_pages, ps, room), H.rope_axes(torch.ones(8, device="cuda"), [0, 1] * 4)
    tok, cache = H.make_tokens(q, k, v, n, out_dtype=torch.float32), H.make_cache(*pool, table)
    ws, opts = workspace(H, tok), H.score_opts(softcap=30.0, window=20)

    def step():
        H.hash_attn_plan_pages(paging, new, lens, lens, cu, table, free, n_free, n_free, slots=slots, dev_flags=flags)
        H.hash_attn_append_axes(tok, cache, q, k, v, table, cu, lens, pos, q_out, *pool, rope=rope)
        H.hash_attn_chunk_ex(tok, cache, opts, q_out, *pool, table, cu, lens, out, lse, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    history = [np.zeros((0, Hkv, d))] * n
    keys = [np.zeros((0, Hkv, d))] * n
    for i, (ms, want) in enumerate([([20, 1, 10], [20, 1, 10]), ([1, 16, 1], [21, 17, 11]), ([1, 1, 30], [22, 18, -12]), ([1, -1, 0], [23, 0, -12]),
                                    ([1, 0, 30], [24, 0, 41])]):
        if i == 4:
            lens[2] = 11  # the host lets it go on
        new.copy_(ints(ms))
        flags.zero_()
        out.fill_(NAN)
        graph.replay()
        assert lens.tolist() == want, i
        assert flags.item() == (H.HA_DEVERR_PAGES if i == 2 else 0), i
        st = H.hash_attn_device_status(ws)
        assert st == ((H.HA_ERR_DEVICE, H.HA_DEVERR_SEQLEN) if i in (2, 3) else (0, 0)), i
        a = 0
        for s, m in enumerate(ms):
            if m < 0:
                history[s] = keys[s] = np.zeros((0, Hkv, d))
                continue
            if want[s] < 0:
                assert torch.all(out[a:a + m] == 0) and torch.all(torch.isneginf(lse[a:a + m])) and torch.all(slots[a:a + m] == -1)
            elif m:
                keys[s] = np.concatenate([keys[s], k[a:a + m].double().cpu().numpy()])   # (positions are 0: nothing turns)
                history[s] = np.concatenate([history[s], v[a:a + m].double().cpu().numpy()])
                for h in (0, 5):
                    ref = SO.attention(q[a:a + m, h].double().cpu().numpy(), keys[s][:, h // 4], history[s][:, h // 4], cap=30.0, window=20)
                    check_rows(out[a:a + m, h], lse[a:a + m, h], ref, f"step {i} seq {s} head {h}")
            a += max(m, 0)
        assert torch.isnan(out[a:]).all()
