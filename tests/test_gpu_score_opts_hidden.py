"""Scores with options: what a token does not see, and rows that are not its sequence's, leave its result's bits as
they are, whatever numbers they hold."""
import pytest
import torch

import test_gpu_score_opts as S
from test_gpu_score_opts import H  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

# capped with a reference that stays, with one that moves, biased, masked alone
OPTIONS = {"cap-50": dict(cap=50.0), "cap-200": dict(cap=200.0), "cap-bias": dict(cap=50.0, slopes=True), "bias": dict(slopes=True),
           "scale": dict(scale=0.2), "cap-window": dict(cap=50.0, window=40)}
TYPES = pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])


def options(name, Hq, **kw):
    o = dict(OPTIONS[name], **kw)
    return S.Opts(**{**o, "slopes": S.alibi(Hq) if o.get("slopes") else None})


def same(a, b, rows):
    return torch.equal(a[0][rows], b[0][rows]) and torch.equal(a[1][rows], b[1][rows])


@TYPES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [3, 4])
@pytest.mark.parametrize("name", OPTIONS)
def test_prompts_of_others(H, name, G, d, out_dtype):  # noqa: F811
    """The prompts before and behind one have ordinary queries and keys, or large ones."""
    g = torch.Generator(device="cuda").manual_seed(61)
    new, Hkv = [37, 133, 9, 60], 2
    T, mine = sum(new), slice(37, 179)
    q, k, v = S.rand(g, T, G * Hkv, d, scale=2.0), S.rand(g, T, Hkv, d), S.rand(g, T, Hkv, d)
    o = options(name, G * Hkv)
    want = S.prefill(H, q, k, v, new, o, out_dtype)
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[mine] = False
    for by in (100.0, 1e4):
        qo, ko = q.clone(), k.clone()
        qo[others] *= by
        ko[others] *= by
        assert same(S.prefill(H, qo, ko, v, new, o, out_dtype), want, mine), by


@TYPES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [3, 4])
@pytest.mark.parametrize("name", OPTIONS)
def test_new_tokens_of_others(H, name, G, d, out_dtype):  # noqa: F811
    """A token over 700 keys and a chunk, each followed by other sequences' tokens, whose rows lie in the same tile of
    queries; the others' queries are ordinary, or large."""
    g = torch.Generator(device="cuda").manual_seed(62)
    new, lens, Hkv = [1, 30, 40, 25], [700, 100, 330, 64], 1
    o = options(name, G)
    K, V, table = S.pages(g, new, lens, 16, Hkv, d, "token", o)
    q = S.rand(g, sum(new), G, d, scale=2.0)
    want = S.chunk(H, q, K, V, table, new, lens, Hkv, o, out_dtype)
    for by in (100.0, 1e4):
        qo = q.clone()
        qo[1:31] *= by
        qo[71:] *= by
        got = S.chunk(H, qo, K, V, table, new, lens, Hkv, o, out_dtype)
        assert same(got, want, slice(0, 1)) and same(got, want, slice(31, 71)), by


@TYPES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", OPTIONS)
def test_unseen_cache_rows(H, name, d, out_dtype):  # noqa: F811
    """Rows before the first key and behind the last one hold zeros, large numbers or infinities."""
    g = torch.Generator(device="cuda").manual_seed(63)
    new, lens, Hkv, G = [1, 50, 3], [333, 210, 70], 1, 4
    o = options(name, G, first=[37, 21, 5])
    K, V, table = S.pages(g, new, lens, 16, Hkv, d, "token", o)
    q = S.rand(g, sum(new), G, d, scale=2.0)
    hidden, got = torch.isnan(K), []
    assert hidden.any()
    for x in (0.0, 1e4, -1e4, float("inf"), float("nan")):
        K[hidden] = x
        V[hidden] = x
        got.append(S.chunk(H, q, K, V, table, new, lens, Hkv, o, out_dtype))
    assert all(same(x, got[0], slice(None)) for x in got)


@TYPES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", OPTIONS)
def test_later_keys_of_the_own_prompt(H, name, d, out_dtype):  # noqa: F811
    """128 heads to a KV head: a tile is one token, so its keys are all that its rows see. The tokens behind it bring
    ordinary keys, or large ones."""
    g = torch.Generator(device="cuda").manual_seed(64)
    n, G, at = 90, 128, 70
    q, k, v = S.rand(g, n, G, d, scale=2.0), S.rand(g, n, 1, d), S.rand(g, n, 1, d)
    o = options(name, G)
    want = S.prefill(H, q, k, v, [n], o, out_dtype)
    for by in (100.0, 1e4):
        ko = k.clone()
        ko[at:] *= by
        assert same(S.prefill(H, q, ko, v, [n], o, out_dtype), want, slice(0, at)), by


@TYPES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [3, 5, 7, 100])
@pytest.mark.parametrize("name", ["cap-50", "cap-200", "cap-bias"])
def test_what_an_earlier_call_left(H, name, G, d, out_dtype):  # noqa: F811
    """Rows of a tile that belong to no token (G does not divide 128) hold what was there before."""
    g = torch.Generator(device="cuda").manual_seed(65)
    n = 200
    q, k, v = S.rand(g, n, G, d, scale=2.0), S.rand(g, n, 1, d), S.rand(g, n, 1, d)
    o = options(name, G)
    want = S.prefill(H, q, k, v, [n], o, out_dtype)
    big = [S.rand(g, 152 * 64, 4, d, scale=1e4), S.rand(g, 152 * 64, 1, d, scale=1e4), S.rand(g, 152 * 64, 1, d)]
    for _ in range(2):
        S.prefill(H, *big, [64] * 152, S.Opts(), out_dtype)
        assert same(S.prefill(H, q, k, v, [n], o, out_dtype), want, slice(None))
