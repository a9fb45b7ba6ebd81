"""Packed attention and append where a wait, a bound or a rounding is at its edge
(tolerances as in test_gpu_packed unless a test derives its own)."""
import math
from fractions import Fraction

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


def pi_scaled(bits):
    """floor(pi 2^bits), nearly: Machin's formula in integers."""
    one = 1 << (bits + 32)

    def arctan_of_inverse(x):
        term, n, sign, total = one // x, 3, -1, one // x
        while term:
            term //= x * x
            total += sign * (term // n)
            n, sign = n + 2, -sign
        return total
    return 4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239)) >> 32


def test_every_pair_keeps_its_angle_at_every_position(H):  # noqa: F811
    """cos and sin of pos inv_freq, each pair by itself, against the angle modulo a turn from whole
    numbers. The angle is off by 2^-25 + 2^-32 + (|w| + 2) pos 2^-64 half turns at most, its cosine by pi
    times that; sincospif adds 2 steps of a value below 1 (2^-23)."""
    d, ps, bits = 64, 1 << 10, 256
    pi = pi_scaled(bits)
    assert abs(pi / 2 ** bits - math.pi) < 1e-15
    x = torch.zeros(1, 1, d, device="cuda")
    x[..., : d // 2] = 1.0  # a pair (1, 0) becomes (cos, sin)
    K, V = torch.zeros(1, 1, ps, d, device="cuda"), torch.zeros(1, 1, ps, d, device="cuda")
    table = torch.zeros(1, 1 << 20, dtype=torch.int32, device="cuda")
    w = torch.cat([P.inv_freq(d)[:14], torch.tensor([1.0, 0.3333333, 0.99999994, 3.0, 1e-9, 1e-30, 1e-40, 0.0, -0.7, -1e-4, 65504.0],
                                                    device="cuda"), P.inv_freq(d)[25:]])
    ws = [Fraction(float(f)) for f in w.cpu()]
    rng = np.random.default_rng(5)
    for pos in [0, 1, 2, 12345, 1 << 20, (1 << 24) + 1, (1 << 30) - 1] + [int(p) for p in rng.integers(0, 1 << 30, 20)]:
        q_out = torch.empty(1, 1, d, device="cuda")
        P.run_append(H, x, x, x, table, [1], [pos + 1], q_out, K, V, H.rope(w))
        got = q_out[0, 0].double().cpu().numpy()
        for p, f in enumerate(ws):
            half = f * pos * (1 << bits) / pi  # half turns
            a = math.pi * float(half - 2 * round(half / 2))
            tol = math.pi * (2.0 ** -25 + 2.0 ** -32 + (abs(float(f)) + 2) * pos * 2.0 ** -64) + 2.0 ** -23 + 1e-15
            err = max(abs(got[p] - math.cos(a)), abs(got[p + d // 2] - math.sin(a)))
            assert err <= tol, (pos, float(f), err, tol)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_scores_in_the_thousands_that_are_exact(H, d, out_dtype):  # noqa: F811
    """Scores S = 256 h + l of whole numbers: exact in float32, up to 65,535 / sqrt(d), growing from
    tile to tile, so that O is rescaled again and again and nothing hides in the products' rounding.

    With t = log2(e) S / sqrt(d) at its largest and u = 2^-24: a weight's exponent is x qscale - m qscale
    with m qscale rounded (u t), which differs between the references m that the sums passed through (2 u t
    between two of them); qscale itself and the product of each rescaling are rounded (u t each over
    all of them), and the same once more where parts are joined: 8 u t in all. Then 2^-22 for an
    exponential, twice, and 2 u for each of n terms."""
    g = torch.Generator(device="cuda").manual_seed(d)
    T, Hkv, lens, new = 700, 2, [3000, 700, 900], [1, 90, 3]
    u = 2.0 ** -24

    def keys(n):
        k = torch.zeros(n, Hkv, d, device="cuda")
        step = torch.randint(0, 2, (n // 64 + 1,), generator=g, device="cuda") * torch.randint(1, 9, (n // 64 + 1,), generator=g, device="cuda")
        k[:, :, 0] = torch.cumsum(step, 0).clamp(max=255)[torch.arange(n, device="cuda") // 64][:, None]
        k[:, :, 1] = torch.randint(0, 256, (n, Hkv), generator=g, device="cuda")
        return k.bfloat16()

    def queries(n):
        q = torch.zeros(n, 4 * Hkv, d, device="cuda")
        q[:, :, 0], q[:, :, 1] = 256.0, 1.0
        return q.bfloat16()

    def check(out, lse, ref, what):
        ro, rl, mag, zmax, n = ref
        t = zmax * math.log2(math.e)
        E = math.log(2) * 8 * u * t + 2.0 ** -21 + 2 * u * (n + 16)
        tol = 2 * E[:, None] * mag + 1e-30
        if out_dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * mag * (1 + 2 * E[:, None]) + 2.0 ** -8 * np.abs(ro) * (1 + 2.0 ** -7)
        err = np.abs(out.flatten(0, 1).double().cpu().numpy() - ro)
        assert np.all(err <= tol), f"{what}: out off by {err.max():.3g}, worst ratio {(err / tol).max():.3g}"
        el = np.abs(lse.flatten().double().cpu().numpy() - rl)
        assert np.all(el <= E + 2.0 ** -22 * (1 + np.abs(rl))), f"{what}: lse off by {el.max():.3g}"

    q, k, v = queries(T), keys(T), P.rand(g, T, Hkv, d)
    out, lse, st = P.run_prefill(H, q, k, v, [T], out_dtype)
    assert st == (0, 0)
    check(out, lse, P.reference(q, lambda s: k, lambda s: v, [T], [T]), "prefill")

    K, V, table = P.pages(g, lens, 16, Hkv, d)
    seqs = [keys(n) for n in lens]
    for s, n in enumerate(lens):
        j = torch.arange(n, device="cuda")
        K[table[s].long()[j // 16], :, j % 16] = seqs[s]
    q = queries(sum(new))
    out, lse, st = P.run_chunk(H, q, K, V, table, new, lens, Hkv, out_dtype)
    assert st == (0, 0)

    def values(s):
        j = torch.arange(lens[s], device="cuda")
        return V[table[s].long()[j // 16], :, j % 16]
    check(out, lse, P.reference(q, lambda s: seqs[s], values, new, lens), "chunk")


def test_an_infinity_in_v_stays_in_its_sequence_and_behind_its_key_tile(H):  # noqa: F811
    """V has to be finite within a sequence. Where it is not, rows whose key tiles end before that
    token, other sequences and other heads keep their values."""
    g = torch.Generator(device="cuda").manual_seed(8)
    new, Hkv, d = [640, 200], 2, 128
    T = sum(new)
    q, k, v = P.rand(g, T, 4 * Hkv, d), P.rand(g, T, Hkv, d), P.rand(g, T, Hkv, d)
    for out_dtype, tile in ((torch.bfloat16, 128), (torch.float32, 64)):
        want = P.run_prefill(H, q, k, v, new, out_dtype)
        bad = v.clone()
        bad[500, 0, 7] = float("inf")
        out, lse, st = P.run_prefill(H, q, k, bad, new, out_dtype)
        assert st == (0, 0) and torch.equal(lse, want[1])
        first = 500 // tile * tile
        # an item is 64 tokens, all of whose rows take the key tiles that its last token sees
        first = first // 64 * 64
        assert torch.equal(out[:first], want[0][:first]) and torch.equal(out[640:], want[0][640:])
        assert torch.equal(out[:, 4:], want[0][:, 4:])
        other = torch.arange(d, device="cuda") != 7
        assert torch.equal(out[:640, :4][..., other], want[0][:640, :4][..., other])
        assert not torch.isfinite(out[500:640, :4, 7]).any()


@pytest.mark.parametrize("n", [100, 5000, 1 << 20])
@pytest.mark.parametrize("d", [64, 128])
def test_a_few_sequences_among_many_without_new_tokens(H, d, n):  # noqa: F811
    """The longest list of sequences, nearly all without new tokens (some of those have keys)."""
    g = torch.Generator(device="cuda").manual_seed(n + d)
    Hkv, ps, wide = 2, 128, 8
    own = {0: (3, 500), 5: (1, 1), 6: (0, 300), n // 2 - 30: (70, 800), n // 2: (200, 200), n - 40: (0, 7), n - 1: (2, 1000)}
    new, lens = torch.zeros(n, dtype=torch.int32), torch.zeros(n, dtype=torch.int32)
    for s, (a, b) in own.items():
        new[s], lens[s] = a, b
    table = torch.full((n, wide), -1, dtype=torch.int32, device="cuda")
    perm = torch.randperm(wide * len(own), generator=g, device="cuda").to(torch.int32)
    for i, s in enumerate(own):
        table[s] = perm[i * wide:(i + 1) * wide]
    rows = [s for s, (a, _) in own.items() if a]
    T, cu = int(new.sum()), torch.cat([torch.zeros(1, dtype=torch.int32), torch.cumsum(new, 0).int()]).cuda()
    K, V = P.rand(g, wide * len(own), Hkv, ps, d), P.rand(g, wide * len(own), Hkv, ps, d)
    q, k, v = P.rand(g, T, 8, d), P.rand(g, T, Hkv, d), P.rand(g, T, Hkv, d)
    tok = H.make_tokens(q, k, v, n, out_dtype=torch.bfloat16)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    H.hash_attn_append(tok, H.make_cache(K, V, table), None, k, v, table, cu, lens.cuda(), None, K, V, dev_flags=flags)
    assert int(flags) == 0

    def cached(X, s):
        j = torch.arange(own[s][1], device="cuda")
        return X[table[s].long()[j // ps], :, j % ps]
    at = 0
    for s in rows:
        a, b = own[s]
        assert torch.equal(cached(K, s)[b - a:], k[at:at + a]) and torch.equal(cached(V, s)[b - a:], v[at:at + a])
        at += a
    for out_dtype in (torch.bfloat16, torch.float32):
        out, lse, st = P.run_chunk(H, q, K, V, table, new.tolist(), lens.tolist(), Hkv, out_dtype, cu=cu, lens_t=lens.cuda())
        assert st == (0, 0), hex(st[1])
        ref = P.reference(q, lambda i: cached(K, rows[i]), lambda i: cached(V, rows[i]), [own[s][0] for s in rows],
                          [own[s][1] for s in rows])
        P.check_rows(out.flatten(0, 1), lse.flatten(), ref, out_dtype == torch.bfloat16, f"{n} sequences")
