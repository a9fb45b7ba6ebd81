"""The page plan (hash_attn_plan_pages) and the append with several axes (hash_attn_append_axes)
against their oracle.

Plans are whole numbers: equal. Rotations: with u = 2^-24, the angle is off by at most 2^-25 + 2^-32
of a half turn (pi times that in radians, below 1.0e-7), cosine and sine by 2 units in the last
place (1.2e-7) more, a product and the sum are rounded (0.6e-7 each): below 3.4e-7 (|a| + |b|), for which
2^-21 stands; then once to the type of the row (2^-8 relative in bf16, 2^-24 in float32)."""
import random

import numpy as np
import pytest
import torch

from oracle import serving_oracle as SO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def H():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from long_context_sparse_score_gb300 import _build
    _build.build()
    from long_context_sparse_score_gb300 import hashattn
    hashattn.lib()
    return hashattn


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Plan:
    """A plan's inputs on the host, its call and its comparison."""

    def __init__(self, new, had, page_size, spare, total=None, cols=None, seed=0):
        r = random.Random(seed)
        self.new, self.had, self.ps = list(new), list(had), page_size
        held = [-(-max(h, -1 - h) // page_size) for h in had]
        self.n_pages = max(1, sum(held) + spare)
        self.cols = cols or max(1, max(-(-(max(h, -1 - h) + max(m, 0)) // page_size) for m, h in zip(new, had)))
        perm = list(range(self.n_pages))
        r.shuffle(perm)
        self.table, at = [], 0
        for n in held:
            self.table.append((perm[at:at + n] + [-9] * self.cols)[:self.cols])
            at += n
        self.free, self.n_free = perm[at:] + [-3] * at, self.n_pages - at
        self.total = sum(max(m, 0) for m in new) if total is None else total

    def want(self):
        return SO.plan_pages(self.new, self.had, self.table, self.free, self.n_free, self.n_pages, self.ps, self.total)

    def put(self, H, in_place=False, slots=True, pad=0):
        """The device's side: a table with rows of `pad` more entries."""
        self.t = {k: ints(getattr(self, k)) for k in ("new", "had", "free")}
        wide = torch.full((len(self.new), self.cols + pad), -77, dtype=torch.int32, device="cuda")
        wide[:, :self.cols] = ints(self.table)
        self.t["table"] = wide[:, :self.cols]
        self.t["n_free"] = ints([self.n_free])
        self.t["lens"] = self.t["had"] if in_place else torch.full_like(self.t["had"], -55)
        self.t["n_out"] = self.t["n_free"] if in_place else torch.full_like(self.t["n_free"], -55)
        self.t["cu"] = torch.full((len(self.new) + 1,), -55, dtype=torch.int32, device="cuda")
        self.t["slots"] = torch.full((self.total + 4,), -55, dtype=torch.int32, device="cuda") if slots else None
        self.t["flags"] = ints([0])
        self.paging = H.make_paging(self.t["table"], self.n_pages, self.ps, self.total)
        self.wide = wide
        return self

    def run(self, H):
        t = self.t
        H.hash_attn_plan_pages(self.paging, t["new"], t["had"], t["lens"], t["cu"], t["table"], t["free"], t["n_free"], t["n_out"],
                               slots=None if t["slots"] is None else t["slots"][:self.total], dev_flags=t["flags"])
        return self

    def check(self, what=""):
        w, t = self.want(), {k: v.cpu().tolist() for k, v in self.t.items() if v is not None}
        assert t["cu"] == w["cu"], what
        assert t["lens"] == w["lens"], what
        assert t["table"] == w["table"], what
        assert t["free"] == w["free"], what
        assert t["n_out"] == [w["n_free"]], what
        assert t["flags"] == [w["flags"]], (what, t["flags"], w["flags"])
        if self.t["slots"] is not None:
            assert t["slots"] == w["slots"] + [-55] * 4, what  # and nothing behind them
        assert (self.wide[:, self.cols:] == -77).all(), what


PLANS = {
    # new, had, page size, spare pages
    "one": ([1], [0], 16, 1), "one-of-none": ([0], [0], 16, 1), "fills-a-page": ([1], [15], 16, 0), "begins-a-page": ([1], [16], 16, 1),
    "page-of-one": ([3, 1], [2, 0], 1, 9), "ends": ([-1], [33], 16, 0), "ends-empty": ([-1, 2], [0, 0], 16, 1),
    "rows-of-8": ([8, 9, 7, 8], [15, 8, 0, 16], 8, 8), "taken-over": ([-1, 40, -5, 20], [40, 0, 17, 3], 16, 0),
    "short": ([1, 5, 1, 1], [4, 0, 8, 1], 4, 2), "short-long": ([10, 600, 300, 1, 9, 400], [0] * 6, 16, 30),
    "none-free": ([1, 1, 0], [16, 5, 16], 16, 0), "long-prompts": ([5000, 1, 2049], [0, 700, 31], 48, 300),
    "stopped": ([1, 0, -1, 700], [-6, -33, -18, -1], 16, 4),
    # a cluster's CTAs that look at all sequences, and at a part of them each
    "shared": ([40, -1, 33, 1] * 32, [0, 50, 7, 16] * 32, 16, 400), "parted": ([40, -1, 33, 1] * 32 + [900], [0, 50, 7, 16] * 32 + [3], 16, 460),
    "parted-short": ([40, -1, 33, 1] * 64, [0, 50, 7, 16] * 64, 16, 20),
}


@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in-place"])
@pytest.mark.parametrize("case", PLANS)
def test_plan(H, case, in_place):
    p = Plan(*PLANS[case]).put(H, in_place, pad=3).run(H)
    p.check()


@pytest.mark.parametrize("case", PLANS)
def test_plan_without_slots_or_room_to_spare(H, case):
    Plan(*PLANS[case]).put(H, slots=False).run(H).check()
    new = PLANS[case][0]
    Plan(*PLANS[case], total=sum(max(m, 0) for m in new) + 5000).put(H).run(H).check()


def test_plan_again_from_the_same_inputs(H):
    p = Plan([40, -1, 3, -1, 300], [5, 50, 16, 99, 0], 16, 10).put(H).run(H)
    p.check()
    p.run(H).run(H).check()


def random_plan(seed):
    r = random.Random(seed)
    n = r.choice([1, 2, 31, 33, 64, 200, 1023, 1024, 1025, 2500, 9000])
    hi = r.choice([1, 1, 8, 9, 40, 700 if n < 300 else 60])
    ps = r.choice([1, 3, 16, 16, 48, 64])
    had = [r.randint(0, r.choice([1, 40, 200])) for _ in range(n)]
    ends, many = r.choice([0, 0.1, 0.6]), r.choice([0, 0.2, 1])
    new = [-r.randint(1, 3) if r.random() < ends else (r.randint(0, hi) if r.random() < many else r.randint(0, 1)) for _ in range(n)]
    need = sum(-(-(h + m) // ps) - -(-h // ps) for m, h in zip(new, had) if m > 0)
    if r.random() < 0.3:  # some that were stopped before, or outgrow their row
        for _ in range(min(n, 5)):
            had[r.randrange(n)] = -1 - r.randint(0, 40)
    cols = r.choice([None, None, max(1, -(-max(had) // ps))])
    return Plan(new, had, ps, r.choice([need, need + 7, need // 2]), cols=cols, seed=seed, total=sum(max(m, 0) for m in new) + r.choice([0, 0, 77]))


@pytest.mark.parametrize("seed", range(40))
def test_plan_of_random_batches(H, seed):
    p = random_plan(seed)
    p.put(H, in_place=bool(seed & 1), pad=seed % 3).run(H)
    p.check(f"n {len(p.new)}")


def test_plan_that_has_no_room(H):
    """More rows than the packed buffers: nothing is planned, and nothing is lost."""
    for n in (3, 1500):
        p = Plan([4, -1, 9] * (n // 3), [3, 20, 0] * (n // 3), 16, 3000, total=13 * (n // 3) - 1).put(H, in_place=True).run(H)
        p.check()
        assert p.t["had"].tolist() == p.had


def test_plan_of_lengths_that_cannot_be(H):
    p = Plan([1, 0, 3, -1, 2, 1], [100, 97, 0, -5, 10, 0], 16, 40, cols=6)
    p.had[2] = -1 - (1 << 30)
    p.new[2] = (1 << 24) + 7  # and more rows than any buffer: nothing is planned
    p.total = 1 << 10
    p.put(H).run(H).check()
    p.new[2] = 3
    p.put(H).run(H).check()


def test_plan_flags_pages_that_are_none_and_pages_given_back_twice(H):
    p = Plan([-1, 40, -1], [40, 0, 20], 16, 3)
    p.table[0][1] = 4000        # not a page: left out
    p.free[p.n_free - 1] = -2   # nor this one: entered as -1
    p.put(H).run(H).check()
    p = Plan([-1, -1], [64, 64], 16, 0)
    p.table[1] = list(p.table[0])
    p.n_free = 6  # two places are left for eight pages
    p.put(H).run(H).check()
    for n in (-1, 99):
        p = Plan([1, 1], [16, 3], 16, 5)
        p.n_free = n
        p.put(H).run(H).check()


def test_plan_of_many_sequences(H):
    """2^20 sequences, in closed form: pages of 4, lengths 0 to 7, one token each, every eighth ends."""
    n, ps = 1 << 20, 4
    s = torch.arange(n, device="cuda")
    had = (s % 8).int()
    new = torch.where(s % 8 == 7, -1, 1).int()
    table = torch.stack([2 * s, 2 * s + 1], 1).int()
    n_pages = 4 * n
    free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    free[:n] = (2 * n + s).int()
    flags, n_free, n_out = ints([0]), ints([n]), ints([0])
    lens, cu = torch.empty_like(had), torch.empty(n + 1, dtype=torch.int32, device="cuda")
    total = n
    slots = torch.empty(total, dtype=torch.int32, device="cuda")
    paging = H.make_paging(table, n_pages, ps, total)
    H.hash_attn_plan_pages(paging, new, had, lens, cu, table, free, n_free, n_out, slots=slots, dev_flags=flags)
    assert flags.item() == 0
    ends, takes = new < 0, (had == 0) | (had == 4)
    assert torch.equal(lens, torch.where(ends, 0, had + 1))
    assert torch.equal(cu[1:].long(), torch.cumsum((~ends).long(), 0)) and cu[0] == 0
    back = torch.stack([2 * s[ends], 2 * s[ends] + 1], 1).flatten()
    assert torch.equal(free[n:n + n // 4].long(), back) and n_out.item() == n
    top, k = n + n // 4, torch.cumsum(takes.long(), 0) - 1
    got = free.long()[top - 1 - k]
    assert torch.equal(table[:, 0].long(), torch.where(had == 0, got, 2 * s))
    assert torch.equal(table[:, 1].long(), torch.where(had == 4, got, 2 * s + 1))
    place = table.long()[s, (had // ps).long()] * ps + had % ps
    assert torch.equal(slots[:n - n // 8].long(), place[~ends]) and (slots[n - n // 8:] == -1).all()


def test_plans_of_a_captured_graph(H):
    """Steps of a serving loop: one captured call, new lengths written between its replays."""
    ps, n = 4, 5
    p = Plan([1] * n, [0] * n, ps, 60, total=40, cols=12)
    p.put(H, in_place=True)
    t = p.t
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        p.run(H)
    r = random.Random(5)
    state = dict(lens=p.had, table=p.table, free=p.free, n_free=p.n_free)
    for step in range(12):
        new = [r.choice([-1, 0, 1, 1, 1, 7, 11]) for _ in range(n)]
        want = SO.plan_pages(new, state["lens"], state["table"], state["free"], state["n_free"], p.n_pages, ps, p.total)
        t["new"].copy_(ints(new))
        t["flags"].zero_()
        graph.replay()
        got = {k: v.cpu().tolist() for k, v in t.items()}
        assert got["lens"] == want["lens"] and got["table"] == want["table"] and got["cu"] == want["cu"], step
        assert got["n_out"] == [want["n_free"]] and got["free"] == want["free"] and got["flags"] == [want["flags"]], step
        assert got["slots"][:p.total] == want["slots"], step
        state = want


def test_plans_on_two_streams(H):
    a, b = random_plan(7), random_plan(12)
    a.put(H)
    b.put(H)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for p, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                p.run(H)
    torch.cuda.synchronize()
    a.check()
    b.check()


# ---------------------------------------------------------------- several axes

def rand(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


AXES = [
    # new, lens, Hq, Hkv, d, page, rot, axes, in turn, interleaved
    ("one", [1], [1], 1, 1, 128, 16, 128, 3, False, False),
    ("decode", [1] * 5, [1, 16, 17, 300, 64], 8, 2, 128, 16, 128, 3, True, False),
    ("images", [70, 0, 33, 5], [100, 7, 33, 900], 4, 4, 64, 48, 64, 3, False, True),
    ("eight-axes", [40, 9], [40, 1000], 6, 2, 128, 64, 96, 8, True, False),
    ("one-axis", [25], [60], 2, 1, 64, 32, 32, 1, False, False),
    ("part", [3, 21], [3, 500], 7, 1, 128, 80, 16, 2, False, True),
]


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")], ids=str)
@pytest.mark.parametrize("case", AXES, ids=[c[0] for c in AXES])
def test_append_axes(H, case, types):
    _, new, lens, Hq, Hkv, d, ps, rot, n_axes, turn, inter = case
    dt, ct = ({"bf16": torch.bfloat16, "f32": torch.float32}[x] for x in types)
    g = torch.Generator(device="cuda").manual_seed(5)
    T = sum(new)
    qkv = rand(g, T, Hq + 2 * Hkv, d, dtype=dt)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    need = [-(-n // ps) for n in lens]
    n_pages = sum(need) + 1
    perm = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.full((len(new), max(need)), -4, dtype=torch.int32, device="cuda")
    for i, n in enumerate(need):
        table[i, :n] = perm[sum(need[:i]):sum(need[:i]) + n]
    K, V = rand(g, n_pages, Hkv, ps, d, dtype=ct), rand(g, n_pages, ps, Hkv, d, dtype=ct).permute(0, 2, 1, 3)
    K0, V0 = K.clone(), V.clone()
    n = rot // 2
    axis = [p % n_axes for p in range(n)] if turn else [p * n_axes // n for p in range(n)]
    inv = torch.tensor([10000.0 ** (-p / n) for p in range(n)], device="cuda")
    # rows of positions that lie apart; values of any size and sign
    wide = torch.randint(-(1 << 31), (1 << 31) - 1, (n_axes, T + 3), generator=g, device="cuda").int()
    wide[:, ::2] %= 1000
    pos = wide[:, :T]
    q_out = torch.empty(T, Hq, d, dtype=dt, device="cuda")
    flags = ints([0])
    H.hash_attn_append_axes(H.make_tokens(q, k, v, len(new)), H.make_cache(K, V, table), q, k, v, table,
                            ints([sum(new[:i]) for i in range(len(new) + 1)]), ints(lens), pos, q_out, K, V,
                            rope=H.rope_axes(inv, axis, inter), dev_flags=flags)
    assert flags.item() == 0
    f = inv.double().cpu().numpy()
    ph, th = pos.cpu().numpy(), table.cpu().numpy()
    step = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}

    def close(got, x, t, u, what):
        x = x.double().cpu().numpy()
        want = SO.rotate_axes(x, ph[:, t], axis, f, inter)
        # |a| + |b| of each pair; the angle's bound for far positions (of float64's pos * inv_freq, 2^-53 of it)
        mag = np.abs(x).copy()
        i, j = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if inter else (np.arange(n), np.arange(n) + n)
        mag[..., i] = mag[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
        far = np.zeros(x.shape[-1])
        far[i] = far[j] = 2.0 ** -52 * np.abs(ph[axis, t] * f)
        err = np.abs(got.double().cpu().numpy() - want)
        tol = (2.0 ** -21 + far) * mag
        assert np.all(err <= tol + u * (np.abs(want) + tol)), f"{what} row {t}"

    a = 0
    K1, V1 = K0.clone(), V0.clone()
    for s, (m, t) in enumerate(zip(new, lens)):
        for i in range(m):
            r, at = a + i, t - m + i
            pg, row = int(th[s, at // ps]), at % ps
            close(q_out[r], q[r], r, step[dt], "q")
            close(K[pg, :, row], k[r], r, step[ct], "k")
            assert torch.equal(V[pg, :, row], v[r].to(ct))
            K1[pg, :, row], V1[pg, :, row] = K[pg, :, row], V[pg, :, row]
        a += m
    assert torch.equal(K, K1) and torch.equal(V, V1)  # nothing else was written


def test_append_axes_with_equal_positions_is_the_append(H):
    """Axes that all hold a token's place in the sequence: the bits of hash_attn_append, codes too."""
    g = torch.Generator(device="cuda").manual_seed(6)
    new, lens, Hq, Hkv, d, ps = [1, 60, 7], [500, 60, 7], 8, 2, 128, 16
    T = sum(new)
    q, k, v = rand(g, T, Hq, d), rand(g, T, Hkv, d), rand(g, T, Hkv, d)
    W = torch.randn(Hkv, 32, d, generator=g, device="cuda")
    table = torch.randperm(200, generator=g, device="cuda").int()[:96].view(3, 32).contiguous()
    inv = torch.rand(64, generator=g, device="cuda")
    cu, lt = ints([0, 1, 61, 68]), ints(lens)
    pos = torch.cat([torch.arange(t - m, t) for m, t in zip(new, lens)]).int().cuda().expand(3, T).contiguous()
    res = []
    for axes in (False, True):
        K, V, sig = torch.zeros(200, Hkv, ps, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(200, Hkv, ps, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(200, Hkv, ps, dtype=torch.int32, device="cuda")
        q_out = torch.empty_like(q)
        tok, cache = H.make_tokens(q, k, v, 3), H.make_cache(K, V, table, sig)
        if axes:
            H.hash_attn_append_axes(tok, cache, q, k, v, table, cu, lt, pos, q_out, K, V, rope=H.rope_axes(inv, [0, 2, 1, 0] * 16), W=W, k_sig=sig)
        else:
            H.hash_attn_append(tok, cache, q, k, v, table, cu, lt, q_out, K, V, rope=H.rope(inv), W=W, k_sig=sig)
        res.append((q_out, K, V, sig))
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_append_axes_device_errors(H):
    """Bad lengths and stopped sequences are passed by, a bad page too; queries are rotated all the same
    where the place is known."""
    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = rand(g, 3, 2, 64), rand(g, 3, 1, 64), rand(g, 3, 1, 64)
    table, K, V = ints([[0], [1], [9]]), torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    q_out, flags = torch.zeros_like(q), ints([0])
    H.hash_attn_append_axes(H.make_tokens(q, k, v, 3), H.make_cache(K, V, table), q, k, v, table, ints([0, 1, 2, 3]), ints([4, -4, 4]),
                            ints([[0, 0, 0]] * 2), q_out, K, V, rope=H.rope_axes(torch.ones(8, device="cuda"), [0, 1] * 4), dev_flags=flags)
    assert flags.item() == H.HA_DEVERR_SEQLEN | H.HA_DEVERR_INDEX
    assert torch.equal(K[0, 0, 3], k[0, 0]) and torch.equal(V[0, 0, 3], v[0, 0]) and K.count_nonzero() == k[0].count_nonzero()
    assert torch.equal(q_out[0], q[0]) and torch.equal(q_out[2], q[2]) and not q_out[1].any()
