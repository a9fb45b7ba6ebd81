"""Measured cases of what surrounds the paged cache: its page plan, the append with several
position axes, and attention with capped, biased and masked scores.

plan     page tables, row bounds, lengths and slots of a serving step from the sequences'
         new lengths; ended sequences give their pages back
append   new tokens go into the paged cache, queries and keys rotated by positions of
         several axes (time, height, width)
prefill  attention over packed prompts, and
chunk    attention of new tokens over their pages, with a tanh cap on the scores, a bias by
         distance, a sliding window, a prefix that every token sees, and keys that begin
         inside the sequence

``run`` computes a case either in plain torch operations (``own`` false) or by the
library's entry points (``own`` true); ``exact`` is the definition in 64 bits, written
apart from both.
"""

import math
import random

import torch

own = False

_F = {"bf16": torch.bfloat16, "f32": torch.float32}
_SCORE_BYTES = 8 << 30  # float32 scores that the plain form holds at a time


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a full batch: a token each, a page for every sixteenth sequence
        dict(name="plan-64x1", op="plan", n_seq=64, hi=1, prompts=0.0, ends=0.0, ctx_hi=65536, page=16, short=False, len_seed=1),
        # a few long prompts are taken in
        dict(name="plan-6-prompts", op="plan", n_seq=6, hi=16384, prompts=1.0, ends=0.0, ctx_hi=1, page=64, short=False, len_seed=2),
        # a large serving batch: most decode, some read their prompts, some end
        dict(name="plan-3000-mixed", op="plan", n_seq=3000, hi=500, prompts=0.1, ends=0.05, ctx_hi=8000, page=16, short=False, len_seed=3),
        # one decode step of sequences that began with images
        dict(name="axes-32x1", op="append", n_seq=32, lo=1, hi=1, ctx_hi=20000, h_q=32, h_kv=8, d=128, page=16, rot=128, inter=False,
             dtype="bf16", order="token", axes=3, blocks=True, len_seed=4),
        # images and their questions, in turn: axes taken in turn by the pairs
        dict(name="axes-6-images", op="append", n_seq=6, lo=1000, hi=6000, ctx_hi=3000, h_q=32, h_kv=8, d=128, page=64, rot=128,
             inter=False, dtype="bf16", order="token", axes=3, blocks=False, len_seed=5),
        # a small float32 model, neighbouring pairs, half of each head rotated, two axes
        dict(name="axes-5-ragged-f32", op="append", n_seq=5, lo=30, hi=300, ctx_hi=700, h_q=8, h_kv=2, d=64, page=48, rot=32, inter=True,
             dtype="f32", order="head", axes=2, blocks=True, len_seed=6),
        # one sequence's next token, capped scores: latency alone
        dict(name="decode-1x700-cap", op="chunk", n_seq=1, lo=1, hi=1, ctx_lo=699, ctx_hi=699, h_q=8, h_kv=2, d=128, page=16, order="token",
             out="f32", cap=50.0, bias=False, window=0, prefix=False, first=False, len_seed=7),
        # a decode step of a full batch in a layer that looks 4,096 tokens back
        dict(name="decode-64-cap-window", op="chunk", n_seq=64, lo=1, hi=1, ctx_lo=1000, ctx_hi=16000, h_q=32, h_kv=8, d=128, page=16,
             order="token", out="bf16", cap=50.0, bias=False, window=4096, prefix=False, first=False, len_seed=8),
        # a batch of prompts of mixed lengths, bias by distance
        dict(name="prefill-24-bias", op="prefill", n_seq=24, lo=33, hi=2500, h_q=32, h_kv=8, d=128, out="bf16", cap=0.0, bias=True, window=0,
             prefix=False, first=False, len_seed=9),
        # a document, capped scores
        dict(name="prefill-16384-cap", op="prefill", n_seq=1, lo=16384, hi=16384, h_q=32, h_kv=8, d=128, out="bf16", cap=50.0, bias=False,
             window=0, prefix=False, first=False, len_seed=10),
        # prompts that begin with a part which sees itself both ways (an image, an instruction)
        dict(name="prefill-5-prefix-f32", op="prefill", n_seq=5, lo=300, hi=1500, h_q=12, h_kv=4, d=64, out="f32", cap=30.0, bias=False,
             window=0, prefix=True, first=False, len_seed=11),
        # a serving batch whose sequences hold several documents and see the last one
        dict(name="chunk-48-documents", op="chunk", n_seq=48, lo=1, hi=256, ctx_lo=0, ctx_hi=4000, h_q=16, h_kv=2, d=64, page=32, order="head",
             out="bf16", cap=0.0, bias=True, window=1000, prefix=False, first=True, len_seed=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["plan", "append", "prefill", "prefill", "chunk", "chunk"])
    while True:
        h_kv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 16])
        c = dict(op=op, n_seq=_log_int(rng, 1, 64), len_seed=rng.randrange(1 << 30))
        if op == "plan":
            c.update(n_seq=_log_int(rng, 1, 3000), hi=rng.choice([1, _log_int(rng, 2, 16384)]), prompts=rng.choice([0.0, 0.1, 0.5, 1.0]),
                     ends=rng.choice([0.0, 0.0, 0.05, 0.5]), ctx_hi=_log_int(rng, 1, 65536), page=rng.choice([1, 16, 16, 32, 48, 64, 80, 128, 256]),
                     short=rng.random() < 0.15)
            if c["n_seq"] * c["hi"] <= 3000 * 500 and c["n_seq"] * (c["hi"] + c["ctx_hi"]) <= 3000 * 8500 * c["page"] // 16:
                return c
            continue
        c.update(h_q=h_kv * G, h_kv=h_kv, d=rng.choice([64, 128]))
        if op != "prefill":
            c.update(page=rng.choice([16, 16, 32, 48, 64, 80, 128, 256]), order=rng.choice(["token", "head"]))
        if op == "append":
            c["hi"] = rng.choice([1, _log_int(rng, 2, 8192)])
            c["lo"] = rng.randint(1, c["hi"])
            c["ctx_hi"] = _log_int(rng, 1, 131072)
            c["rot"] = rng.choice([c["d"], c["d"], c["d"] // 2, 16])
            c["inter"] = rng.random() < 0.3
            c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
            c["axes"] = rng.choice([1, 2, 3, 3, 4])
            c["blocks"] = rng.random() < 0.6
            size = 2 if c["dtype"] == "bf16" else 4
            if c["n_seq"] * c["hi"] * (c["h_q"] + 2 * h_kv) * c["d"] * size <= 36000 * 48 * 128 * 2:
                return c
            continue
        c["out"] = rng.choice(["bf16", "bf16", "f32"])
        c["cap"] = rng.choice([0.0, 30.0, 50.0])
        c["bias"] = rng.random() < 0.4
        c["window"] = rng.choice([0, 0, _log_int(rng, 1, 8192)])
        c["prefix"] = rng.random() < 0.3
        c["first"] = rng.random() < 0.3
        if op == "prefill":
            c["hi"] = _log_int(rng, 1, 16384)
            c["lo"] = rng.randint(1, c["hi"])
            if c["n_seq"] * c["hi"] ** 2 * max(c["h_q"] * c["d"], 256 * G) <= 16384 ** 2 * 32 * 128 // (2 if c["prefix"] else 1):
                return c
        else:
            c["hi"] = rng.choice([1, 1, _log_int(rng, 2, 1024)])
            c["lo"] = 1
            c["ctx_hi"] = _log_int(rng, 1, 131072)
            c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
            keys = c["n_seq"] * (c["ctx_hi"] + c["hi"])
            if keys * h_kv * c["d"] <= 64 * 16000 * 8 * 128 and keys * c["hi"] * c["h_q"] * c["d"] <= 16384 ** 2 * 16 * 128:
                return c


def _lens(case):
    """New tokens and total lengths of the case's sequences (plan: -1 new tokens ends one, its total is what it had)."""
    r = random.Random(case["len_seed"])
    if case["op"] == "plan":
        had = [r.randint(0 if case["prompts"] else 1, case["ctx_hi"]) for _ in range(case["n_seq"])]
        kind = [r.random() for _ in had]
        new = [-1 if k < case["ends"] else (r.randint(1, case["hi"]) if r.random() < case["prompts"] else 1) for k in kind]
        return new, [h + max(n, 0) for h, n in zip(had, new)]
    new = [r.randint(case["lo"], case["hi"]) for _ in range(case["n_seq"])]
    if case["op"] == "chunk" and case["hi"] > 1:  # most sequences of a serving batch decode
        new = [n if r.random() < 0.3 else 1 for n in new]
    if case["op"] == "prefill":
        return new, list(new)
    return new, [n + r.randint(case.get("ctx_lo", 0), case["ctx_hi"]) for n in new]


def _bounds(case):
    """First key and prefix of the sequences: numbers that go by the case alone."""
    r = random.Random(case["len_seed"] + 1)
    new, tot = _lens(case)
    first = [r.randint(0, max(0, t - n) // 2) if case["op"] == "chunk" else r.randint(0, t // 4) for n, t in zip(new, tot)]
    prefix = [r.randint(0, max(1, t // 2)) for t in tot]
    return first if case["first"] else None, prefix if case["prefix"] else None


def _axis(case):
    """The axis of every pair: one block of pairs after the other (the first the smaller), or in turn."""
    n, a = case["rot"] // 2, case["axes"]
    return [min(a - 1, p * (a + 1) // (n + 1)) if case["blocks"] else p % a for p in range(n)]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, tot = _lens(case)
    n, s = case["n_seq"], dict(case)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["op"] == "plan":
        ps = case["page"]
        had = [t - max(m, 0) for m, t in zip(new, tot)]
        held = [(h + ps - 1) // ps for h in had]
        fresh = sum((t + ps - 1) // ps - p for t, p in zip(tot, held))
        spare = fresh // 2 if case["short"] else fresh + 5
        s["n_pages"] = sum(held) + spare
        perm = torch.randperm(s["n_pages"], generator=g, device="cuda").to(torch.int32)
        s["pages"] = max(1, max((t + ps - 1) // ps for t in tot)) + 1
        cols = torch.arange(s["pages"], device="cuda")
        counts = ints(held).long()
        at = torch.cumsum(counts, 0) - counts
        table = perm[(at[:, None] + cols).clamp(max=s["n_pages"] - 1)]
        s["table"] = torch.where(cols < counts[:, None], table, torch.full_like(table, -1)).contiguous()
        s["free"] = torch.full((s["n_pages"],), -1, dtype=torch.int32, device="cuda")
        s["free"][:spare] = perm[sum(held):]
        s["n_free"], s["new"], s["had"] = ints([spare]), ints(new), ints(had)
        s["total"] = sum(max(m, 0) for m in new) + 3  # rows that the packed buffers have room for
        s["spare"] = spare
        if own:
            from long_context_sparse_score_gb300 import hashattn as H
            s["paging"] = H.make_paging(s["table"], s["n_pages"], ps, s["total"])
            s["lens"], s["cu"], s["slots"], s["n_free_out"] = (
                torch.empty(m, dtype=torch.int32, device="cuda") for m in (n, n + 1, s["total"], 1))
        return s

    T, d, hq, hkv = sum(new), case["d"], case["h_q"], case["h_kv"]
    dt = _F[case.get("dtype", "bf16")]

    def rand(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dt)

    # scores of a trained layer spread over several units (three here), not one
    s["q"] = rand(T, hq, d, scale=1.0 if case["op"] == "append" else 3.0)
    s["cu"] = ints([sum(new[:i]) for i in range(n + 1)])
    s["max_new"], s["max_len"] = max(new), max(tot)
    if case["op"] != "chunk":
        s["k"], s["v"] = rand(T, hkv, d), rand(T, hkv, d)
    if case["op"] != "prefill":
        s["lens"] = ints(tot)
        ps = case["page"]
        # an append needs pages for the new tokens only (the earlier ones are someone else's reads)
        begin = [(t - m) // ps if case["op"] == "append" else 0 for m, t in zip(new, tot)]
        held = [(t + ps - 1) // ps - f for t, f in zip(tot, begin)]
        n_pages = sum(held) + 3
        perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(n, max((t + ps - 1) // ps for t in tot), dtype=torch.int32, device="cuda")
        at = 0
        for i in range(n):
            table[i, begin[i]:begin[i] + held[i]] = perm[at:at + held[i]]
            at += held[i]
        s["table"] = table
        if case["order"] == "token":  # [page, token, head, d] in memory
            s["K"] = rand(n_pages, ps, hkv, d).permute(0, 2, 1, 3)
            s["V"] = rand(n_pages, ps, hkv, d).permute(0, 2, 1, 3)
        else:                         # [page, head, token, d]
            s["K"], s["V"] = rand(n_pages, hkv, ps, d), rand(n_pages, hkv, ps, d)
    if case["op"] == "append":
        r = case["rot"]
        s["inv_freq"] = torch.tensor([500000.0 ** (-2.0 * i / r) for i in range(r // 2)], device="cuda")
        # the first axis goes on from token to token, the others begin anew with every image
        base = torch.repeat_interleave(ints([t - m for m, t in zip(new, tot)]), ints(new).long())
        s["pos"] = torch.stack([base + torch.arange(T, dtype=torch.int32, device="cuda")] +
                               [torch.randint(0, 200, (T,), generator=g, device="cuda", dtype=torch.int32) for _ in range(case["axes"] - 1)])
        s["axis"] = _axis(case)
    else:
        first, prefix = _bounds(case)
        s["first_key"] = None if first is None else ints(first)
        s["prefix_len"] = None if prefix is None else ints(prefix)
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device="cuda") if case["bias"] else None
    if own:
        from long_context_sparse_score_gb300 import hashattn as H
        # a serving loop keeps the buffers of its step's results
        s["out_rows"] = torch.empty(T, hq, d, dtype=_F[case.get("out", case.get("dtype"))], device="cuda")
        s["lse"] = torch.empty(T, hq, device="cuda")
        if case["op"] == "append":
            s["tokens"] = H.make_tokens(s["q"], s["k"], s["v"], n)
            s["rope"] = H.rope_axes(s["inv_freq"], s["axis"], interleaved=case["inter"])
        else:
            s["tokens"] = H.make_tokens(s["q"], s.get("k"), s.get("v"), n, h_kv=hkv, out_dtype=_F[case["out"]])
            s["ws"] = torch.empty(H.hash_attn_packed_workspace_size(s["tokens"]), dtype=torch.uint8, device="cuda")
            H.hash_attn_workspace_init(s["ws"])
            s["opts"] = H.score_opts(softcap=case["cap"], window=case["window"], slopes=s["slopes"], prefix=s["prefix_len"],
                                     first=s["first_key"])
        if case["op"] != "prefill":
            s["cache"] = H.make_cache(s["K"], s["V"], s["table"])
    return s


# ---------------------------------------------------------------- the library's calls

def _own(s):
    from long_context_sparse_score_gb300 import hashattn as H
    if s["op"] == "plan":
        H.hash_attn_plan_pages(s["paging"], s["new"], s["had"], s["lens"], s["cu"], s["table"], s["free"], s["n_free"], s["n_free_out"],
                               slots=s["slots"])
        return {"table": s["table"], "lens": s["lens"], "cu": s["cu"], "slots": s["slots"], "free": s["free"], "n_free": s["n_free_out"]}
    q, out, lse = s["q"], s["out_rows"], s["lse"]
    if s["op"] == "append":
        H.hash_attn_append_axes(s["tokens"], s["cache"], q, s["k"], s["v"], s["table"], s["cu"], s["lens"], s["pos"], out, s["K"], s["V"],
                                rope=s["rope"])
        return {"q": out, "K": s["K"], "V": s["V"]}
    if s["op"] == "prefill":
        H.hash_attn_prefill_ex(s["tokens"], s["opts"], q, s["k"], s["v"], s["cu"], out, lse, workspace=s["ws"])
    else:
        H.hash_attn_chunk_ex(s["tokens"], s["cache"], s["opts"], q, s["K"], s["V"], s["table"], s["cu"], s["lens"], out, lse,
                             workspace=s["ws"])
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------- the plain form

def _plain_plan(s):
    ps, new, had, table = s["page"], s["new"].long(), s["had"].long(), s["table"]
    n, ends = new.shape[0], new < 0
    nq = new.clamp(min=0)
    cu = torch.cat([nq.new_zeros(1), torch.cumsum(nq, 0)])
    lens = torch.where(ends, 0, had + nq)
    p0, p1 = (had + ps - 1) // ps, (lens + ps - 1) // ps
    cols = torch.arange(table.shape[1], device="cuda")
    back = table[ends[:, None] & (cols < p0[:, None])]  # in order of (sequence, page)
    top = s["n_free"].long() + back.shape[0]
    place = torch.arange(s["n_pages"], device="cuda") - s["n_free"].long()
    pushed = (place >= 0) & (place < back.shape[0])
    free = torch.where(pushed, torch.cat([back, back.new_zeros(1)])[place.clamp(0, back.shape[0])], s["free"])
    takes = (p1 - p0).clamp(min=0)
    upto = torch.cumsum(takes, 0)
    goes = (takes == 0) | (upto <= top)  # the others are stopped: their pages have run out
    lens = torch.where(goes, lens, ~had)
    k = top - 1 - ((upto - takes)[:, None] + cols - p0[:, None])
    got = free[k.clamp(0, s["n_pages"] - 1)]
    table = torch.where(goes[:, None] & (cols >= p0[:, None]) & (cols < p1[:, None]), got, table)
    t = torch.arange(s["total"], device="cuda")
    seq = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=n - 1)
    pos = had[seq] + t - cu[seq]
    page = table[seq, (pos // ps).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where((t < cu[-1]) & goes[seq], page * ps + pos % ps, -1)
    left = top - torch.where(upto <= top, upto, 0).amax()
    i = lambda x: x.to(torch.int32)  # noqa: E731
    return {"table": i(table), "lens": i(lens), "cu": i(cu), "slots": i(slots), "free": i(free), "n_free": i(left.reshape(1))}


def _places(s):
    """Sequence and index among the new tokens of every packed token."""
    t = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(s["cu"].long(), t, right=True) - 1
    return seq, t - s["cu"].long()[seq]


def _rotate(x, cos, sin, rot, inter):
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., : rot // 2], x[..., rot // 2 : rot])
    y = x.clone()
    if inter:
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        y[..., : rot // 2], y[..., rot // 2 : rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_append(s):
    seq, i = _places(s)
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    at = s["lens"].long()[seq] - new[seq] + i
    angle = s["pos"].double()[s["axis"]].T * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _rotate(s["q"], cos, sin, s["rot"], s["inter"]).to(s["q"].dtype)
    k = _rotate(s["k"], cos, sin, s["rot"], s["inter"]).to(s["k"].dtype)
    page = s["table"].long()[seq, at // s["page"]]
    s["K"].permute(0, 2, 1, 3)[page, at % s["page"]] = k
    s["V"].permute(0, 2, 1, 3)[page, at % s["page"]] = s["v"]
    return {"q": q, "K": s["K"], "V": s["V"]}


def _plain_attention(s):
    q, cu, n, hkv = s["q"], s["cu"].long(), s["n_seq"], s["h_kv"]
    T, hq, d = q.shape
    G, mq, mk = hq // hkv, s["max_new"], s["max_len"]
    new = cu[1:] - cu[:-1]
    lens = new if s["op"] == "prefill" else s["lens"].long()
    qi, kj = torch.arange(mq, device="cuda"), torch.arange(mk, device="cuda")
    rows = (cu[:-1, None] + qi).clamp(max=T - 1)
    qp = q[rows].float().view(n, mq, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, G * mq, d)
    pos = (lens - new)[:, None, None] + qi[:, None]  # [n, mq, 1]
    sees = kj <= pos
    if s["prefix_len"] is not None:
        sees = sees | (kj < s["prefix_len"][:, None, None])
    if s["window"]:
        sees = sees & (kj > pos - s["window"])
    if s["first_key"] is not None:
        sees = sees & (kj >= s["first_key"][:, None, None])
    sees = sees & (kj < lens[:, None, None])
    far = (pos.float() - kj.float()).abs() if s["slopes"] is not None else None
    if s["op"] == "prefill":
        at = (cu[:-1, None] + kj).clamp(max=T - 1)
        take = lambda X, h0, h1: X[:, h0:h1][at].float().permute(0, 2, 1, 3)  # noqa: E731
        K, V = s["k"], s["v"]
    else:
        page = s["table"].long()[:, kj // s["page"]]
        take = lambda X, h0, h1: X[:, h0:h1].permute(0, 2, 1, 3)[page, kj % s["page"]].float().permute(0, 2, 1, 3)  # noqa: E731
        K, V = s["K"], s["V"]
    step = max(1, min(hkv, _SCORE_BYTES // (4 * n * G * mq * mk)))
    outs, lses = [], []
    for h0 in range(0, hkv, step):  # one pass unless the scores of all heads are too large to hold
        h1 = min(hkv, h0 + step)
        z = qp[:, h0:h1] @ take(K, h0, h1).transpose(-1, -2) / math.sqrt(d)
        if s["cap"]:
            z = s["cap"] * torch.tanh(z / s["cap"])
        z = z.view(n, h1 - h0, G, mq, mk)
        if far is not None:
            z = z - s["slopes"].view(hkv, G)[h0:h1, :, None, None] * far[:, None, None]
        z = z.masked_fill(~sees[:, None, None], -math.inf)
        m = z.amax(-1, keepdim=True)
        e = torch.exp(z - m.masked_fill(m == -math.inf, 0.0))
        l = e.sum(-1, keepdim=True)
        o = (e.view(n, h1 - h0, G * mq, mk) @ take(V, h0, h1)).view(n, h1 - h0, G, mq, d)
        outs.append(o / l.masked_fill(l == 0, 1.0))
        lses.append((m + l.log()).squeeze(-1))
    seq, i = _places(s)
    out = torch.cat(outs, 1).flatten(1, 2)[seq, :, i]   # [T, hq, d]
    lse = torch.cat(lses, 1).flatten(1, 2)[seq, :, i]
    return {"out": out.to(_F[s["out"]]), "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "append": _plain_append}.get(state["op"], _plain_attention)(state)


# ---------------------------------------------------------------- cost and definition

def _seen(case):
    """Pairs of a new token and a key that it sees, and keys that any new token of their sequence sees."""
    new, tot = _lens(case)
    first, prefix = _bounds(case)
    pairs = keys = 0
    for i, (n, t) in enumerate(zip(new, tot)):
        f, p, w = first[i] if first else 0, min(prefix[i], t) if prefix else 0, case["window"] or t + 1
        lo_all, hi_all = t, 0
        for at in range(t - n, t):
            lo, hi = max(f, at + 1 - w, 0), max(at + 1, p)
            if lo < hi:
                pairs += hi - lo
                lo_all, hi_all = min(lo_all, lo), max(hi_all, hi)
        keys += max(0, hi_all - lo_all)
    return pairs, keys


def work(case):
    """Each input once, each output once; the products of the pairs that the mask leaves."""
    new, tot = _lens(case)
    if case["op"] == "plan":
        ps, n = case["page"], case["n_seq"]
        had = [t - max(m, 0) for m, t in zip(new, tot)]
        back = sum((h + ps - 1) // ps for h, m in zip(had, new) if m < 0)
        takes = sum((t + ps - 1) // ps - (h + ps - 1) // ps for h, t in zip(had, tot))
        rows = sum(max(m, 0) for m in new) + 3
        return {"bytes": 4 * (4 * n + 3 + rows + 2 * back + 2 * takes), "flops": 3 * n + 4 * rows}
    T, d, hq, hkv = sum(new), case["d"], case["h_q"], case["h_kv"]
    if case["op"] == "append":
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * T * (hq + 2 * hkv) * d * size, "flops": 3 * T * (hq + hkv) * case["rot"]}
    pairs, keys = _seen(case)
    out = 2 if case["out"] == "bf16" else 4
    return {"bytes": T * hq * d * (2 + out) + T * hq * 4 + keys * hkv * d * 4, "flops": 4 * pairs * hq * d}


def _exact_plan(case, s):
    """The plan, one sequence and one page after the other, in Python's own numbers."""
    ps, new, had = case["page"], s["new"].tolist(), s["had"].tolist()
    table, stack = s["table"].tolist(), s["free"].tolist()
    n_free = s["spare"]
    for i, m in enumerate(new):
        if m < 0:
            for j in range(-(-had[i] // ps)):
                stack[n_free] = table[i][j]
                n_free += 1
    cu, lens, slots, wanted, top = [0], [], [], 0, n_free
    for i, m in enumerate(new):
        cu.append(cu[-1] + max(m, 0))
        if m < 0:
            lens.append(0)
            continue
        fresh = -(-(had[i] + m) // ps) - -(-had[i] // ps)
        wanted += fresh
        if fresh and wanted > top:  # those behind it that need pages are stopped as well
            lens.append(-1 - had[i])
            slots += [-1] * m
            continue
        for pos in range(had[i], had[i] + m):
            if pos % ps == 0:
                n_free -= 1
                table[i][pos // ps] = stack[n_free]
            slots.append(table[i][pos // ps] * ps + pos % ps)
        lens.append(had[i] + m)
    slots += [-1] * (s["total"] - len(slots))
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"table": ints(table), "lens": ints(lens), "cu": ints(cu), "slots": ints(slots), "free": ints(stack), "n_free": ints([n_free])}


def exact(case, seed):
    new, tot = _lens(case)
    if case["op"] in ("prefill", "chunk") and 4 * case["h_q"] * case["d"] * sum(n * t for n, t in zip(new, tot)) > 6e12:
        return None  # over about 20 seconds in 64 bits
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(case, s)
    T, d, hq, hkv = sum(new), case["d"], case["h_q"], case["h_kv"]
    starts = [sum(new[:i]) for i in range(len(new))]
    if case["op"] == "append":
        res = {x: s[x].double() for x in ("q", "K", "V")}
        ps, rot = case["page"], case["rot"]
        # the turn of each pair of dims as a complex number
        turns = torch.stack([s["pos"][a].double() * float(f) for a, f in zip(_axis(case), s["inv_freq"].tolist())], -1)
        turns = torch.polar(torch.ones_like(turns), turns)[:, None]

        def turn(x):
            y, head = x.double().clone(), x.double()[..., :rot]
            if case["inter"]:
                y[..., :rot] = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous()) * turns).flatten(-2)
            else:
                z = torch.complex(head[..., : rot // 2].contiguous(), head[..., rot // 2 :].contiguous()) * turns
                y[..., :rot] = torch.cat([z.real, z.imag], -1)
            return y

        res["q"], k = turn(s["q"]), turn(s["k"])
        for i, (a, n, t) in enumerate(zip(starts, new, tot)):
            at = torch.arange(t - n, t, device="cuda")
            pg, row = s["table"][i].long()[at // ps], at % ps
            for h in range(hkv):
                res["K"][pg, h, row], res["V"][pg, h, row] = k[a:a + n, h], s["v"][a:a + n, h].double()
        return res
    out = torch.zeros(T, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device="cuda")
    G = hq // hkv
    first, prefix = _bounds(case)
    slopes = [2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)]
    if s["slopes"] is not None:
        slopes = s["slopes"].tolist()  # as rounded to 32 bits
    for i, (a, n, t) in enumerate(zip(starts, new, tot)):
        at = torch.arange(t, device="cuda")
        for h in range(hkv):
            if case["op"] == "prefill":
                k, v = s["k"][a:a + t, h].double(), s["v"][a:a + t, h].double()
            else:
                pg, row = s["table"][i].long()[at // case["page"]], at % case["page"]
                k, v = s["K"][pg, h, row].double(), s["V"][pg, h, row].double()
            block = max(1, (1 << 28) // (G * t))
            for r0 in range(0, n, block):
                r1 = min(n, r0 + block)
                p = t - n + torch.arange(r0, r1, device="cuda")[:, None]
                hidden = at >= torch.clamp(p + 1, min=prefix[i] if prefix else 0)
                hidden |= at < (first[i] if first else 0)
                if case["window"]:
                    hidden |= at + case["window"] <= p
                x = s["q"][a + r0:a + r1, h * G:(h + 1) * G].double()
                z = torch.einsum("rgd,kd->rgk", x, k) * d ** -0.5
                if case["cap"]:
                    z = torch.tanh(z / case["cap"]) * case["cap"]
                if case["bias"]:
                    m = torch.tensor(slopes[h * G:(h + 1) * G], dtype=torch.float64, device="cuda")
                    z -= m[None, :, None] * (p - at).abs().double()[:, None]
                z.masked_fill_(hidden[:, None], -math.inf)
                l = torch.logsumexp(z, -1)
                w = torch.exp(z - torch.where(l == -math.inf, 0.0, l)[..., None])
                out[a + r0:a + r1, h * G:(h + 1) * G] = torch.einsum("rgk,kd->rgd", w, v)
                lse[a + r0:a + r1, h * G:(h + 1) * G] = l
    return {"out": out, "lse": lse}
