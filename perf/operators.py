"""Measured cases of the prompt and cache operators: append, prefill, chunk.

append   new tokens' keys and values go into a paged KV cache, the rotary
         position rotation applied to the keys (and to the queries) on the way
prefill  causal attention over whole prompts, packed one after the other,
         with grouped heads; returns the output and its log-normaliser
chunk    attention of each sequence's new tokens (one or many) over its pages
         of the cache, causal from the sequence's end

``run`` computes a case either in plain torch operations (``own`` false) or by
the library's entry points (``own`` true); ``exact`` is the definition in 64
bits, written apart from both.
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
        # one decode step of a full batch: 64 sequences append one token each
        dict(name="append-64x1", op="append", n_seq=64, lo=1, hi=1, ctx_lo=500, ctx_hi=65536, h_q=32, h_kv=8, d=128,
             page=16, rot=128, inter=False, dtype="bf16", order="token", len_seed=1),
        # a few short prompts into a float32 cache, half of each head rotated, neighbouring pairs
        dict(name="append-5-ragged-f32", op="append", n_seq=5, lo=40, hi=400, ctx_lo=0, ctx_hi=900, h_q=8, h_kv=2, d=64,
             page=48, rot=32, inter=True, dtype="f32", order="head", len_seed=2),
        # four long prompts at once
        dict(name="append-4x8192", op="append", n_seq=4, lo=8192, hi=8192, ctx_lo=0, ctx_hi=0, h_q=32, h_kv=8, d=128,
             page=64, rot=128, inter=False, dtype="bf16", order="token", len_seed=3),
        # one short question: latency alone
        dict(name="prefill-77", op="prefill", n_seq=1, lo=77, hi=77, h_q=8, h_kv=2, d=64, out="bf16", len_seed=4),
        # a batch of prompts of mixed lengths
        dict(name="prefill-24-ragged", op="prefill", n_seq=24, lo=33, hi=2500, h_q=32, h_kv=8, d=128, out="bf16",
             len_seed=5),
        # a document
        dict(name="prefill-16384", op="prefill", n_seq=1, lo=16384, hi=16384, h_q=32, h_kv=8, d=128, out="bf16",
             len_seed=6),
        # float32 results (segments that are merged later), three heads per KV head
        dict(name="prefill-3-g3-f32", op="prefill", n_seq=3, lo=700, hi=1900, h_q=12, h_kv=4, d=64, out="f32",
             len_seed=7),
        # one sequence's next token: latency alone
        dict(name="decode-1x700", op="chunk", n_seq=1, lo=1, hi=1, ctx_lo=699, ctx_hi=699, h_q=8, h_kv=2, d=128,
             page=16, order="token", out="f32", len_seed=8),
        # a decode step of a full batch, ragged contexts
        dict(name="decode-64-ragged", op="chunk", n_seq=64, lo=1, hi=1, ctx_lo=1000, ctx_hi=16000, h_q=32, h_kv=8,
             d=128, page=16, order="token", out="bf16", len_seed=9),
        # one long document, its next token, result to be merged
        dict(name="decode-1x131072", op="chunk", n_seq=1, lo=1, hi=1, ctx_lo=131071, ctx_hi=131071, h_q=32, h_kv=8,
             d=128, page=64, order="head", out="f32", len_seed=10),
        # the next piece of four long prompts
        dict(name="chunk-4x512-32k", op="chunk", n_seq=4, lo=512, hi=512, ctx_lo=20000, ctx_hi=32000, h_q=32, h_kv=8,
             d=128, page=128, order="token", out="bf16", len_seed=11),
        # a serving batch: sequences that decode beside sequences that read their prompts
        dict(name="chunk-48-mixed", op="chunk", n_seq=48, lo=1, hi=256, ctx_lo=0, ctx_hi=4000, h_q=16, h_kv=2, d=64,
             page=32, order="head", out="bf16", len_seed=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["append", "prefill", "prefill", "chunk", "chunk"])
    while True:
        h_kv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 16])
        c = dict(op=op, n_seq=_log_int(rng, 1, 64), h_q=h_kv * G, h_kv=h_kv, d=rng.choice([64, 128]),
                 len_seed=rng.randrange(1 << 30))
        if op != "prefill":
            c.update(page=rng.choice([16, 16, 32, 48, 64, 80, 128, 256]), order=rng.choice(["token", "head"]))
        if op == "append":
            c["hi"] = rng.choice([1, _log_int(rng, 2, 8192)])
            c["lo"] = rng.randint(1, c["hi"])
            c["ctx_hi"] = _log_int(rng, 1, 131072)
            c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
            c["rot"] = rng.choice([c["d"], c["d"], c["d"] // 2, 16])
            c["inter"] = rng.random() < 0.3
            c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
            size = 2 if c["dtype"] == "bf16" else 4
            if c["n_seq"] * c["hi"] * (c["h_q"] + 2 * h_kv) * c["d"] * size <= 32768 * 48 * 128 * 2:
                return c
        elif op == "prefill":
            c["hi"] = _log_int(rng, 1, 16384)
            c["lo"] = rng.randint(1, c["hi"])
            c["out"] = rng.choice(["bf16", "bf16", "f32"])
            if c["n_seq"] * c["hi"] ** 2 * max(c["h_q"] * c["d"], 256 * G) <= 16384 ** 2 * 32 * 128:
                return c
        else:
            c["hi"] = rng.choice([1, 1, _log_int(rng, 2, 1024)])
            c["lo"] = 1
            c["ctx_hi"] = _log_int(rng, 1, 131072)
            c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
            c["out"] = rng.choice(["bf16", "bf16", "f32"])
            keys = c["n_seq"] * (c["ctx_hi"] + c["hi"])
            if (keys * h_kv * c["d"] <= 64 * 16000 * 8 * 128 and
                    keys * c["hi"] * c["h_q"] * c["d"] <= 4 * 32512 * 512 * 32 * 128):
                return c


def _lens(case):
    """New tokens and total lengths of the case's sequences."""
    r = random.Random(case["len_seed"])
    new = [r.randint(case["lo"], case["hi"]) for _ in range(case["n_seq"])]
    if case["op"] == "chunk" and case["hi"] > 1 and case["lo"] == 1:  # most sequences of a serving batch decode
        new = [n if r.random() < 0.3 else 1 for n in new]
    if case["op"] == "prefill":
        return new, list(new)
    return new, [n + r.randint(case["ctx_lo"], case["ctx_hi"]) for n in new]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, tot = _lens(case)
    T, n, d, hq, hkv = sum(new), case["n_seq"], case["d"], case["h_q"], case["h_kv"]
    dt = _F[case.get("dtype", "bf16")]

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    s = dict(case)
    s["q"] = rand(T, hq, d)
    s["cu"] = torch.tensor([sum(new[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
    s["max_new"], s["max_len"] = max(new), max(tot)
    if case["op"] != "chunk":
        s["k"], s["v"] = rand(T, hkv, d), rand(T, hkv, d)
    if case["op"] != "prefill":
        s["lens"] = torch.tensor(tot, dtype=torch.int32, device="cuda")
        ps = case["page"]
        # an append needs pages for the new tokens only (the earlier ones are someone else's reads)
        first = [(t - m) // ps if case["op"] == "append" else 0 for m, t in zip(new, tot)]
        pages = [(t + ps - 1) // ps - f for t, f in zip(tot, first)]
        n_pages = sum(pages) + 3
        perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(n, max((t + ps - 1) // ps for t in tot), dtype=torch.int32, device="cuda")
        at = 0
        for i in range(n):
            table[i, first[i]:first[i] + pages[i]] = perm[at:at + pages[i]]
            at += pages[i]
        s["table"] = table
        if case["order"] == "token":  # [page, token, head, d] in memory
            s["K"] = rand(n_pages, ps, hkv, d).permute(0, 2, 1, 3)
            s["V"] = rand(n_pages, ps, hkv, d).permute(0, 2, 1, 3)
        else:                         # [page, head, token, d]
            s["K"], s["V"] = rand(n_pages, hkv, ps, d), rand(n_pages, hkv, ps, d)
    if case["op"] == "append":
        r = case["rot"]
        s["inv_freq"] = torch.tensor([500000.0 ** (-2.0 * i / r) for i in range(r // 2)], device="cuda")
    if own:
        from long_context_sparse_score_gb300 import hashattn as H
        if case["op"] == "append":
            s["tokens"] = H.make_tokens(s["q"], s["k"], s["v"], n)
            s["rope"] = H.rope(s["inv_freq"], interleaved=case["inter"])
        else:
            s["tokens"] = H.make_tokens(s["q"], s.get("k"), s.get("v"), n, h_kv=hkv, out_dtype=_F[case["out"]])
            s["ws"] = torch.empty(H.hash_attn_packed_workspace_size(s["tokens"]), dtype=torch.uint8, device="cuda")
            H.hash_attn_workspace_init(s["ws"])
        if case["op"] != "prefill":
            s["cache"] = H.make_cache(s["K"], s["V"], s["table"])
    return s


# ---------------------------------------------------------------- the library's calls

def _own(s):
    from long_context_sparse_score_gb300 import hashattn as H
    q = s["q"]
    if s["op"] == "append":
        q_out = torch.empty_like(q)
        H.hash_attn_append(s["tokens"], s["cache"], q, s["k"], s["v"], s["table"], s["cu"], s["lens"], q_out, s["K"],
                           s["V"], rope=s["rope"])
        return {"q": q_out, "K": s["K"], "V": s["V"]}
    out = torch.empty(q.shape, dtype=_F[s["out"]], device="cuda")
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    if s["op"] == "prefill":
        H.hash_attn_prefill(s["tokens"], q, s["k"], s["v"], s["cu"], out, lse, workspace=s["ws"])
    else:
        H.hash_attn_chunk(s["tokens"], s["cache"], q, s["K"], s["V"], s["table"], s["cu"], s["lens"], out, lse,
                          workspace=s["ws"])
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------- the plain form

def _places(s):
    """Sequence, index among the new tokens and position of every packed token."""
    t = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(s["cu"].long(), t, right=True) - 1
    i = t - s["cu"].long()[seq]
    return seq, i


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
    pos = s["lens"].long()[seq] - new[seq] + i
    angle = pos.double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _rotate(s["q"], cos, sin, s["rot"], s["inter"]).to(s["q"].dtype)
    k = _rotate(s["k"], cos, sin, s["rot"], s["inter"]).to(s["k"].dtype)
    page = s["table"].long()[seq, pos // s["page"]]
    s["K"].permute(0, 2, 1, 3)[page, pos % s["page"]] = k
    s["V"].permute(0, 2, 1, 3)[page, pos % s["page"]] = s["v"]
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
    sees = kj <= (lens - new)[:, None, None] + qi[:, None]  # [n, mq, mk]
    sees &= kj < lens[:, None, None]
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
        z = z.view(n, h1 - h0, G, mq, mk).masked_fill(~sees[:, None, None], -math.inf)
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
    return _plain_append(state) if state["op"] == "append" else _plain_attention(state)


# ---------------------------------------------------------------- cost and definition

def work(case):
    """Each input once, each output once; the products of the pairs that the mask leaves."""
    new, tot = _lens(case)
    T, d, hq, hkv = sum(new), case["d"], case["h_q"], case["h_kv"]
    if case["op"] == "append":
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * T * (hq + 2 * hkv) * d * size, "flops": 3 * T * (hq + hkv) * case["rot"]}
    keys = sum(tot)
    pairs = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(new, tot))
    out = 2 if case["out"] == "bf16" else 4
    return {"bytes": T * hq * d * (2 + out) + T * hq * 4 + keys * hkv * d * 4, "flops": 4 * pairs * hq * d}


def exact(case, seed):
    new, tot = _lens(case)
    if case["op"] != "append" and 4 * case["h_q"] * case["d"] * sum(n * t for n, t in zip(new, tot)) > 6e12:
        return None  # over about 20 seconds in 64 bits
    s = prepare(case, seed)
    T, d, hq, hkv = sum(new), case["d"], case["h_q"], case["h_kv"]
    starts = [sum(new[:i]) for i in range(len(new))]
    if case["op"] == "append":
        res = {x: s[x].double() for x in ("q", "K", "V")}
        w = torch.tensor([float(f) for f in s["inv_freq"].tolist()], dtype=torch.float64, device="cuda")
        ps, rot = case["page"], case["rot"]
        for i, (a, n, t) in enumerate(zip(starts, new, tot)):
            p = torch.arange(t - n, t, device="cuda", dtype=torch.float64)
            c = torch.polar(torch.ones(n, 1, rot // 2, dtype=torch.float64, device="cuda"), p[:, None, None] * w)

            def turn(x):  # each pair of dims is a complex number, turned by the token's angle
                x = x[a:a + n].double()
                y, head = x.clone(), x[..., :rot]
                if case["inter"]:
                    y[..., :rot] = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous()) * c).flatten(-2)
                else:
                    z = torch.complex(head[..., : rot // 2].contiguous(), head[..., rot // 2 :].contiguous()) * c
                    y[..., :rot] = torch.cat([z.real, z.imag], -1)
                return y
            res["q"][a:a + n] = turn(s["q"])
            k, v = turn(s["k"]), s["v"][a:a + n].double()
            at = torch.arange(t - n, t, device="cuda")
            pg, row = s["table"][i].long()[at // ps], at % ps
            for h in range(hkv):
                res["K"][pg, h, row], res["V"][pg, h, row] = k[:, h], v[:, h]
        return res
    out = torch.zeros(T, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device="cuda")
    G = hq // hkv
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
                x = s["q"][a + r0:a + r1, h * G:(h + 1) * G].double()
                z = torch.einsum("rgd,kd->rgk", x, k) * d ** -0.5
                z.masked_fill_((at[None, :] > (t - n + torch.arange(r0, r1, device="cuda"))[:, None])[:, None], -math.inf)
                l = torch.logsumexp(z, -1)
                out[a + r0:a + r1, h * G:(h + 1) * G] = torch.einsum("rgk,kd->rgd", torch.exp(z - l[..., None]), v)
                lse[a + r0:a + r1, h * G:(h + 1) * G] = l
    return {"out": out, "lse": lse}
