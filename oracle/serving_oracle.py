"""Plain oracle of what surrounds the packed calls: the page plan, rotations by several axes,
and attention with score options.

TEST INFRASTRUCTURE ONLY (imported by the tests). Written from the definitions, one sequence,
page, row and head at a time, in Python numbers and NumPy float64; it shares no code with the
library.
"""
from __future__ import annotations

import math

import numpy as np

SEQLEN, INDEX, COUNT, STATE, PAGES = 0x1, 0x4, 0x8, 0x20, 0x40


def plan_pages(new, had, table, free, n_free, n_pages, page_size, total):
    """A step's plan: a dict of lens, cu, table, slots, free, n_free and flags."""
    table, free = [list(r) for r in table], list(free)
    max_len = len(table[0]) * page_size
    flags, lens, cu, slots = 0, [], [0], []
    if not 0 <= n_free <= n_pages:
        flags |= STATE
        n_free = min(max(n_free, 0), n_pages)
    kept = n_free
    for m, h in zip(new, had):  # lengths that cannot be
        if m >= 0 and (h < 0 and m > 0 or h >= 0 and h + m > max_len):
            flags |= SEQLEN
    over = sum(max(m, 0) for m in new) > total
    for i, (m, h) in enumerate(zip(new, had)):
        if m < 0:
            tokens = min(-1 - h if h < 0 else h, max_len)
            for j in range(-(-tokens // page_size)):
                page = table[i][j]
                if not 0 <= page < n_pages:
                    flags |= INDEX
                elif not over:
                    if n_free < n_pages:
                        free[n_free] = page
                        n_free += 1
                    else:
                        flags |= STATE
    if over:
        return dict(lens=list(had), cu=[0] * (len(new) + 1), table=table, slots=[-1] * total, free=free, n_free=kept,
                    flags=flags | COUNT)
    room, wanted, left = n_free, 0, n_free
    for i, (m, h) in enumerate(zip(new, had)):
        cu.append(cu[-1] + max(m, 0))
        if m < 0:
            lens.append(0)
            continue
        if h < 0 or h + m > max_len:
            lens.append(-1 - h if 0 <= h <= max_len else h)
            slots += [-1] * m
            continue
        held = -(-h // page_size)
        fresh = -(-(h + m) // page_size) - held
        wanted += fresh
        if fresh and wanted > room:
            flags |= PAGES
            lens.append(-1 - h)
            slots += [-1] * m
            continue
        for j in range(held, held + fresh):
            left -= 1
            table[i][j] = free[left] if 0 <= free[left] < n_pages else -1
            if table[i][j] < 0:
                flags |= INDEX
        for pos in range(h, h + m):
            page = table[i][pos // page_size]
            slots.append(page * page_size + pos % page_size if 0 <= page < n_pages else -1)
        lens.append(h + m)
    return dict(lens=lens, cu=cu, table=table, slots=slots + [-1] * (total - len(slots)), free=free, n_free=left, flags=flags)


def rotate_axes(x, positions, axis, inv_freq, interleaved=False):
    """x [..., d] of a token with these positions (one for each axis), rotated in its first 2 len(axis) dims."""
    x = np.array(x, dtype=np.float64)
    n = len(axis)
    for p in range(n):
        a = float(positions[axis[p]]) * float(inv_freq[p])
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + n)
        u, v = x[..., i].copy(), x[..., j].copy()
        x[..., i], x[..., j] = u * math.cos(a) - v * math.sin(a), u * math.sin(a) + v * math.cos(a)
    return x


def attention(q, K, V, *, scale=None, cap=0.0, slope=0.0, window=0, prefix=0, first=0):
    """New tokens q [nq, d] (the last of the sequence) over keys K, V [nk, d] with score options: (out [nq, d],
    lse [nq], tol [nq, d], tol_lse [nq], mag [nq, d]). mag = sum_j p_j |v_j|; tol bounds the error of a
    computation in float32 (see below), before weights or results are rounded to fewer bits.

    A score z sums d exact products (d steps of 2^-23 relative to sum_k |q_k K_jk| scale, if the adder
    truncates); cap tanh(z / cap) costs 2^-20 cap (the polynomial 8e-7, its value less the softmax's
    reference 2^-23 of up to 3 cap more); the bias, formed from the distance of up to 128 columns away, 2^-21 of
    itself; the exponential 2^-22 and the sums 2^-23 a term. A weight's relative error e_j moves
    out by p_j e_j (|v_j| + |out|) and lse by p_j e_j."""
    q, K, V = (np.asarray(x, dtype=np.float64) for x in (q, K, V))
    (nq, d), nk = q.shape, K.shape[0]
    scale = 1 / math.sqrt(d) if scale is None else scale
    out, tol, mag = np.zeros((nq, d)), np.zeros((nq, d)), np.zeros((nq, d))
    lse, tol_lse = np.full(nq, -math.inf), np.zeros(nq)
    for i in range(nq):
        pos = nk - nq + i
        lo = max(0, first, pos - window + 1 if window else 0)
        hi = min(nk, max(pos + 1, prefix))
        if lo >= hi:
            continue
        k, v = K[lo:hi], V[lo:hi]
        z = k @ q[i] * scale
        if cap:
            z = cap * np.tanh(z / cap)
        dist = np.abs(pos - np.arange(lo, hi))
        z = z - slope * dist
        top = z.max()
        w = np.exp(z - top)
        e = 2.0 ** -23 * ((d + 4) * scale * (np.abs(k) @ np.abs(q[i])) + (hi - lo) + 16) + 2.0 ** -20 * cap + 2.0 ** -21 * abs(slope) * (dist + 128)
        p = w / w.sum()
        out[i], mag[i] = p @ v, p @ np.abs(v)
        lse[i] = top + math.log(w.sum())
        tol_lse[i] = p @ e + 2.0 ** -22 * (1 + abs(lse[i]) + 2 * cap)
        tol[i] = (p * e) @ np.abs(v) + (p @ e) * mag[i]
    return out, lse, tol, tol_lse, mag
