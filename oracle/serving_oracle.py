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
