"""A serving step's bookkeeping, ragged rotary append and e4m3 rounding (oracle; test
infrastructure).

Plain loops over requests, tokens and pairs, in the order the definitions are stated in:
requests are admitted one after the other, pages are taken from the end of a Python list.
It shares no code with the CUDA library.
"""

import numpy as np


def pages_of(tokens, page_size):
    return -(-tokens // page_size)


def plan_step(cached, new, table, free, page_size, capacity, num_pages):
    """``table`` is a list of lists, ``free`` the free pages (a stack).  Returns a dict; the
    arguments are left as they are."""
    table = [list(r) for r in table]
    free = list(free)
    width = len(table[0]) * page_size if table else 0
    cu, seqlens, slots, positions, refused, bad = [0], [], [], [], [], []
    open_ = True
    for b, (c, n) in enumerate(zip(cached, new)):
        if not 0 <= c <= width or n < 0 or c + n > width:
            bad.append(b)
            cu.append(cu[-1])
            seqlens.append(c)
            continue
        need = pages_of(c + n, page_size) - pages_of(c, page_size)
        if n and open_ and (need > len(free) or len(slots) + n > capacity):
            open_ = False
        if not open_ and n:
            refused.append(b)
            n = need = 0
        for j in range(need):
            table[b][pages_of(c, page_size) + j] = free.pop()
        for pos in range(c, c + n):
            page = table[b][pos // page_size]
            ok = 0 <= page < num_pages
            slots.append(page * page_size + pos % page_size if ok else -1)
            positions.append(pos)
        cu.append(len(slots))
        seqlens.append(c + n)
    pad = capacity - len(slots)
    return dict(cu_seqlens_q=cu, seqlens_k=seqlens, slot_mapping=slots + [-1] * pad,
                positions=positions + [0] * pad, block_table=table, free=free, refused=refused,
                bad=bad)


def release_pages(cached, keep, table, free, page_size, num_pages):
    """Returns (free pages, kept lengths, refused requests, bad requests)."""
    free, out, refused, bad = list(free), [], [], []
    pushed = len(free)  # entries outside the pool count until the list is closed up
    open_ = True
    for b, (c, k) in enumerate(zip(cached, keep)):
        k = min(k, c)
        if not 0 <= c <= len(table[b]) * page_size or k < 0:
            bad.append(b)
            out.append(c)
            continue
        cols = range(pages_of(k, page_size), pages_of(c, page_size))
        if len(cols) and open_ and pushed + len(cols) > num_pages:
            open_ = False
        if not open_:
            if len(cols):
                refused.append(b)
            out.append(c)
            continue
        pushed += len(cols)
        free += [table[b][j] for j in cols if 0 <= table[b][j] < num_pages]
        out.append(k)
    return free, out, refused, bad


def _e4m3_values():
    """The 127 finite values >= 0, in the order of their codes."""
    return np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
                     for e in range(16) for m in range(8)][:-1])


def e4m3(x):
    """The nearest e4m3 value (ties to the even code), saturating; NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    v = _e4m3_values()
    mid = (v[1:] + v[:-1]) / 2
    a = np.abs(x)
    code = np.searchsorted(mid, a, side="left")  # first code whose upper midpoint is >= a
    at_mid = (code < len(mid)) & (a == mid[np.minimum(code, len(mid) - 1)])
    code = np.where(at_mid & (code % 2 == 1), code + 1, code)
    return np.where(np.isnan(x), np.nan, np.copysign(v[np.minimum(code, len(v) - 1)], x))


def rotary_axes(x, cos, sin, positions, pair_axis, interleaved):
    """x ``[T, H, D]``; positions ``[axes][T]``; pair p of token t turns by row
    positions[pair_axis[p]][t] of the tables.  A token with a position outside them keeps its
    values.  float64, unrounded."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    half = cos.shape[1]
    for t in range(x.shape[0]):
        if any(not 0 <= row[t] < cos.shape[0] for row in positions):
            continue
        for p in range(half):
            i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
            c, s = cos[positions[pair_axis[p]][t], p], sin[positions[pair_axis[p]][t], p]
            y[t, :, i] = x[t, :, i] * c - x[t, :, j] * s
            y[t, :, j] = x[t, :, i] * s + x[t, :, j] * c
    return y
