"""A beam search's step over a paged cache, and cross attention (oracle; test infrastructure).

Plain loops in the order the definitions are stated in, in float64; it shares no code with the
CUDA library.
"""

import numpy as np


def select(logits, scores, num_out, finished=None, end_token=-1):
    """logits ``[B][K][V]``, scores ``[B][K]``.  Returns (scores, parents, tokens, finished) as lists,
    -inf, -1, -1, False where there are fewer candidates."""
    out = ([], [], [], [])
    for b in range(len(logits)):
        found = []
        for k in range(len(logits[b])):
            s = float(scores[b][k])
            if not np.isfinite(s):
                continue
            if finished is not None and finished[b][k]:
                found.append((s, k, end_token))
                continue
            x = np.asarray(logits[b][k], dtype=np.float64)
            if np.isnan(x).any() or (x == np.inf).any() or (x == -np.inf).all():
                continue
            top = x.max()
            lse = top + np.log(np.exp(x - top).sum())
            found += [(s + (float(x[v]) - lse), k, v) for v in range(len(x)) if x[v] > -np.inf]
        found.sort(key=lambda c: (-c[0], c[1], c[2]))
        found = found[:num_out]
        lack = num_out - len(found)
        out[0].append([c[0] for c in found] + [-np.inf] * lack)
        out[1].append([c[1] for c in found] + [-1] * lack)
        out[2].append([c[2] for c in found] + [-1] * lack)
        out[3].append([c[2] == end_token or bool(finished is not None and finished[b][c[1]])
                       for c in found] + [False] * lack)
    return out


def reorder(parents, lens, table, free, page, num_pages):
    """parents ``[B][K]``, lens ``[B * K]``, table a list of rows, free the free pages (a stack).
    Returns a dict with the new rows (each only as long as the child's pages), lengths, stack,
    copies, the first refused request (or None) and those left out as malformed."""
    free = list(free)
    rows, new_lens, copies, bad = [], [], [], []
    fail, todo = None, []
    K = len(parents[0]) if parents else 1
    pages = lambda n: -(-n // page)  # noqa: E731
    balance = len(free)
    for b, par in enumerate(parents):
        mine = range(b * K, b * K + K)
        sound = all(-1 <= p < K for p in par) and all(
            0 <= lens[r] <= len(table[r]) * page for r in mine)
        held = [table[r][:pages(lens[r])] if 0 <= lens[r] <= len(table[r]) * page else []
                for r in mine]
        if sound:
            sound = all(0 <= e < num_pages for row in held for e in row)
        stay = dict(rows=[list(h) for h in held], lens=[lens[r] for r in mine],
                    copies=[(-1, -1, 0)] * K, wants=[])
        if not sound:
            bad.append(b)
            todo.append((stay, []))
            continue
        child = [list(held[p]) if p >= 0 else [] for p in par]
        length = [lens[b * K + p] if p >= 0 else 0 for p in par]
        given = []
        for j in range(max(len(h) for h in held)):
            kept = [c[j] for c in child if j < len(c)]
            for k in range(K):
                if j < len(held[k]) and held[k][j] not in kept and held[k][j] not in [
                        held[q][j] for q in range(k) if j < len(held[q])]:
                    given.append(held[k][j])
        partly = [length[i] // page if length[i] % page else -1 for i in range(K)]
        wants = []
        for i in range(K):
            j = partly[i]
            if j < 0:
                continue
            for o in range(K):
                if o != i and j < len(child[o]) and child[o][j] == child[i][j] and (
                        o < i or partly[o] != j):
                    wants.append((j, i))
                    break
        wants.sort()
        balance += len(given) - len(wants)
        if fail is None and balance < 0 and wants:
            fail = b
        if fail is not None:
            todo.append((stay, []))
            continue
        todo.append((dict(rows=child, lens=length, copies=[(-1, -1, 0)] * K, wants=wants), given))
    for _, given in todo:
        free += given
    for t, _ in todo:
        for j, i in t["wants"]:
            fresh = free.pop()
            t["copies"][i] = (t["rows"][i][j], fresh, t["lens"][i] % page)
            t["rows"][i][j] = fresh
        rows += t["rows"]
        new_lens += t["lens"]
        copies += t["copies"]
    return dict(rows=rows, lens=new_lens, free=free, copies=copies, fail=fail, bad=bad)


def cross(q, k, v, cu_q, cu_k, lens_k=None, mask=None, scale=None):
    """q ``[rows, Hq, D]``, k and v ``[keys, Hkv, D]``; returns (O, LSE ``[Hq, rows]``), zero and -inf
    for rows without a key; rows of no entry are NaN."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    rows, hq, d = q.shape
    group = hq // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out, lse = np.full(q.shape, np.nan), np.full((hq, rows), np.nan)
    for b in range(len(cu_q) - 1):
        n = cu_k[b + 1] - cu_k[b] if lens_k is None else lens_k[b]
        at = [t for t in range(cu_k[b], cu_k[b] + n) if mask is None or mask[t]]
        for r in range(cu_q[b], cu_q[b + 1]):
            for h in range(hq):
                if not at:
                    out[r, h], lse[h, r] = 0.0, -np.inf
                    continue
                x = k[at, h // group] @ q[r, h] * scale
                top = x.max()
                e = np.exp(x - top)
                out[r, h] = e @ v[at, h // group] / e.sum()
                lse[h, r] = top + np.log(e.sum())
    return out, lse
