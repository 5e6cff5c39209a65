"""pa_beam_reorder and pa_copy_pages against the oracle's lists: whole numbers and copies, all equal."""

import random

import pytest
import torch

import paged_kv_cache_page_gb300 as pa
from oracle import beam

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def grown(rng, B, K, page, steps, extra):
    """Tables of beams that have been reordered before: (lens, table, free, num_pages)."""
    lens, rows, free, parents = [0] * (B * K), [[] for _ in range(B * K)], list(range(extra)), None
    rng.shuffle(free)
    width = 0
    for step in range(steps):
        if parents is not None:
            r = beam.reorder(parents, lens, rows, free, page, extra)
            assert r["fail"] is None and not r["bad"]
            lens, rows, free = r["lens"], r["rows"], r["free"]
        for b in range(B):
            add = rng.randint(0, 3 * page) if step == 0 else rng.choice((0, 1, 1, rng.randint(1, page)))
            for k in range(K):
                row = b * K + k
                if step == 0 and k > 0:
                    continue
                new = add if k != K - 1 or step == 0 else add * rng.randint(0, 1)
                while len(rows[row]) < -(-(lens[row] + new) // page):
                    rows[row].append(free.pop())
                lens[row] += new
        parents = [[0] * K if step == 0 else [rng.randint(0, K - 1) for _ in range(K)]
                   for _ in range(B)]
        width = max([width] + [len(r) for r in rows])
    return lens, rows, free, width + 1


def run(parents, lens, rows, free, page, num_pages, width, in_place=False, pad=0):
    n = len(lens)
    K = len(parents[0])
    full = torch.full((n, width + pad), -7, dtype=torch.int32)
    for i, r in enumerate(rows):
        full[i, :len(r)] = torch.tensor(r, dtype=torch.int32)
    wide = full.to(DEV)
    table = wide[:, :width]
    pool = i32(free + [12345678] * (num_pages - len(free)))
    count, seqlens, err = i32([len(free)]), i32(lens), pa.new_err_word(DEV)
    out = None if in_place else torch.full((n, width), -3, dtype=torch.int32, device=DEV)
    left = None if in_place else i32([-5])
    new_lens = None if in_place else i32([-5] * n)
    out, new_lens, copies = pa.pa_beam_reorder(
        i32(parents).view(-1, K), seqlens, table, pool, count, page, block_table_out=out,
        seqlens_out=new_lens, free_count_out=left, err=err)
    torch.cuda.synchronize()
    if in_place:
        left = count
        if pad:
            assert (wide[:, width:] == -7).all()
    else:
        assert seqlens.tolist() == lens and torch.equal(wide.cpu(), full) and count.item() == len(free)
    got = dict(lens=new_lens.tolist(), copies=[tuple(c) for c in copies.tolist()],
               free=pool.tolist()[:left.item()], table=out.tolist())
    return got, err.tolist()


def check(parents, lens, rows, free, page, num_pages, width, **kw):
    want = beam.reorder(parents, lens, rows, free, page, num_pages)
    got, err = run(parents, lens, rows, free, page, num_pages, width, **kw)
    for name in ("lens", "copies", "free"):
        assert got[name] == want[name], name
    for i, r in enumerate(want["rows"]):
        assert got["table"][i][:len(r)] == r, i
        if not kw.get("in_place"):
            assert all(e == -3 for e in got["table"][i][len(r):]), i
    return want, err


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("B,K,steps", [(1, 1, 3), (1, 2, 6), (1, 4, 20), (3, 5, 9), (2, 32, 6),
                                       (17, 8, 5), (64, 3, 4), (130, 16, 3), (1000, 4, 3),
                                       (4096, 1, 2)])
def test_reorder(page, B, K, steps):
    rng = random.Random(B * 100 + K + page)
    extra = B * (K * steps * 3 + 8)
    lens, rows, free, width = grown(rng, B, K, page, steps, extra)
    for kind in range(3):
        parents = [[rng.randint(-1 if kind else 0, K - 1) for _ in range(K)] for _ in range(B)]
        if kind == 2:  # requests that end, and such that stay as they are
            for b in range(0, B, 3):
                parents[b] = [-1] * K
            for b in range(1, B, 3):
                parents[b] = list(range(K))
        want, err = check(parents, lens, rows, free, page, extra, width, in_place=kind == 1, pad=kind)
        assert err[0] == 0
    # a pool that lacks pages
    want = beam.reorder([[0] * K] * B, lens, rows, [], page, extra)
    for some in (0, 1, B // 3):
        want, err = check([[0] * K] * B, lens, rows, free[:some], page, extra, width,
                          in_place=B % 2 == 0)
        if want["fail"] is not None:
            assert err[:2] == [pa.PA_DEVERR_CAPACITY, want["fail"]]


def test_long_tables_and_no_requests():
    rng = random.Random(5)
    for width, K in ((700, 4), (5000, 2)):
        pool = list(range(2 * width + 10))
        rng.shuffle(pool)
        rows = [pool[:width - 1]] + [pool[:width // 2 + i] + pool[width * i:width * i + 90]
                                     for i in range(1, 2)]
        rows += [list(rows[1][:300]) for _ in range(K - 2)]
        rows = [r[:width - 1] for r in rows]
        rows = [list(dict.fromkeys(r)) for r in rows]
        lens = [len(r) * 16 for r in rows]
        used = {e for r in rows for e in r}
        free = [e for e in pool if e not in used]
        for parents in ([1] * K, [0] * K, [-1] * K, [K - 1, 0] + [1] * (K - 2)):
            check([parents], lens, rows, free, 16, len(pool), width)
    e = torch.empty((0, 4), dtype=torch.int32, device=DEV)
    out, lens, copies = pa.pa_beam_reorder(e, e.view(-1), e, i32([0, 0]), i32([1]), 16)
    assert out.shape == (0, 4) and copies.shape == (0, 3)


def test_malformed_requests_stay_as_they_are():
    rows = [[1, 2], [1, 3], [4, 5], [4, 6], [7], [8]]
    lens = [20, 20, 20, 30, 3, 3]
    good = [[0, 0], [1, 1], [1, 0]]
    for b, par in ((0, [2, 0]), (1, [-2, 0]), (2, [0, 99])):
        parents = [list(p) for p in good]
        parents[b] = par
        want, err = check(parents, lens, rows, [9, 10], 16, 11, 3)
        i = 0 if not -1 <= par[0] < 2 else 1
        assert want["bad"] == [b] and err[:3] == [pa.PA_DEVERR_VALUE, 2 * b + i, par[i]]
    for b, length in ((0, -1), (1, 49), (2, 2 ** 31 - 1)):
        bad = list(lens)
        bad[2 * b + 1] = length
        want, err = check(good, bad, rows, [9, 10], 16, 11, 3, in_place=True)
        assert want["bad"] == [b] and err[:3] == [pa.PA_DEVERR_LENGTH, 2 * b + 1, length]
    for b, entry in ((0, -1), (1, 11)):
        bad = [list(r) for r in rows]
        bad[2 * b + 1][1] = entry
        want, err = check(good, lens, bad, [9, 10], 16, 11, 3)
        assert want["bad"] == [b] and err[:3] == [pa.PA_DEVERR_PAGE_OOB, 2 * b + 1, 1]
    # a malformed pool
    for count in (-1, 12):
        err = pa.new_err_word(DEV)
        pa.pa_beam_reorder(i32([[0, 1]]), i32([3, 3]), i32([[1], [2]]), i32(list(range(11))),
                           i32([count]), 16, free_count_out=i32([0]), err=err)
        assert err.tolist()[:3] == [pa.PA_DEVERR_CAPACITY, -1, count]
    # a fresh page outside the pool is not handed out
    err, table = pa.new_err_word(DEV), i32([[1], [2]])
    _, _, copies = pa.pa_beam_reorder(i32([[0, 0]]), i32([3, 0]), table, i32([99] + [0] * 10), i32([1]),
                                      16, err=err)
    assert copies.tolist() == [[-1, -1, 0]] * 2 and err.tolist()[:2] == [pa.PA_DEVERR_PAGE_OOB, 1]


@pytest.mark.parametrize("kind", [torch.float16, torch.bfloat16, torch.float8_e4m3fn, torch.float32])
@pytest.mark.parametrize("page,heads,d,layers", [(16, 1, 64, 1), (16, 12, 64, 3), (64, 8, 128, 2),
                                                 (256, 2, 16, 150)])
def test_copy_pages(kind, page, heads, d, layers):
    g = torch.Generator().manual_seed(page + heads)
    pages, size = 23, torch.empty((), dtype=kind).element_size()
    raw = [torch.randint(0, 256, (pages, page, heads + 1, d * size), generator=g, dtype=torch.uint8)
           .to(DEV) for _ in range(2 * layers)]
    wide = [r.view(kind) for r in raw]
    for caches in (wide, [w[:, :, :heads] for w in wide]):  # whole rows, and slices of them
        before = [r.clone() for r in raw]
        order = torch.randperm(pages, generator=g).tolist()
        copies = [[order[0], order[1], page], [order[2], order[3], 1], [-1, order[4], 3],
                  [order[5], -1, 3], [order[6], order[7], 0], [order[0], order[8], page - 1]]
        err = pa.new_err_word(DEV)
        pa.pa_copy_pages(i32(copies), caches, err=err)
        torch.cuda.synchronize()
        assert err[0].item() == 0
        used = caches[0].shape[2]
        for r, old in zip(raw, before):
            for s, t, n in copies:
                if s >= 0 and t >= 0:
                    old[t, :n, :used] = old[s, :n, :used]
            assert torch.equal(r, old)
    for bad, code, value in (([99, 1, 2], pa.PA_DEVERR_PAGE_OOB, 99), ([1, 23, 2], pa.PA_DEVERR_PAGE_OOB, 23),
                             ([1, 2, page + 1], pa.PA_DEVERR_LENGTH, page + 1),
                             ([1, 2, -1], pa.PA_DEVERR_LENGTH, -1)):
        before = [r.clone() for r in raw]
        err = pa.new_err_word(DEV)
        pa.pa_copy_pages(i32([[0, 3, 0], bad]), wide, err=err)
        assert err.tolist()[:3] == [code, 1, value]
        assert all(torch.equal(r, o) for r, o in zip(raw, before))


def test_graph_replays():
    """A captured reorder and its copies, replayed while parents change, against the oracle."""
    rng = random.Random(3)
    B, K, page = 5, 4, 16
    extra = 400
    lens, rows, free, _ = grown(rng, B, K, page, 6, extra)
    width = 24
    full = torch.full((B * K, width), -1, dtype=torch.int32)
    for i, r in enumerate(rows):
        full[i, :len(r)] = torch.tensor(r, dtype=torch.int32)
    table, seqlens, count = full.to(DEV), i32(lens), i32([len(free)])
    pool = i32(free + [0] * (extra - len(free)))
    parents, copies = i32([[0] * K] * B), i32([[0] * 3] * (B * K))
    cache = torch.randn((extra, page, 2, 64), device=DEV).half()
    err = pa.new_err_word(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_beam_reorder(parents, seqlens, table, pool, count, page, copies=copies, err=err)
        pa.pa_copy_pages(copies, [cache], err=err)
    for _ in range(6):
        par = [[rng.randint(0, K - 1) for _ in range(K)] for _ in range(B)]
        parents.copy_(i32(par))
        old = cache.clone()
        graph.replay()
        torch.cuda.synchronize()
        r = beam.reorder(par, lens, rows, free, page, extra)
        lens, rows, free = r["lens"], r["rows"], r["free"]
        assert err[0].item() == 0 and seqlens.tolist() == lens
        assert pool.tolist()[:count.item()] == free
        for i, row in enumerate(rows):
            assert table[i, :len(row)].tolist() == row
        for s, t, n in r["copies"]:
            if s >= 0:
                old[t, :n] = old[s, :n]
        assert torch.equal(cache, old)
