"""pa_plan_step and pa_release_pages against the oracle's loops: whole numbers, all equal."""

import random

import pytest
import torch

import paged_kv_cache_page_gb300 as pa
from oracle import serving as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def batch(rng, B, ctx, page, width, extra):
    cached = [rng.randint(0, ctx) for _ in range(B)]
    held = [sv.pages_of(c, page) for c in cached]
    num_pages = sum(held) + extra
    order = list(range(num_pages))
    rng.shuffle(order)
    table = [[-1] * width for _ in range(B)]
    for b in range(B):
        for j in range(held[b]):
            table[b][j] = order.pop()
    return cached, table, order, num_pages


def run_plan(cached, new, table, free, page, capacity, num_pages, in_place=False, pad=0):
    B, width = len(cached), len(table[0])
    wide = torch.full((B, width + pad), -7, dtype=torch.int32, device=DEV)
    wide[:, :width] = i32(table)
    tab = wide[:, :width]
    lens, count = i32(cached), i32([len(free)])
    pool = i32(free + [12345678] * (num_pages - len(free)))
    slots = torch.full((capacity,), -9, dtype=torch.int64, device=DEV)
    err = pa.new_err_word(DEV)
    out_count = count if in_place else i32([-5])
    cu, lk, slots, pos = pa.pa_plan_step(
        lens, i32(new), tab, pool, count, page, seqlens_k=lens if in_place else None,
        slot_mapping=slots, free_count_out=out_count, err=err)
    torch.cuda.synchronize()
    if not in_place:
        assert lens.tolist() == cached and count.item() == len(free)
    if pad:
        assert (wide[:, width:] == -7).all()
    left = out_count.item()
    return dict(cu_seqlens_q=cu.tolist(), seqlens_k=lk.tolist(), slot_mapping=slots.tolist(),
                positions=pos.tolist(), block_table=tab.tolist(), free=pool.tolist()[:left]), err.tolist()


def check_plan(cached, new, table, free, page, capacity, num_pages, **kw):
    want = sv.plan_step(cached, new, table, free, page, capacity, num_pages)
    got, err = run_plan(cached, new, table, free, page, capacity, num_pages, **kw)
    for name, value in got.items():
        assert value == want[name], name
    return want, err


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("B,ctx,chunk", [(1, 0, 1), (1, 100, 3000), (3, 40, 17), (67, 500, 300),
                                         (1023, 90, 9), (1025, 60, 5), (4096, 40, 3)])
def test_plan(B, ctx, chunk, page):
    rng = random.Random(B * 1000 + page)
    new = [rng.choice((0, 1, 1, rng.randint(1, chunk))) for _ in range(B)]
    width = sv.pages_of(ctx + chunk, page) + 1
    cached, table, free, n = batch(rng, B, ctx, page, width, B * sv.pages_of(chunk, page) + B)
    rows = sum(new)
    want, err = check_plan(cached, new, table, free, page, rows + 5, n, in_place=B % 2 == 1, pad=3)
    assert err[0] == 0 and not want["refused"]
    # a pool that is too small, and rows that are too few
    if B > 1 and rows > B:
        few = free[:len(free) - len(want["free"]) - 1] if len(want["free"]) < len(free) else free
        want, err = check_plan(cached, new, table, few, page, rows, n, in_place=B % 2 == 0)
        if want["refused"]:
            assert err[0] == pa.PA_DEVERR_CAPACITY and err[1] == want["refused"][0]
        want, err = check_plan(cached, new, table, free, page, rows - 1, n)
        assert want["refused"] and err[0] == pa.PA_DEVERR_CAPACITY


def test_plan_edges():
    # nothing at all; no rows; a full table row; exactly the free pages
    check_plan([5], [0], [[3]], [], 16, 0, 8)
    check_plan([5], [0], [[3]], [1, 2], 16, 4, 8)
    want, err = check_plan([15, 16], [1, 16], [[3, -1], [4, -1]], [6], 16, 17, 8)
    assert want["free"] == [] and err[0] == 0
    # the exact capacities are not enough by one
    want, err = check_plan([15, 16, 3], [2, 16, 1], [[3, -1], [4, -1], [5, -1]], [6], 16, 99, 8)
    assert want["refused"] == [1, 2] and err[:3] == [pa.PA_DEVERR_CAPACITY, 1, 1]
    cu, lk, slots, pos = pa.pa_plan_step(i32([]), i32([]), torch.empty((0, 4), dtype=torch.int32,
                                                                       device=DEV),
                                         i32([0]), i32([1]), 16, token_capacity=3)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 3 and pos.tolist() == [0] * 3


@pytest.mark.parametrize("c,n,value", [(-1, 1, -1), (33, 1, 33), (30, 3, 3), (5, -2, -2),
                                       (2 ** 31 - 1, 1, 2 ** 31 - 1), (5, 2 ** 31 - 1, 2 ** 31 - 1)])
def test_plan_reports_bad_lengths(c, n, value):
    want, err = check_plan([3, c, 10], [2, n, 1], [[0, -1], [1, 2], [3, -1]], [7, 6, 5], 16, 40, 8)
    assert want["bad"] == [1] and err[:3] == [pa.PA_DEVERR_LENGTH, 1, value]


def test_plan_reports_bad_pages():
    # an old entry and a free page outside the pool: their tokens have no slot
    want, err = check_plan([20], [1], [[3, 99]], [], 16, 4, 8)
    assert want["slot_mapping"] == [-1] * 4 and err[:3] == [pa.PA_DEVERR_PAGE_OOB, 0, 1]
    want, err = check_plan([16], [1], [[3, -1]], [-2], 16, 4, 8)
    assert want["block_table"] == [[3, -2]] and err[:3] == [pa.PA_DEVERR_PAGE_OOB, 0, 1]
    err = pa.new_err_word(DEV)
    out = i32([0])
    pa.pa_plan_step(i32([0]), i32([1]), i32([[-1]]), i32([4, 2]), i32([3]), 16, token_capacity=1,
                    free_count_out=out, err=err)
    assert err.tolist()[:3] == [pa.PA_DEVERR_CAPACITY, -1, 3] and out.item() == 1


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("B,ctx", [(1, 1), (1, 5000), (5, 100), (64, 3000), (1025, 300), (4096, 90)])
def test_release(B, ctx, page):
    rng = random.Random(B * 7 + page)
    cached, table, free, n = batch(rng, B, ctx, page, sv.pages_of(ctx, page) + 2, 9)
    keep = [rng.choice((0, c, c + 3, max(0, c - rng.randint(0, 40)))) for c in cached]
    for space, in_place in ((n, True), (len(free) + sum(sv.pages_of(c, page) for c in cached) // 3,
                                        False)):
        want, lens, refused, _ = sv.release_pages(cached, keep, table, free, page, space)
        bad = any(p >= space for row in table for p in row)
        pool = i32(free + [0] * (space - len(free)))
        cl, count, err = i32(cached), i32([len(free)]), pa.new_err_word(DEV)
        out, left = pa.pa_release_pages(cl, i32(keep), i32(table), pool, count, page,
                                        seqlens_out=None if in_place else i32([0] * B),
                                        free_count_out=None if in_place else i32([0]), err=err)
        torch.cuda.synchronize()
        assert out.tolist() == lens and left.item() == len(want)
        assert pool.tolist()[:len(want)] == want
        if not bad and not refused:
            assert err[0].item() == 0


def test_release_drops_bad_entries_and_reports():
    rng = random.Random(5)
    for B in (3, 300, 4096):
        cached, table, free, n = batch(rng, B, 200, 16, 14, 4)
        for b in range(0, B, 3):
            if cached[b] > 16:
                table[b][rng.randrange(sv.pages_of(cached[b], 16))] = rng.choice((-1, n, n + 77))
        want, lens, _, _ = sv.release_pages(cached, [0] * B, table, free, 16, n)
        pool, err = i32(free + [0] * (n - len(free))), pa.new_err_word(DEV)
        out, left = pa.pa_release_pages(i32(cached), i32([0] * B), i32(table), pool,
                                        i32([len(free)]), 16, err=err)
        assert left.item() == len(want) and pool.tolist()[:len(want)] == want
        assert out.tolist() == lens and err[0].item() == pa.PA_DEVERR_PAGE_OOB
    err = pa.new_err_word(DEV)
    out, left = pa.pa_release_pages(i32([20, -1, 99]), i32([-1, 0, 0]), i32([[1, 2]] * 3),
                                    i32([0, 0, 0]), i32([1]), 16, err=err)
    assert out.tolist() == [20, -1, 99] and left.item() == 1 and err[0].item() == pa.PA_DEVERR_LENGTH


def test_plan_and_release_replayed_from_a_graph():
    """A captured step whose lengths and pool live on the device: decode steps until the pool is
    empty, then everything is released and taken again."""
    B, page, width = 5, 16, 8
    n = 24
    lens, table = i32([0] * B), i32([[-1] * width] * B)
    pool, count, new = i32(list(range(n))), i32([n]), i32([7, 16, 1, 0, 30])
    slots = torch.zeros(80, dtype=torch.int64, device=DEV)
    cu, pos, keep = i32([0] * (B + 1)), i32([0] * 80), i32([0] * B)

    def step():
        pa.pa_plan_step(lens, new, table, pool, count, page, cu, lens, slots, pos)

    def drop():
        pa.pa_release_pages(lens, keep, table, pool, count, page)

    s = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(s):
        for fn in (step, drop):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                fn()
            graphs.append(g)
    torch.cuda.synchronize()
    cl, tab, free = [0] * B, [[-1] * width for _ in range(B)], list(range(n))
    for _ in range(2):
        for _ in range(5):
            want = sv.plan_step(cl, new.tolist(), tab, free, page, 80, n)
            graphs[0].replay()
            torch.cuda.synchronize()
            cl, tab, free = want["seqlens_k"], want["block_table"], want["free"]
            assert lens.tolist() == cl and slots.tolist() == want["slot_mapping"]
            assert cu.tolist() == want["cu_seqlens_q"] and count.item() == len(free)
        free, cl, _, _ = sv.release_pages(cl, [0] * B, tab, free, page, n)
        graphs[1].replay()
        torch.cuda.synchronize()
        assert pool.tolist()[:len(free)] == free and lens.tolist() == cl and count.item() == n
