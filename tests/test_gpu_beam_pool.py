"""pa_beam_reorder at the end of the pool."""

import random

import pytest
import torch

import paged_kv_cache_page_gb300 as pa
from oracle import beam

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def reorder(parents, lens, rows, free, num_pages, in_place):
    width = max(len(r) for r in rows)
    table = i32([r + [-7] * (width - len(r)) for r in rows])
    seqlens, count = i32(lens), i32([len(free)])
    pool = i32(free + [-9] * (num_pages - len(free)))
    out = table if in_place else torch.full_like(table, -3)
    err = pa.new_err_word(DEV)
    out, new_lens, copies = pa.pa_beam_reorder(
        i32(parents), seqlens, table, pool, count, 16, block_table_out=out,
        seqlens_out=seqlens if in_place else torch.full_like(seqlens, -5), free_count_out=count, err=err)
    held = [out[i].tolist()[:-(-n // 16)] for i, n in enumerate(new_lens.tolist())]
    return dict(lens=new_lens.tolist(), rows=held, copies=[tuple(c) for c in copies.tolist()],
                free=pool.tolist()[:count.item()]), err.tolist()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,K", [(1, 2), (3, 4), (40, 5), (100, 32), (300, 8)])
def test_a_free_page_outside_the_pool_is_its_end(B, K, in_place):
    """Requests whose fresh pages would reach such an entry stay as they are, whole."""
    rng = random.Random(B + K)
    num_pages = 2 * B * K + 20
    pages = list(range(num_pages))
    rng.shuffle(pages)
    rows, lens, parents = [], [], []
    for b in range(B):
        common = pages.pop()
        for k in range(K):  # a common page and one that each beam writes to, or a prompt's first step
            n = rng.choice((16, 17, 31, 32)) if b % 3 else 21 if k == 0 else 0
            rows.append([common][:n] + ([pages.pop()] if n > 16 else []))
            lens.append(n)
        parents.append([rng.randint(0, K - 1) if b % 3 else 0 for _ in range(K)])
    whole = beam.reorder(parents, lens, rows, pages, 16, num_pages)
    assert whole["fail"] is None
    for depth in {0, 1, B, len(pages) // 2, len(pages) - 1}:
        free = list(pages)
        if not 0 <= depth < len(free):
            continue
        free[-1 - depth] = rng.choice((-1, num_pages, 2 ** 31 - 1, -2 ** 31))
        # what lies below the entry is out of reach
        want = beam.reorder(parents, lens, rows, free[len(free) - depth:], 16, num_pages)
        got, err = reorder(parents, lens, rows, free, num_pages, in_place)
        for name in ("lens", "rows", "copies"):
            assert got[name] == want[name], (name, depth)
        assert got["free"] == free[:len(free) - depth] + want["free"]
        if want["fail"] is None:
            assert err[0] == 0
        else:
            b = want["fail"]
            assert err[0] == pa.PA_DEVERR_PAGE_OOB and b * K <= err[1] < b * K + K
            assert err[2] == whole["lens"][err[1]] // 16
