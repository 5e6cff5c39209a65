"""pa_beam_reorder: calls of every size behind small ones, whose clusters are chosen for their own blocks."""

import pytest
import torch

import paged_kv_cache_page_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_small_calls_in_front_of_large_ones():
    for B, K, pages in ((17, 1, 40), (4096, 1, 8), (128, 32, 40), (2000, 2, 1)):
        num_pages = B * K * pages + B
        rows = torch.arange(B * K * pages, dtype=torch.int32).view(B * K, pages)
        table, lens = rows.to(DEV), i32([16 * pages] * (B * K))
        parents = torch.full((B, K), K - 1, dtype=torch.int32, device=DEV)
        pool, count, err = i32([0] * num_pages), i32([0]), pa.new_err_word(DEV)
        out, new_lens, copies = pa.pa_beam_reorder(parents, lens, table, pool, count, 16, err=err)
        last = rows.view(B, K, pages)[:, K - 1:].expand(B, K, pages).reshape(B * K, pages)
        assert err[0].item() == 0 and torch.equal(out.cpu(), last) and (copies[:, 0] == -1).all()
        gone = rows.view(B, K, pages)[:, :K - 1].transpose(1, 2).reshape(-1)
        assert torch.equal(pool[:count.item()].cpu(), gone)
