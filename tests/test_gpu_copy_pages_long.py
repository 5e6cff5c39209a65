"""pa_copy_pages with a list whose last entries' places do not fit in 32 bits."""

import pytest
import torch

import paged_kv_cache_page_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_a_list_of_copies_beyond_32_bits():
    n = 2 ** 31 // 3 + 7
    copies = torch.full((n, 3), -1, dtype=torch.int32, device=DEV)
    copies[-1] = i32([1, 2, 5])
    copies[-4] = i32([3, 99, 5])
    cache = torch.randn((4, 16, 1, 8), device=DEV).half()
    before, err = cache.clone(), pa.new_err_word(DEV)
    pa.pa_copy_pages(copies, [cache], err=err)
    before[2, :5] = before[1, :5]
    assert torch.equal(cache, before)
    assert err.tolist()[:3] == [pa.PA_DEVERR_PAGE_OOB, n - 4, 99]
