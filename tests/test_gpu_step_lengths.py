"""Requests with a malformed cached length keep it through pa_plan_step, in place too, so that a later
call still finds their pages."""

import pytest
import torch

import paged_kv_cache_page_gb300 as pa
from oracle import serving as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("bad", [-1, -(2 ** 31), 33, 2 ** 31 - 1])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B", [3, 300, 1500])
def test_malformed_lengths_are_kept(B, in_place, bad):
    cached, new = [5] * B, [1] * B
    cached[1] = cached[B - 1] = bad
    new[B - 1] = 0
    table = [[2 * b, -1] for b in range(B)]
    lens, err = i32(cached), pa.new_err_word(DEV)
    out = lens if in_place else i32([0] * B)
    cu, lk, slots, pos = pa.pa_plan_step(lens, i32(new), i32(table), i32([1] * (2 * B)), i32([1]), 16,
                                         seqlens_k=out, token_capacity=B, err=err)
    want = sv.plan_step(cached, new, table, [1], 16, B, 2 * B)
    assert lk.tolist() == want["seqlens_k"] == [bad if b in (1, B - 1) else 6 for b in range(B)]
    assert cu.tolist() == want["cu_seqlens_q"] and slots.tolist() == want["slot_mapping"]
    assert err.tolist()[0] == pa.PA_DEVERR_LENGTH and err.tolist()[2] == bad
