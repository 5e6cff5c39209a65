"""What reaches a result of pa_fwd_varlen_e4m3: small probabilities beside large ones in one tile, NaN in
values of keys that hardly count."""

import math

import pytest
import torch

from e4m3_util import DEV, batch, call, check

pytestmark = pytest.mark.gpu


def by_first_feature(scores, rows, d, dtype, page=16):
    """One sequence of one head whose row r scores key t with scores[t] powers of two."""
    w = batch([rows], [len(scores)], 1, 1, d, dtype, page=page, seed=len(scores))
    w["k_scale"] = w["v_scale"] = None
    w["q"].zero_()
    w["q"][:, 0, 0] = 1
    k = torch.zeros(-(-len(scores) // page) * page)
    k[:len(scores)] = torch.tensor(scores)
    ids = w["block_table"][0, :k.numel() // page].long()
    w["k_cache"][ids, :, :, 0] = k.view(-1, page, 1).to(torch.float8_e4m3fn).to(DEV)
    w["v_cache"][ids] = torch.zeros((), dtype=torch.float8_e4m3fn, device=DEV)
    return w, ids


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 100])
@pytest.mark.parametrize("top", [24.0, 26.0, 28.0])
def test_probabilities_of_a_tile_whose_maximum_rises(rows, top, d, dtype):
    """64 keys at 2^5, then one of 2^top in the same tile of 128: the value of the 64 in a feature where
    the last key holds nothing is 2^(11 - top) of its own, not zero."""
    scores = [0.0] * 32 + [5.0] * 64 + [0.0] * 31 + [top]
    w, ids = by_first_feature(scores, rows, d, dtype)
    v = torch.zeros((128, 1, d))
    v[32:96, :, 3] = 1
    v[127, :, 5] = 1
    w["v_cache"][ids] = v.view(-1, 16, 1, d).to(torch.float8_e4m3fn).to(DEV)
    out, lse = call(w, scale=math.log(2.0), causal=False)
    check(w, out, lse, scale=math.log(2.0), causal=False)


@pytest.mark.parametrize("rows", [1, 150])
@pytest.mark.parametrize("n", [200, 9001])
def test_nan_of_a_key_that_hardly_counts(rows, n):
    """A NaN in V at a visible key reaches the row however small the key's weight is, in one piece and
    joined from splits."""
    scores = [0.0] * (n - 7) + [208.0] * 7
    w, ids = by_first_feature(scores, rows, 64, "f16")
    w["v_cache"].view(torch.uint8)[ids[0], 2, 0, 3] = 0x7f
    w["v_cache"][ids[0], 2, 0, 4] = torch.ones((), dtype=torch.float8_e4m3fn, device=DEV)
    out, lse = call(w, scale=math.log(2.0), causal=False)
    assert torch.isnan(out[:, 0, 3]).all()
    rest = torch.arange(64, device=DEV) != 3
    assert (out[:, 0, rest] == 0).all() and torch.isfinite(lse).all()
