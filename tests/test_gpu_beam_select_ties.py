"""pa_beam_select for equal beams: a tie in every token, wherever their rows lie, and the lower beam comes first."""

import pytest
import torch

import paged_kv_cache_page_gb300 as pa
from oracle import beam

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V,K", [(3, 4), (33, 9), (1001, 4), (4099, 8), (50257, 5), (128001, 3)])
def test_equal_beams_in_rows_of_any_alignment(V, K, dtype):
    g = torch.Generator().manual_seed(V)
    row = (torch.randn((3, 1, V), generator=g) * 3).to(TYPES[dtype])
    x = row.expand(3, K, V).contiguous().to(DEV)
    if K > 4:  # others between them
        x[1, 1:K - 1:2] = torch.randn((V,), generator=g).to(TYPES[dtype]).to(DEV)
    if V > 100:
        x[2, :, 50:70] = -float("inf")
    scores = torch.zeros((3, K), device=DEV)
    scores[1, ::2] = -0.5
    n = min(3 * K, 64, K * V)
    err = pa.new_err_word(DEV)
    got = pa.pa_beam_select(x, scores, n, err=err)
    want = beam.select(x.double().cpu().numpy(), scores.cpu().numpy(), n)
    assert err[0].item() == 0
    assert got[1].tolist() == want[1] and got[2].tolist() == want[2]
    # a beam's score is the same wherever its row lies
    s, p, t = (y.tolist() for y in got[:3])
    for v in set(t[0]):
        assert len({s[0][i] for i in range(n) if t[0][i] == v}) == 1


@pytest.mark.parametrize("dtype", list(TYPES))
def test_zeros_of_either_sign_are_equal(dtype):
    row = torch.randn((1003,), generator=torch.Generator().manual_seed(2)).to(TYPES[dtype])
    row[::3] = 0.0
    x = row.expand(2, 3, 1003).contiguous().to(DEV)
    x[:, 1, ::3] = -0.0
    x[1, 2, ::6] = -0.0
    scores = torch.zeros((2, 3), device=DEV)
    got, want = pa.pa_beam_select(x, scores, 9), beam.select(x.double().cpu().numpy(), scores.cpu().numpy(), 9)
    assert got[1].tolist() == want[1] and got[2].tolist() == want[2]
