"""pa_beam_select with more than 32 candidates over large vocabularies; scores as in test_gpu_beam_select."""

import numpy as np
import pytest
import torch

import paged_kv_cache_page_gb300 as pa
from oracle import beam

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
LSE = 2.0 ** -17


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,K,V,N", [(1, 32, 32000, 33), (1, 32, 32000, 64), (2, 16, 50257, 64),
                                     (1, 4, 20011, 48), (70, 3, 9001, 40)])
def test_more_than_32_candidates(B, K, V, N, dtype):
    g = torch.Generator().manual_seed(V + N)
    x = (torch.randn((B, K, V), generator=g) * 2.5).to(TYPES[dtype]).to(DEV)
    scores = (-torch.rand((B, K), generator=g).cumsum(1) * 3).to(DEV)
    got = pa.pa_beam_select(x, scores, N)
    some = [0, B - 1]
    want = beam.select(x[some].double().cpu().numpy(), scores[some].cpu().numpy(), N)
    assert got[1][some].tolist() == want[1] and got[2][some].tolist() == want[2]
    assert (np.abs(got[0][some].double().cpu().numpy() - np.array(want[0]))
            <= LSE + 2.0 ** -23 * np.abs(np.array(want[0]))).all()
