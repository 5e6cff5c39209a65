"""pa_beam_select over long rows, whose sums are as good as the header says.

Scores.  A step of a lane adds at most 64 exponentials and an extra one in four sums, 16 deep, and these
in two more steps: (16 + 3) 2^-24 of the sum.  What a lane's steps add up to lacks 2^-24, however many
they are; a warp's sum 5 2^-24, and the row's parts nothing that counts.  An exponent is rounded twice
(2^-24 |t| ln 2 of a term that weighs 2^t, |t| at most log2(V) on the mean: 17 for 2^24), 2^t is good to
2^-22: together (19 + 1 + 5 + 34 + 4) 2^-24 < 2^-18, so of lse.  The fp32 score is off by 2^-24 of itself.
"""

import numpy as np
import pytest
import torch

import paged_kv_cache_page_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
LSE = 2.0 ** -17


@pytest.mark.parametrize("dtype,B,V,constant", [("f32", 160, 1 << 22, 0.4), ("f32", 1, 1 << 24, 0.4),
                                                ("f16", 160, 1 << 23, 0.45), ("bf16", 160, 1 << 23, None),
                                                ("f32", 160, (1 << 22) - 3, None)])
def test_sums_of_long_rows(dtype, B, V, constant):
    """Up to 2048 steps a lane.  All beams and requests read one row."""
    K = 32
    if constant is None:
        row = torch.randn((V,), generator=torch.Generator().manual_seed(V)).to(TYPES[dtype])
    else:
        row = torch.full((V,), constant).to(TYPES[dtype])
    x = row.to(DEV).expand(B, K, V)
    scores = -torch.arange(K, dtype=torch.float32, device=DEV).expand(B, K).contiguous()
    s, p, t, _ = pa.pa_beam_select(x, scores, 4)
    y = row.double().numpy()
    lse = y.max() + np.log(np.exp(y - y.max()).sum())
    best = np.argsort(-y, kind="stable")[:4]
    want = sorted((float(k) - (y[v] - lse), k, v) for k in range(4) for v in best.tolist())[:4]
    assert (t == t[0]).all() and (p == p[0]).all() and (s == s[0]).all()
    assert p[0].tolist() == [w[1] for w in want] and t[0].tolist() == [w[2] for w in want]
    ref = -np.array([w[0] for w in want])
    assert (np.abs(s[0].double().cpu().numpy() - ref) <= LSE + 2.0 ** -23 * np.abs(ref)).all()
