"""pa_beam_select against the oracle's lists: parents and tokens equal, scores to their rounding.

Scores.  A sum of V exponentials of 2^t in fp32: the exponent is rounded once (2^-24 |t| ln 2 of a
term that weighs 2^t: less than 2^-24 of the sum), 2^t to 2^-22, and the sums of a lane (at most 65
elements a step and 8 steps here), a warp and the units add at most (66 + 8 + 5) 2^-24: together
below 2^-17 of the sum, so of lse.  The fp32 score is off by 2^-24 of itself.
"""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_page_gb300 as pa
from oracle import beam

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def check(x, scores, n, finished=None, end=-1, err_code=0, **kw):
    """x: the logits as the call gets them (a view on the GPU)."""
    err = pa.new_err_word(DEV)
    s = torch.as_tensor(scores, dtype=torch.float32).to(DEV)
    f = None if finished is None else torch.as_tensor(finished).to(DEV)
    got = pa.pa_beam_select(x, s, n, finished=f, end_token=end, err=err, **kw)
    torch.cuda.synchronize()
    assert err[0].item() == err_code
    want = beam.select(x.double().cpu().numpy(), s.cpu().numpy(), n, finished, end)
    assert got[1].tolist() == want[1]
    assert got[2].tolist() == want[2]
    if end >= 0:
        assert got[3].tolist() == want[3]
    a, b = got[0].double().cpu().numpy(), np.array(want[0])
    assert np.array_equal(np.isfinite(a), np.isfinite(b))
    live = np.isfinite(b)
    assert (np.abs(a - b)[live] <= 2.0 ** -17 + 2.0 ** -23 * np.abs(b)[live]).all()
    return got, err


def logits(seed, B, K, V, dtype, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, K, V), generator=g) * spread).to(TYPES[dtype]).to(DEV)


def some_scores(seed, B, K):
    g = torch.Generator().manual_seed(seed + 1000)
    return -torch.rand((B, K), generator=g).cumsum(1) * 3


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,K,V,N", [(1, 1, 1, 1), (1, 4, 7, 4), (3, 2, 8, 4), (2, 5, 9, 10),
                                     (1, 3, 255, 6), (2, 4, 257, 8), (1, 4, 2049, 4),
                                     (2, 8, 4099, 16), (1, 32, 1001, 64), (20, 3, 3001, 3),
                                     (1, 4, 32000, 4), (3, 5, 50001, 10), (40, 2, 5003, 4),
                                     (80, 3, 1999, 6), (160, 2, 2050, 4), (400, 1, 515, 2)])
def test_sizes(dtype, B, K, V, N):
    check(logits(V + N, B, K, V, dtype), some_scores(V, B, K), N)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_rows_of_any_alignment_and_stride(dtype):
    for start, V, pad in ((0, 1000, 3), (1, 1001, 0), (3, 515, 6), (5, 2, 1), (7, 33, 2)):
        wide = logits(start, 2, 3, start + V + pad, dtype)
        x = wide[:, :, start:start + V]
        check(x, some_scores(V, 2, 3), min(6, 3 * V))
        # beams and requests in another order of memory
        check(x.transpose(0, 1), some_scores(V, 3, 2), min(4, 2 * V))
        check(x[:, :1].expand(2, 3, V), [[0.0, -1.0, -2.5]] * 2, min(6, 3 * V))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_ties_go_to_the_lowest_place(dtype):
    # few values, many of each: the candidates pass the bound by the thousand
    V = 20000
    x = torch.zeros((2, 4, V), dtype=TYPES[dtype], device=DEV)
    check(x, [[0.0] * 4, [0.0, -0.25, -0.5, 0.0]], 8)
    check(x, [[0.0] * 4, [-2.0, -1.0, 0.0, -1.0]], 64)
    x[:, :, 777::1000] = 1.5
    check(x, [[0.0] * 4, [-2.0, -1.0, 0.0, -1.0]], 64)
    # equal beams side by side
    y = logits(5, 1, 1, 4096, dtype).expand(2, 4, 4096).contiguous()
    check(y, [[0.0] * 4, [-1.0, -1.0, 0.0, 0.0]], 10)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_masked_tokens(dtype):
    x = logits(9, 3, 4, 3001, dtype)
    x[0, :, :2990] = -math.inf
    x[1, 0] = -math.inf       # nothing to choose
    x[1, 1:, 5:] = -math.inf
    x[2] = -math.inf
    x[2, 3, 3000] = 2.0       # one candidate in all
    check(x, some_scores(3, 3, 4), 12)
    low = logits(10, 2, 3, 2000, dtype)
    low[:, :, ::2] = torch.finfo(low.dtype).min
    check(low, some_scores(4, 2, 3), 6)


def test_dead_and_finished_beams():
    x = logits(11, 4, 4, 1000, "bf16")
    x[0, 1] = math.nan        # (of beams that are not read)
    x[1, 2] = math.inf
    scores = [[0.0, -math.inf, -math.inf, -math.inf], [-1.0, -2.0, -0.5, math.nan],
              [-math.inf] * 4, [-3.0, -0.1, -0.2, -0.3]]
    finished = [[False, True, False, False], [False, False, True, True], [True] * 4,
                [False, True, True, True]]
    check(x, scores, 8, finished, 3)
    check(x, scores, 8, [[False] * 4, [False, False, True, False], [False] * 4, [True] * 4], 999)
    # the end token as an ordinary choice
    y = logits(12, 2, 2, 300, "f32")
    y[:, :, 7] = 20.0
    got, _ = check(y, [[0.0, -1.0]] * 2, 4, [[False, False]] * 2, 7)
    assert got[3][:, 0].all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_rows_without_a_distribution_are_reported(bad):
    for at in (0, 1500, 2999):
        x = logits(13, 2, 3, 3000, "f16")
        x[1, 2, at] = bad
        got, err = check(x, some_scores(6, 2, 3), 6, err_code=pa.PA_DEVERR_VALUE)
        assert err[1].item() == 5


@pytest.mark.parametrize("dtype,K,V", [("f32", 1, 1 << 21), ("bf16", 2, 1 << 21), ("f32", 32, 40000)])
def test_large_vocabularies(dtype, K, V):
    x = logits(14, 1, K, V, dtype)
    x[0, 0, V - 1] = 30.0
    check(x, some_scores(7, 1, K), 4)
    # large offsets from the base of the tensor, one vocabulary in the middle of a batch
    if dtype == "f32" and K == 1:
        y = torch.zeros((1100, 1, V), dtype=torch.bfloat16, device=DEV)
        y[1099] = x[0]
        s, p, t, _ = pa.pa_beam_select(y, torch.zeros((1100, 1), device=DEV), 2)
        w = beam.select(y[1099:].double().cpu().numpy(), [[0.0]], 2)
        assert t[1099].tolist() == w[2][0] and t[5].tolist() == [0, 1]


def test_extreme_values():
    x = logits(15, 2, 3, 5000, "f32", spread=1e4)
    check(x, some_scores(8, 2, 3), 5)
    x = logits(16, 2, 3, 5000, "f32")
    x[0] += 1000.0
    check(x, [[-1e4, -1e4 - 0.5, -1e4 - 1.0], [1e5, 1e5 - 1, -1e5]], 6)
    # one token has nearly all of the weight
    x[1, :, 4000] = 80.0
    check(x, [[0.0] * 3, [0.0, -1.0, -2.0]], 6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [2.0 ** 27, 2.0 ** 28.9, 2.0 ** 29, 1e9, 1e10, 1e15, 2.0 ** 61, 1e30, 2e38,
                                  "the type's largest"])
def test_logits_far_from_zero(size, dtype):
    """Next to each other such logits differ by 32 and more from 2^29 on: lse is the largest and the logarithm
    of how many there are.  Up to there the exponent 2^t has |t| <= 32 + 2: 2^-24 34 ln 2 < 2^-19."""
    lowest = torch.finfo(TYPES[dtype]).min
    size = -lowest if isinstance(size, str) else size
    near = size * (1 + 2.0 ** -21 * logits(20, 2, 3, 3001, "f32", spread=4.0).double())
    near = near.clamp(max=-lowest).to(TYPES[dtype])
    for x in (near, -near):
        x = x.clone()
        x[0, 1, 100:] = 3.0     # ordinary ones beside them
        x[1, 0, ::2] = -math.inf
        x[1, 1] = lowest        # nothing but the mask's value
        x[1, 2, 7:] = lowest
        check(x, some_scores(11, 2, 3), 5)


def test_streams_and_graph_replays():
    x = logits(17, 4, 4, 8001, "bf16")
    s = some_scores(9, 4, 4).to(DEV)
    ref = pa.pa_beam_select(x, s, 8, end_token=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = pa.pa_beam_select(x, s, 8, end_token=2)
    out = [torch.empty_like(t) for t in ref]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_beam_select(x, s, 8, end_token=2, scores_out=out[0], parents=out[1], tokens=out[2],
                          finished_out=out[3])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(ref, got, out):
        assert torch.equal(a, b) and torch.equal(a, c)
    y = logits(18, 4, 4, 8001, "bf16")
    x.copy_(y)
    graph.replay()
    ref = pa.pa_beam_select(y, s, 8, end_token=2)
    for a, c in zip(ref, out):
        assert torch.equal(a, c)
