"""pa_fwd_cross where many keys of small weight make up the result.

One key, or one of sixteen, has nearly all of the weight and no value, n others 2^-25 to 2^-30 of its weight
each and the value 1000: O is 1000 n w / (heavy keys + n w).  The others' probabilities are fp16 numbers
against a reference 2^8 below the largest, so each is rounded to 2^-11 of itself or to 2^-25 2^-8 of the
largest weight (half a step of fp16's subnormals), twice where it was written under another reference; the
result is rounded to 2^-11 of itself (2^-25 at least) once more.  bf16 has no such border: 2^-8.  A warp or
CTA has at most 128 tiles here (65536 keys of head dim 128: 16 CTAs, 2 warps a head, 16 keys): their sums are
off by 2^-24 each, 2^-17, and O by at most 2^-23 in each of two additions a tile, 2^-15; scores by
2^-23 30 ln 2, below 2^-18.
"""

import math

import pytest
import torch

import paged_kv_cache_page_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 5, 80])
@pytest.mark.parametrize("n,power", [(8192, -25.203125), (65536, -25.203125), (65536, -28.0), (65536, -30.0)])
def test_many_small_weights(n, power, rows, d, dtype):
    q = torch.zeros((rows, 2, d), dtype=dtype, device=DEV)
    q[:, :, 0] = 1
    power = torch.tensor(power, dtype=dtype).double().item()
    w, value = 2.0 ** power, 1000.0
    for heavy in ([0], [n // 2 + 5], [n], list(range(3, n, 16))):
        k = torch.zeros((n + len(heavy), 2, d), dtype=dtype, device=DEV)
        k[:, :, 0] = power
        v = torch.full((n + len(heavy), 2, d), value, dtype=dtype, device=DEV)
        k[heavy], v[heavy] = 0, 0
        out, lse = pa.pa_fwd_cross(q, k, v, i32([0, rows]), i32([0, k.shape[0]]), rows, k.shape[0],
                                   scale=math.log(2))
        weights = len(heavy) + n * w
        want = n * w * value / weights
        if dtype == torch.float16:
            room = n * 2 * (2.0 ** -11 * w + 2.0 ** -33) * value / weights + 2.0 ** -11 * want + 2.0 ** -25
        else:
            room = (2 * 2.0 ** -8 + 2.0 ** -8) * want
        off = (out.double() - want).abs().max().item()
        assert off <= room + 2.0 ** -14 * want, (heavy[:2], want)
        off = (lse.double() - math.log(weights)).abs().max().item()
        assert off <= 2.0 ** -16, (heavy[:2], weights)
