"""pa_fwd_cross for few rows where a warp's ring goes round many times: batches that leave few CTAs a cluster,
two rounds of clusters, long states of one kv head; against the softmax in 64 bits.

Tolerances as in test_gpu_cross: u for P and for the result (fp16 2^-11, bf16 2^-8), scores below 1e-4,
exponentials, sums and joins below 2^-18.
"""

import math

import pytest
import torch

import paged_kv_cache_page_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def starts(n):
    out = [0]
    for x in n:
        out.append(out[-1] + x)
    return out


def plain(q, k, v, cu_q, cu_k, mask):
    """(O, sum p |v|, LSE) in 64 bits, an entry at a time."""
    hq, d = q.shape[1:]
    group = hq // k.shape[1]
    out, size = (torch.zeros(q.shape, dtype=torch.float64, device=DEV) for _ in range(2))
    lse = torch.full((hq, q.shape[0]), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(len(cu_q) - 1):
        rows, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        kk, vv = k[keys], v[keys]
        if mask is not None:
            kk, vv = kk[mask[keys]], vv[mask[keys]]
        if kk.shape[0] == 0 or cu_q[b] == cu_q[b + 1]:
            continue
        kk, vv = (x.double().repeat_interleave(group, 1).transpose(0, 1) for x in (kk, vv))
        s = q[rows].double().transpose(0, 1) @ kk.transpose(1, 2) * d ** -0.5
        lse[:, rows] = s.logsumexp(-1)
        p = s.softmax(-1)
        out[rows], size[rows] = (p @ vv).transpose(0, 1), (p @ vv.abs()).transpose(0, 1)
    return out, size, lse


# entries, rows, keys, query and kv heads, head dim: tiles of a warp at most
CASES = [
    (256, lambda i: 1 + i % 3, lambda i: 2000 - 7 * i if i % 5 else i, 4, 4, 64),     # 63: two rounds, 21 each
    (100, lambda i: i % 5, lambda i: 1500 - 11 * i, 4, 2, 128),                       # 2 slices: 11
    (300, lambda i: 2, lambda i: (i * 37) % 1000, 8, 1, 64),                          # 4 slices: 8
    (500, lambda i: 1, lambda i: 600 - i, 8, 4, 128),                                 # two rounds, one CTA: 38
    (600, lambda i: 1 + (i == 7), lambda i: 1100 if i % 6 == 0 else i, 4, 4, 128),    # 69
    (1, lambda i: 3, lambda i: 20000, 4, 1, 128),                                     # 16 CTAs: 20
    (2, lambda i: 4, lambda i: 33333 + i, 2, 2, 64),                                  # 16 CTAs, 2 slices: 33
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("n,rows,keys,hq,hkv,d", CASES)
def test_many_tiles_a_warp(n, rows, keys, hq, hkv, d, masked, dtype):
    rows, keys = [rows(i) for i in range(n)], [keys(i) for i in range(n)]
    assert max(rows) * hq // hkv <= 16
    cu_q, cu_k = starts(rows), starts(keys)
    g = torch.Generator(DEV).manual_seed(n + d)
    q = torch.randn((cu_q[-1], hq, d), generator=g, device=DEV).to(TYPES[dtype])
    kv = torch.randn((cu_k[-1], 2, hkv, d), generator=g, device=DEV).to(TYPES[dtype])
    k, v = kv[:, 0], kv[:, 1]
    mask = None
    if masked:
        mask = torch.rand(cu_k[-1], generator=g, device=DEV) < 0.7
        for b in range(0, n, 3):  # whole tiles behind the third, and all that follows the twelfth
            mask[cu_k[b]:cu_k[b + 1]][96:192] = False
            if b % 2:
                mask[cu_k[b]:cu_k[b + 1]][384:] = False
        if n > 9:
            mask[cu_k[9]:cu_k[10]] = False
        kv[~mask] = math.nan
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full((hq, q.shape[0]), 7.0, device=DEV)
    err = pa.new_err_word(DEV)
    pa.pa_fwd_cross(q, k, v, i32(cu_q), i32(cu_k), max(rows), max(keys), key_mask=mask, out=out, lse=lse,
                    err=err)
    o, size, l = plain(q, k, v, cu_q, cu_k, mask)
    assert err.tolist()[0] == 0
    u = torch.finfo(q.dtype).eps / 2
    assert torch.isfinite(out).all()
    off = (out.double() - o).abs() - ((u + 2e-4) * size + u * o.abs() + 2.0 ** -24)
    assert off.max().item() <= 0, (off.max().item(), off.argmax().item())
    assert torch.equal(torch.isinf(lse), torch.isinf(l))
    seen = torch.isfinite(l)
    assert (lse.double() - l)[seen].abs().max().item() <= 1.1e-4


@pytest.mark.parametrize("d", [64, 128])
def test_nan_far_into_a_stream(d):
    """A NaN in the last tiles of a warp's share reaches its rows and no others."""
    n, keys, heads = 500, 600, 4
    g = torch.Generator(DEV).manual_seed(d)
    q = torch.randn((2 * n, heads, d), generator=g, device=DEV).half()
    k, v = (torch.randn((n * keys, heads, d), generator=g, device=DEV).half() for _ in range(2))
    k[17 * keys + 599, 2] = math.nan
    v[33 * keys + 577, 1, 5] = math.nan
    cu_q, cu_k = i32(list(range(0, 2 * n + 1, 2))), i32(list(range(0, n * keys + 1, keys)))
    out, lse = pa.pa_fwd_cross(q, k, v, cu_q, cu_k, 2, keys)
    want = torch.zeros(q.shape, dtype=torch.bool, device=DEV)
    want[34:36, 2] = True
    want[66:68, 1, 5] = True
    assert torch.equal(torch.isnan(out), want)
    want = torch.zeros(lse.shape, dtype=torch.bool, device=DEV)
    want[2, 34:36] = True
    assert torch.equal(torch.isnan(lse), want)
