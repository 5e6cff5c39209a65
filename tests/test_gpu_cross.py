"""pa_fwd_cross against the oracle's softmax in 64 bits.

Tolerances.  u is half a step of the type (fp16 2^-11, bf16 2^-8).  P is rounded to the type (u of
every term of sum p |v|), the result once more (u |O|); a score is a sum of D products in fp32, off
by at most (D + 1) 2^-24 scale sum |q k|, below 1e-4 for the N(0, 1) inputs here (129 * 2^-24 *
128^-0.5 * 130), which moves O by at most 2e-4 sum p |v| and LSE by 1e-4; exponentials, sums and the
join add less than 2^-18.
"""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_page_gb300 as pa
from oracle import beam

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def np64(t):
    return t.double().cpu().numpy()


def cu_of(n):
    return np.concatenate([[0], np.cumsum(n)]).tolist()


def inputs(seed, rows, keys, hq, hkv, d, dtype, spare=0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((sum(rows) + spare, hq, d), generator=g).to(TYPES[dtype]).to(DEV)
    kv = torch.randn((sum(keys), 2, hkv, d), generator=g).to(TYPES[dtype]).to(DEV)
    return q, kv[:, 0], kv[:, 1]


def compare(out, lse, q, k, v, cu_q, cu_k, lens_k=None, mask=None, scale=None):
    a = np64(q), np64(k), np64(v)
    mask = None if mask is None else mask.cpu().numpy()
    if mask is not None:  # (what is masked counts for nothing, whatever it is)
        for x in a[1:]:
            x[~mask] = 0
    o, l = beam.cross(*a, cu_q, cu_k, lens_k, mask, scale)
    size, _ = beam.cross(a[0], a[1], np.abs(a[2]), cu_q, cu_k, lens_k, mask, scale)
    u = torch.finfo(out.dtype).eps / 2
    live = ~np.isnan(o[:, 0, 0])
    got = np64(out)
    assert np.isfinite(got[live]).all()
    bound = (u + 2e-4) * size + u * np.abs(o) + 2.0 ** -24
    assert (np.abs(got - o)[live] <= bound[live]).all(), np.abs(got - o)[live].max()
    if lse is not None:
        got = np64(lse)[:, live]
        want = l[:, live]
        assert np.array_equal(np.isinf(got), np.isinf(want))
        fin = np.isfinite(want)
        assert (np.abs(got - want)[fin] <= 1.1e-4).all()


def check(rows, keys, hq, hkv, d, dtype, seed=0, mask=None, spare=0):
    q, k, v = inputs(seed, rows, keys, hq, hkv, d, dtype, spare)
    cu_q, cu_k = cu_of(rows), cu_of(keys)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full((hq, q.shape[0]), 7.0, device=DEV)
    err = pa.new_err_word(DEV)
    pa.pa_fwd_cross(q, k, v, i32(cu_q), i32(cu_k), max(rows), max(keys), key_mask=mask, out=out,
                    lse=lse, err=err)
    torch.cuda.synchronize()
    assert err.tolist()[0] == 0, err.tolist()
    compare(out, lse, q, k, v, cu_q, cu_k, mask=mask)
    if spare:
        assert (out[sum(rows):] == 7.0).all() and (lse[:, sum(rows):] == 7.0).all()


HEADS = [(4, 2, 64), (8, 1, 64), (3, 3, 64), (12, 12, 64), (16, 4, 128), (10, 2, 128), (4, 4, 128)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_ragged(hq, hkv, d, dtype):
    check([4, 1, 0, 5, 3, 8], [100, 1, 33, 0, 17, 257], hq, hkv, d, dtype, seed=hq + d, spare=3)
    check([5], [1000], hq, hkv, d, dtype, seed=1)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("hq,hkv,d", HEADS + [(7, 1, 64), (20, 1, 128), (66, 2, 64), (130, 1, 64)])
def test_ragged_with_many_rows(hq, hkv, d, dtype):
    check([70, 1, 0, 37, 131], [300, 1, 33, 0, 129], hq, hkv, d, dtype, seed=hq + d, spare=3)


@pytest.mark.parametrize("dtype,d", [("f16", 128), ("bf16", 64)])
def test_long_streams_are_cut_and_joined(dtype, d):
    check([90, 3], [9000, 130], 2, 2, d, dtype, seed=1)
    # groups without rows in cut streams; a mask that leaves a whole part unseen
    mask = torch.ones(9130, dtype=torch.bool, device=DEV)
    mask[:4000] = False
    mask[9000:] = False
    check([90, 3], [9000, 130], 2, 2, d, dtype, seed=2, mask=mask)
    check([300], [2000], 4, 1, d, dtype, seed=3)


@pytest.mark.parametrize("rows", [1, 70])
def test_many_entries(rows):
    n = 1000
    check([rows if i % 100 == 7 else i % 3 for i in range(n)], [i * 7 % 50 for i in range(n)], 2, 1, 64,
          "f16", spare=1)


@pytest.mark.parametrize("n,rows,keys,hq,hkv,d", [
    (20, lambda i: 18 + i % 20, lambda i: 100 + 37 * i, 12, 12, 64),
    (32, lambda i: 300 if i % 7 == 0 else 5 + i, lambda i: 50 + 29 * i, 16, 4, 128),
    (33, lambda i: 300 if i % 7 == 0 else 5 + i, lambda i: 50 + 29 * i, 16, 4, 128),
    (32, lambda i: 10 + i % 3, lambda i: 150 * (i % 9 != 4), 40, 20, 64),
])
def test_hundreds_of_streams(n, rows, keys, hq, hkv, d):
    """Two to five streams a CTA, of one and two tiles of rows, dealt whole (up to 32 entries) and cut."""
    rows, keys = [rows(i) for i in range(n)], [keys(i) for i in range(n)]
    check(rows, keys, hq, hkv, d, "bf16", seed=n, spare=2)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,d", [(3, 64), (3, 128), (40, 64), (200, 128)])
def test_a_single_key_is_its_value(rows, d, dtype):
    """O = P V / l with one P, a power of two to 2^-21: V itself, whose half a step is 2^-12 of it or more."""
    q, k, v = inputs(12, [rows, rows], [1, 150], 4, 2, d, dtype)
    mask = torch.zeros(151, dtype=torch.bool, device=DEV)
    mask[0] = mask[90] = True
    out, _ = pa.pa_fwd_cross(q, k, v, i32([0, rows, 2 * rows]), i32([0, 1, 151]), rows, 150, key_mask=mask)
    for b, at in ((0, 0), (1, 90)):
        want = v[at].repeat_interleave(2, 0).expand(rows, 4, d)
        assert torch.equal(out[b * rows:(b + 1) * rows], want)


@pytest.mark.parametrize("rows", [5, 80])
def test_nan_in_seen_places_reaches_its_rows(rows):
    q, k, v = inputs(9, [rows, rows], [300, 200], 4, 2, 64, "bf16")
    q[2] = math.nan
    k[310, 1] = math.nan
    v[5, 0, 3] = math.nan
    out, lse = pa.pa_fwd_cross(q, k, v, i32([0, rows, 2 * rows]), i32([0, 300, 500]), rows, 300)
    bad = torch.isnan(out.float())
    want = torch.zeros_like(bad)
    want[2] = True
    want[rows:, 2:] = True
    want[:rows, :2, 3] = True
    assert torch.equal(bad, want)
    want = torch.zeros_like(lse, dtype=torch.bool)
    want[:, 2] = True
    want[2:, rows:] = True
    assert torch.equal(torch.isnan(lse), want)


@pytest.mark.parametrize("dtype,d", [("f16", 64), ("bf16", 64), ("f16", 128), ("bf16", 128)])
@pytest.mark.parametrize("keys", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 511, 640])
def test_key_counts(keys, dtype, d):
    check([3, 2], [keys, max(1, keys - 1)], 4, 4, d, dtype, seed=keys)


@pytest.mark.parametrize("dtype,d", [("f16", 64), ("bf16", 128)])
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 15, 16, 17, 24, 31, 32, 33, 48, 63, 64, 65, 100, 127, 128,
                                  129, 200, 255, 256, 257, 300])
def test_row_counts(rows, dtype, d):
    check([rows, 1, max(1, rows // 2)], [70, 129, 200], 4, 2, d, dtype, seed=rows, spare=2)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows", [[4, 2, 3, 1], [40, 3, 64, 1], [300, 2, 129, 1]])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (4, 4, 128)])
def test_masks(hq, hkv, d, rows, dtype):
    """Masked keys hold NaN, infinities and the type's lowest value; an entry has no key at all."""
    keys = [70, 129, 40, 300]
    q, k, v = inputs(3, rows, keys, hq, hkv, d, dtype)
    g = torch.Generator().manual_seed(8)
    mask = torch.rand(sum(keys), generator=g) < 0.6
    mask[70:70 + 64] = False    # whole tiles
    mask[199:239] = False       # a whole entry
    mask[239:240] = True
    mask = mask.to(DEV)
    gone = torch.where(~mask)[0]
    for i, bad in enumerate((math.nan, math.inf, -math.inf, torch.finfo(q.dtype).min)):
        k[gone[i::4]], v[gone[i::4]] = bad, bad
    for m in (mask, mask.to(torch.uint8) * 255):
        out, lse = pa.pa_fwd_cross(q, k, v, i32(cu_of(rows)), i32(cu_of(keys)), max(rows), 300,
                                   key_mask=m)
        compare(out, lse, q, k, v, cu_of(rows), cu_of(keys), mask=mask)
    at = slice(cu_of(rows)[2], cu_of(rows)[3])
    assert (out[at] == 0).all() and (lse[:, at] == -math.inf).all()
    # a single key that is seen, at either end of a tile
    for one in (0, 15, 31, 32, 63, 64, 127, 128, 299):
        m = torch.zeros(300, dtype=torch.bool, device=DEV)
        m[one] = True
        qq = torch.randn((5, hq, d), generator=g).to(q.dtype).to(DEV)
        kk = torch.full((300, hkv, d), math.nan, dtype=q.dtype, device=DEV)
        kk[one] = torch.randn((hkv, d), generator=g).to(q.dtype).to(DEV)
        o, _ = pa.pa_fwd_cross(qq, kk, kk, i32([0, 5]), i32([0, 300]), max(rows + [5]), 300,
                               key_mask=m)
        assert torch.equal(o, kk[one].repeat_interleave(hq // hkv, 0).expand_as(o))


@pytest.mark.parametrize("rows", [[3, 3, 3], [90, 20, 150]])
def test_padded_batches_and_neighbours(rows):
    """seqlens_k within slots of one length; what lies behind a length is NaN."""
    lens = [50, 128, 1]
    q, k, v = inputs(5, rows, [128] * 3, 4, 2, 64, "f16")
    for b, n in enumerate(lens):
        k[128 * b + n:128 * b + 128] = math.nan
        v[128 * b + n:128 * b + 128] = math.nan
    out, lse = pa.pa_fwd_cross(q, k, v, i32(cu_of(rows)), i32([0, 128, 256, 384]), max(rows), 128,
                               seqlens_k=i32(lens))
    mask = torch.cat([torch.arange(128) < n for n in lens])
    compare(out, lse, q, k, v, cu_of(rows), [0, 128, 256, 384], lens_k=lens, mask=mask.to(DEV))
    # keys in front of and behind an entry belong to others
    out, _ = pa.pa_fwd_cross(q[:2], k, v, i32([0, 2]), i32([128, 256]), 2, 128)
    o2, _ = pa.pa_fwd_cross(q[:2], k[128:256], v[128:256], i32([0, 2]), i32([0, 128]), 2, 128)
    assert torch.isfinite(out).all() and torch.equal(out, o2)


@pytest.mark.parametrize("rows", [6, 70, 150])
def test_strides(rows):
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn((rows, 3, 12, 64), generator=g).half().to(DEV)
    kv = torch.randn((90, 5, 2, 64 + 8), generator=g).half().to(DEV)
    q, k, v = qkv[:, 1, 2:10], kv[:, 1:5, 0, :64], kv[:, 1:5, 1, 8:]
    out, lse = pa.pa_fwd_cross(q, k, v, i32([0, rows]), i32([0, 90]), rows, 90, scale=0.3)
    compare(out, lse, q, k, v, [0, rows], [0, 90], scale=0.3)
    # heads in another order of memory than tokens; one head, one key
    q, k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
    out, lse = pa.pa_fwd_cross(q, k, v, i32([0, rows]), i32([0, 90]), rows, 90)
    compare(out, lse, q, k, v, [0, rows], [0, 90])
    out, lse = pa.pa_fwd_cross(q[:, :2], k[:1, :1], v[:1, :1], i32([0, rows]), i32([0, 1]), rows, 1)
    compare(out, lse, q[:, :2], k[:1, :1], v[:1, :1], [0, rows], [0, 1])
    # every key alike: the mean of V, here 1
    one = torch.ones((1, 4, 64), dtype=torch.float16, device=DEV).expand(90, 4, 64).contiguous()
    out, _ = pa.pa_fwd_cross(q, k, one, i32([0, rows]), i32([0, 90]), rows, 90)
    assert (out.float() - 1).abs().max().item() <= 2 * 2.0 ** -11


@pytest.mark.parametrize("rows", [5, 80, 200])
def test_large_scores(rows):
    """Scores that grow along the keys: the running maximum moves in every tile."""
    g = torch.Generator().manual_seed(4)
    q = torch.randn((rows, 4, 64), generator=g).abs().half().to(DEV)
    k = (torch.linspace(-4, 4, 700)[:, None, None] * torch.ones(700, 2, 64)).half().to(DEV)
    v = torch.randn((700, 2, 64), generator=g).half().to(DEV)
    for kk in (k, k.flip(0)):
        out, lse = pa.pa_fwd_cross(q, kk, v, i32([0, rows]), i32([0, 700]), rows, 700)
        o, l = beam.cross(np64(q), np64(kk), np64(v), [0, rows], [0, 700])
        # |score| < 40: 65 * 2^-24 * 40 of it; fp16 P
        assert np.abs(np64(out) - o).max() <= 2 * 2.0 ** -11 * np.abs(np64(v)).max()
        assert np.abs(np64(lse) - l).max() <= 65 * 2.0 ** -24 * 60 + 1e-5


def test_malformed_entries_are_reported():
    q, k, v = inputs(6, [4, 4, 4], [50, 50, 50], 4, 2, 64, "f16")
    ok = [0, 4, 8, 12], [0, 50, 100, 150], [50, 50, 50]
    for bad, which in (([0, 4, 8, 13], 0), ([0, 4, 2, 12], 0), ([0, 50, 100, 151], 1),
                       ([0, -1, 100, 150], 1), ([50, 51, 50], 2), ([50, 50, -1], 2)):
        a = [list(x) for x in ok]
        a[which] = bad
        err = pa.new_err_word(DEV)
        out = torch.full_like(q, 7.0)
        # (the keys that count are the first seqlens_k where that is given)
        lens = i32(a[2]) if which != 1 else None
        pa.pa_fwd_cross(q, k, v, i32(a[0]), i32(a[1]), 4, 51, seqlens_k=lens, out=out, err=err)
        torch.cuda.synchronize()
        assert err[0].item() == pa.PA_DEVERR_LENGTH
        assert torch.isfinite(out).all()
    for mq, mk in ((3, 50), (4, 49)):
        err = pa.new_err_word(DEV)
        pa.pa_fwd_cross(q, k, v, i32(ok[0]), i32(ok[1]), mq, mk, err=err)
        assert err[0].item() == pa.PA_DEVERR_LENGTH
    # no keys at all, no rows at all
    out, lse = pa.pa_fwd_cross(q, k[:0], v[:0], i32(ok[0]), i32([0] * 4), 4, 0)
    assert (out == 0).all() and (lse == -math.inf).all()
    out, _ = pa.pa_fwd_cross(q[:0], k, v, i32([0, 0]), i32([0, 50]), 0, 50)
    assert out.shape == (0, 4, 64)
    out = torch.full_like(q, 7.0)
    pa.pa_fwd_cross(q, k, v, i32([0, 0]), i32([0, 50]), 4, 50, out=out)
    assert (out == 7.0).all()


@pytest.mark.parametrize("rows", [4, 60, 180])
def test_streams_and_graph_replays(rows):
    q, k, v = inputs(7, [rows, 3], [300, 90], 8, 4, 64, "bf16")
    cu_q, cu_k = i32([0, rows, rows + 3]), i32([0, 300, 390])
    mask = torch.ones(390, dtype=torch.bool, device=DEV)
    args = (q, k, v, cu_q, cu_k, rows, 300)
    ref, _ = pa.pa_fwd_cross(*args, key_mask=mask)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, _ = pa.pa_fwd_cross(*args, key_mask=mask)
    out, lse = torch.empty_like(ref), torch.empty((8, rows + 3), device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_fwd_cross(*args, key_mask=mask, out=out, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ref, got) and torch.equal(ref, out)
    # other lengths and masks within the same bounds
    cu_k.copy_(i32([0, 100, 390]))
    cu_q.copy_(i32([0, 2, rows + 2]))
    mask[10::3] = False
    out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    compare(out[:rows + 2], lse[:, :rows + 2], q[:rows + 2], k, v, [0, 2, rows + 2], [0, 100, 390],
            mask=mask)
    assert (out[rows + 2] == 7.0).all()
