"""What reaches a result of pa_fwd_varlen_e4m3: small probabilities beside large ones in one tile, NaN
in keys, values and queries across splits, offsets that are not cumulative lengths, calls side by side."""

import math
import threading

import pytest
import torch

import paged_kv_cache_page_gb300 as pa
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


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("q_lens,k_lens,heads", [
    ([1, 3, 1, 9], [70, 300, 1000, 9], (4, 2, 64)),       # whole streams
    ([2, 1], [20011, 9000], (8, 2, 128)),                 # split streams
    ([100, 260], [100, 400], (4, 2, 64)),                 # chunks
    ([150, 1], [9001, 3000], (2, 1, 128)),                # split chunks beside a single token
])
def test_nan_and_infinity_in_a_row_of_q_stay_there(q_lens, k_lens, heads, dtype, bad):
    w = batch(q_lens, k_lens, *heads, dtype, seed=len(q_lens))
    clean, clean_l = call(w)
    q = w["q"].clone()
    # rows that see several keys
    hit = [(q_lens[0] // 2, 1), (q_lens[0] - 1, heads[0] - 1), (q_lens[0], 0),
           (sum(q_lens) - 1, heads[0] - 1)]
    for r, h in hit:
        q[r, h, 11] = bad
    out, lse = call(dict(w, q=q))
    mask = torch.zeros(out.shape[:2], dtype=torch.bool, device=DEV)
    for r, h in hit:
        mask[r, h] = True
    # each of these rows has a score that is NaN or plus infinity: exp(s - max) is NaN
    assert torch.isnan(out[mask]).all() and torch.isnan(lse.T[mask]).all()
    out, lse = out.clone(), lse.clone()
    out[mask] = clean[mask]
    lse.T[mask] = clean_l.T[mask]
    check(w, out, lse)


@pytest.mark.parametrize("cu,like", [([0, 5, 3], [0, 3, 3]), ([-4, 1, 99], [0, 1, 3]), ([2, 2, 2], None),
                                     ([1, 2, 3], None)])
def test_offsets_outside_the_rows_write_nothing_outside(cu, like):
    w = batch([1, 2], [100, 60], 4, 2, 64, "f16", seed=11)
    wide, wide_l = torch.full((9, 4, 64), 7.0, device=DEV).half(), torch.full((3 * 4 * 3,), 7.0, device=DEV)
    out, lse = wide[3:6], wide_l[12:24].view(4, 3)
    w["cu_seqlens_q"].copy_(torch.tensor(cu, dtype=torch.int32))
    call(w, out=out, lse=lse)
    assert (wide[:3] == 7).all() and (wide[6:] == 7).all()
    assert (wide_l[:12] == 7).all() and (wide_l[24:] == 7).all()
    if like is not None:
        w["cu_seqlens_q"].copy_(torch.tensor(like, dtype=torch.int32))
        want, want_l = call(w)
        assert torch.equal(out, want) and torch.equal(lse, want_l)
    else:
        assert (out[:cu[0]] == 7).all() and (lse[:, :cu[0]] == 7).all()
        if cu[2] == cu[0]:
            assert (out == 7).all() and (lse == 7).all()


def test_threads_and_streams_with_chunks_at_once():
    """Two host threads, a stream each, with chunks and single tokens; every call with a workspace of its
    own from the allocator."""
    ws = [batch([1, 70, 1, 200], [3000, 500, 1500, 200], 8, 2, 128, "bf16", seed=20),
          batch([300, 1, 40], [2000, 700, 40], 4, 4, 64, "f16", seed=21)]
    want = [call(w) for w in ws]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(25):
                    o, l = call(ws[i])
                    if not (torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])):
                        wrong.append(i)
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
