"""pa_rotary_append_varlen against the oracle in 64 bits.

Tolerances.  A rotated value is x1 c - x2 s in fp32: one product rounded, then one fused
operation, so its error is at most 2^-24 (|x1 c| + |x2 s|) twice over.  It is rounded once to the
stored type, by at most half a step: 2^-11 of the value for fp16 (2^-25 below its normal range),
2^-8 for bf16.  An e4m3 value is the rounding of y r, r the fp32 reciprocal of the scale: r is off
by half a unit, 2^-24, and the product by another, so x / scale is off by (1 + 2^-24)^2 - 1 < 2^-22
of itself besides y's own error, and the value lies between the roundings of the two ends of that
interval.  Values that do not turn are copied bit by bit; their y has no error.
"""

import numpy as np
import pytest
import torch

import paged_kv_cache_page_gb300 as pa
from oracle import serving as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def np64(t):
    return t.detach().cpu().double().numpy()


def inputs(T, hq, hkv, d, dtype, cache, page, axes, rot, seed=0, length=200, pages=None, table=None):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    qkv = torch.randn((T, hq + 2 * hkv + 1, d), generator=g).to(dt).to(DEV)
    pages = sv.pages_of(max(T, 1), page) + 2 if pages is None else pages
    base = torch.randn((2, pages, page, hkv, d), generator=g)
    base = (base.to(torch.float8_e4m3fn) if cache == "e4m3" else base.to(dt)).to(DEV)
    slots = torch.randperm(pages * page, generator=g)[:T].to(DEV)
    pos = torch.randint(0, length, (axes, T), generator=g).to(torch.int32).to(DEV)
    ang = torch.arange(length).double()[:, None] * 10000.0 ** (-torch.arange(0, rot, 2).double() / d)
    tdt = dt if table is None else table
    pair = [(3 * p + p // 2) % axes for p in range(rot // 2)]
    scale = [0.01 + 0.02 * torch.rand(hkv, generator=g).to(DEV) for _ in range(2)]
    return dict(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:hq + 2 * hkv],
                k_cache=base[0], v_cache=base[1], slots=slots, pos=pos, cos=ang.cos().to(tdt).to(DEV),
                sin=ang.sin().to(tdt).to(DEV), pair=pair, scale=scale if cache == "e4m3" else [None] * 2)


def call(w, inter, q_out=None, err=None, **kw):
    a = dict(positions=w["pos"], rotary_cos=w["cos"], rotary_sin=w["sin"], rotary_interleaved=inter,
             pair_axis=w["pair"], k_scale=w["scale"][0], v_scale=w["scale"][1], q_out=q_out, err=err)
    a.update(kw)
    return pa.pa_rotary_append_varlen(w["q"], w["k"], w["v"], w["k_cache"], w["v_cache"], w["slots"],
                                      **a)


def turned(w, name, inter):
    """(rotated values, their fp32 error bound) in 64 bits."""
    pos, cos, sin = w["pos"].cpu().tolist(), np64(w["cos"]), np64(w["sin"])
    x = np64(w[name])
    y = sv.rotary_axes(x, cos, sin, pos, w["pair"], inter)
    # |x1 c| + |x2 s| of each value, by the same rotation of magnitudes
    big = sv.rotary_axes(np.abs(x), np.abs(cos), np.abs(sin), pos, w["pair"], inter)
    half = cos.shape[1]
    first = [2 * p if inter else p for p in range(half)]
    second = [2 * p + 1 if inter else p + half for p in range(half)]
    a = np.abs(x)
    for t in range(x.shape[0]):
        for p in range(half):
            at = pos[w["pair"][p]][t]
            if 0 <= at < cos.shape[0]:
                big[t, :, first[p]] = (a[t, :, first[p]] * abs(cos[at, p])
                                       + a[t, :, second[p]] * abs(sin[at, p]))
    big[..., 2 * half:] = 0
    return y, big * 2.0 ** -23


def check_cache(got, before, rows, off, slots, scale, dtype, page):
    want = np64(before).reshape(-1, *rows.shape[1:])
    lo = want.copy()
    hi = want.copy()
    for t, s in enumerate(slots):
        if s < 0:
            continue
        for side, sign in ((lo, -1), (hi, 1)):
            x = rows[t] + sign * off[t]
            if scale is not None:
                x = sv.e4m3(x / np64(scale)[:, None] * (1 + sign * np.sign(x) * 2.0 ** -22))
            side[s] = x
    x = np64(got).reshape(lo.shape)
    room = 0 if scale is not None else HALF[dtype] * np.maximum(np.abs(lo), np.abs(hi)) + 2.0 ** -25
    written = np.zeros(len(lo), bool)
    written[[s for s in slots if s >= 0]] = True
    assert np.array_equal(x[~written], want[~written])
    assert (x >= lo - room).all() and (x <= hi + room).all()


CASES = [
    # T, hq, hkv, d, dtype, cache, page, axes, rot, interleaved
    (1, 4, 2, 64, "f16", "f16", 16, 1, 64, False),
    (1, 1, 1, 128, "bf16", "e4m3", 16, 1, 128, False),
    (7, 32, 8, 128, "bf16", "e4m3", 16, 3, 128, False),
    (33, 12, 12, 64, "f16", "f16", 32, 3, 32, True),
    (33, 12, 12, 64, "bf16", "bf16", 64, 2, 48, False),
    (100, 5, 1, 64, "f16", "e4m3", 256, 4, 64, True),
    (257, 8, 8, 128, "f16", "e4m3", 128, 2, 64, False),
    (19, 3, 3, 128, "bf16", "bf16", 16, 1, 16, True),
    # widths that are no multiple of 16 features
    (5, 4, 2, 64, "f16", "f16", 16, 1, 2, False),
    (9, 4, 2, 64, "bf16", "e4m3", 16, 3, 20, False),
    (9, 2, 1, 128, "f16", "bf", 16, 2, 120, True),
    (300, 2, 2, 128, "bf16", "e4m3", 32, 2, 36, True),
]


@pytest.mark.parametrize("table", [None, torch.float32])
@pytest.mark.parametrize("case", CASES)
def test_against_the_oracle(case, table):
    T, hq, hkv, d, dtype, cache, page, axes, rot, inter = case
    cache = dtype if cache == "bf" else cache
    w = inputs(T, hq, hkv, d, dtype, cache, page, axes, rot, seed=T + d, table=table)
    if T > 4:
        w["slots"][1] = -1
        w["slots"][3] = -(2 ** 40)
    before = [w["k_cache"].clone(), w["v_cache"].clone()]
    err = pa.new_err_word(DEV)
    q_out = call(w, inter, err=err)
    torch.cuda.synchronize()
    assert err[0].item() == 0
    y, off = turned(w, "q", inter)
    room = off + HALF[dtype] * (np.abs(y) + off) + 2.0 ** -25
    assert (np.abs(np64(q_out) - y) <= room).all()
    assert torch.equal(q_out[..., rot:], w["q"][..., rot:])
    slots = w["slots"].tolist()
    y, off = turned(w, "k", inter)
    check_cache(w["k_cache"], before[0], y, off, slots, w["scale"][0], dtype, page)
    v = np64(w["v"])
    check_cache(w["v_cache"], before[1], v, 0 * v, slots, w["scale"][1], dtype, page)


def test_values_at_the_ends_of_the_range():
    """Saturation, infinities, NaN, zeros of both signs and subnormal quotients in an e4m3 cache."""
    w = inputs(16, 2, 1, 64, "bf16", "e4m3", 16, 1, 64, pages=1)
    special = [0.0, -0.0, 448.0, 464.0, 470.0, -1e30, float("inf"), -float("inf"), float("nan"),
               2.0 ** -9, 2.0 ** -10, 2.0 ** -11, 3 * 2.0 ** -10, 2.0 ** -133, 1.0625, -17.0]
    w["v"][0, 0, :16] = torch.tensor(special, dtype=torch.bfloat16, device=DEV)
    w["scale"][1] = torch.ones(1, device=DEV)
    call(w, False)
    got = w["v_cache"].view(-1, 64)[w["slots"][0], :16].double().cpu().numpy()
    want = sv.e4m3(w["v"][0, 0, :16].double().cpu().numpy())
    assert np.array_equal(got, want, equal_nan=True)
    assert np.signbit(got[1]) and not np.signbit(got[0])


def test_in_place_no_rotation_and_no_q():
    w = inputs(21, 4, 2, 128, "bf16", "bf16", 16, 2, 128)
    want = call(w, False)
    kc, vc = w["k_cache"].clone(), w["v_cache"].clone()
    # in place on a slice of the projection
    q = w["q"]
    assert not q.is_contiguous()
    assert call(w, False, q_out=q) is q
    assert torch.equal(q, want)
    # k and v alone give the same caches
    w["k_cache"].zero_()
    w["v_cache"].zero_()
    w2 = dict(w, q=None)
    assert call(w2, False) is None
    at = w["slots"]
    assert torch.equal(w["k_cache"].view(-1, 2, 128)[at], kc.view(-1, 2, 128)[at])
    assert torch.equal(w["v_cache"].view(-1, 2, 128)[at], vc.view(-1, 2, 128)[at])
    # without tables everything is copied
    out = call(w, False, positions=None, rotary_cos=None, rotary_sin=None, pair_axis=None)
    assert torch.equal(out, w["q"])
    assert torch.equal(w["k_cache"].view(-1, 2, 128)[at], w["k"])


def test_strided_caches_and_positions():
    """Caches that are head slices of a wider pool, positions that are rows of a wider tensor."""
    w = inputs(40, 4, 2, 64, "f16", "e4m3", 32, 2, 64)
    call(w, True)
    ref = [w["k_cache"].clone(), w["v_cache"].clone()]
    wide = torch.zeros((ref[0].shape[0], 32, 7, 64), device=DEV).to(torch.float8_e4m3fn)
    pos = torch.zeros((2, 99), dtype=torch.int32, device=DEV)
    pos[:, 5:45] = w["pos"]
    w2 = dict(w, k_cache=wide[:, :, 1:3], v_cache=wide[:, :, 4:6], pos=pos[:, 5:45])
    call(w2, True)
    at = w["slots"]
    for got, want in ((wide[:, :, 1:3], ref[0]), (wide[:, :, 4:6], ref[1])):
        g8, w8 = got.contiguous().view(torch.uint8), want.view(torch.uint8)
        assert torch.equal(g8.view(-1, 2, 64)[at], w8.view(-1, 2, 64)[at])
    for h in (0, 3, 6):
        assert (wide[:, :, h].contiguous().view(torch.uint8) == 0).all()


@pytest.mark.parametrize("rot", [64, 20])
def test_positions_and_slots_outside_are_reported(rot):
    w = inputs(6, 2, 1, 64, "f16", "f16", 16, 2, rot, length=50)
    w["pos"][1, 2] = 50
    err = pa.new_err_word(DEV)
    out = call(w, False, err=err)
    assert err.tolist()[:3] == [pa.PA_DEVERR_LENGTH, 2, 50]
    assert torch.equal(out[2], w["q"][2])
    assert torch.equal(w["k_cache"].view(-1, 1, 64)[w["slots"][2]], w["k"][2])
    y, off = turned(w, "q", False)
    assert (np.abs(np64(out) - y) <= off + HALF["f16"] * (np.abs(y) + off) + 2.0 ** -25).all()
    w["pos"][1, 2] = 0
    before = w["k_cache"].clone()
    w["slots"][4] = before.shape[0] * 16
    err = pa.new_err_word(DEV)
    call(w, False, err=err)
    assert err.tolist()[:3] == [pa.PA_DEVERR_PAGE_OOB, 4, before.shape[0]]


def test_many_tokens_and_long_offsets():
    """More tokens than warps in flight, and slots beyond 2^31 elements of the cache."""
    T, hkv, d, page = 9000, 2, 128, 16
    pages = (1 << 31) // (page * hkv * d) + 600
    w = inputs(T, 3, hkv, d, "bf16", "e4m3", page, 1, d, length=64, pages=1)
    pools = [torch.zeros((pages, page, hkv, d), dtype=torch.float8_e4m3fn, device=DEV)
             for _ in range(2)]
    slots = torch.arange(T, device=DEV) + (pages - 580) * page
    w2 = dict(w, k_cache=pools[0], v_cache=pools[1], slots=slots)
    call(w2, False)
    small = [torch.zeros((T // page + 1, page, hkv, d), dtype=torch.float8_e4m3fn, device=DEV)
             for _ in range(2)]
    call(dict(w, k_cache=small[0], v_cache=small[1], slots=torch.arange(T, device=DEV)), False)
    for big, few in zip(pools, small):
        got = big.view(torch.uint8).view(-1, hkv, d)[slots]
        assert torch.equal(got, few.view(torch.uint8).view(-1, hkv, d)[:T])
    x, got = np64(w["v"][-1]) / np64(w["scale"][1])[:, None], np64(pools[1].view(-1, hkv, d)[slots[-1]])
    ends = np.sort([sv.e4m3(x * (1 - 2.0 ** -22)), sv.e4m3(x * (1 + 2.0 ** -22))], axis=0)
    assert (ends[0] <= got).all() and (got <= ends[1]).all()


def test_replay_and_other_stream():
    w = inputs(50, 8, 2, 64, "bf16", "e4m3", 16, 3, 64)
    out = torch.zeros((50, 8, 64), dtype=torch.bfloat16, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(w, False, q_out=out)
    w["pos"].copy_(w["pos"].flip(1))
    g.replay()
    torch.cuda.synchronize()
    kc = w["k_cache"].clone()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        eager = call(w, False)
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    assert torch.equal(kc.view(torch.uint8), w["k_cache"].view(torch.uint8))
