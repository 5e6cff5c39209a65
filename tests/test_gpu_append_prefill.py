"""The forms of pa_rotary_append_varlen that a whole prefill step runs: several rows of a tensor in
flight a thread, one warp for a token's k, v and q; against the oracle on sampled tokens, and in place.
Tolerances: test_gpu_rotary_append."""

import numpy as np
import pytest
import torch

from test_gpu_rotary_append import DEV, HALF, call, check_cache, inputs, np64, turned

pytestmark = pytest.mark.gpu

# T, hq, hkv, d, dtype, cache, page, axes, rot, interleaved: 1 to 7 of 8 (or of 3, of 6) parts a token
CASES = [
    (1300, 32, 8, 128, "bf16", "e4m3", 16, 3, 128, False),
    (5000, 32, 8, 128, "f16", "e4m3", 64, 1, 128, True),
    (9800, 32, 8, 128, "bf16", "bf16", 32, 3, 128, False),
    (5001, 24, 8, 128, "f16", "f16", 16, 2, 64, True),
    (7001, 20, 4, 128, "bf16", "e4m3", 256, 3, 96, True),
    (6000, 12, 12, 64, "bf16", "e4m3", 16, 3, 64, False),
    (9999, 12, 12, 64, "f16", "f16", 128, 2, 32, True),
    (9999, 5, 3, 128, "bf16", "e4m3", 16, 4, 48, False),
]


@pytest.mark.parametrize("case", CASES)
def test_prefill_against_the_oracle_and_in_place(case):
    T, hq, hkv, d, dtype, cache, page, axes, rot, inter = case
    w = inputs(T, hq, hkv, d, dtype, cache, page, axes, rot, seed=T)
    w["slots"][3] = -1
    before = [w["k_cache"].clone(), w["v_cache"].clone()]
    q_out = call(w, inter)
    rng = np.random.RandomState(T)
    rows = np.unique(np.concatenate([np.arange(3), T - 1 - np.arange(5), rng.randint(4, T, 30)]))
    at = torch.from_numpy(rows).to(DEV)
    few = dict(w, q=w["q"][at], k=w["k"][at], v=w["v"][at], pos=w["pos"][:, at])
    y, off = turned(few, "q", inter)
    room = off + HALF[dtype] * (np.abs(y) + off) + 2.0 ** -25
    assert (np.abs(np64(q_out[at]) - y) <= room).all()
    assert torch.equal(q_out[..., rot:], w["q"][..., rot:])
    # the slots of the sampled tokens, as small caches
    slots, live = w["slots"][at], list(range(len(rows)))
    yk, offk = turned(few, "k", inter)
    v = np64(few["v"])
    for name, was, x, o in (("k_cache", before[0], yk, offk), ("v_cache", before[1], v, 0 * v)):
        pick = lambda c: c.view(torch.uint8 if cache == "e4m3" else torch.int16).view(  # noqa: E731
            -1, hkv, d)[slots].view(c.dtype)
        check_cache(pick(w[name]), pick(was), x, o, live, w["scale"][name == "v_cache"], dtype, page)
    # every slot of nobody stays
    idle = torch.ones(before[0].shape[0] * page, dtype=torch.bool, device=DEV)
    idle[w["slots"][w["slots"] >= 0]] = False
    raw = torch.uint8 if cache == "e4m3" else torch.int16
    for name, was in zip(("k_cache", "v_cache"), before):
        assert torch.equal(w[name].view(raw).view(-1, hkv, d)[idle], was.view(raw).view(-1, hkv, d)[idle])
    # in place: the same q, the same caches
    first = [w[n].clone() for n in ("k_cache", "v_cache")]
    for n, b in zip(("k_cache", "v_cache"), before):
        w[n].copy_(b)
    assert call(w, inter, q_out=w["q"]) is w["q"]
    assert torch.equal(w["q"], q_out)
    for n, x in zip(("k_cache", "v_cache"), first):
        assert torch.equal(w[n].view(raw), x.view(raw))


@pytest.mark.parametrize("T", [3, 700])
@pytest.mark.parametrize("rot,inter", [(20, False), (36, True), (2, False)])
def test_in_place_at_widths_of_single_pairs(T, rot, inter):
    w = inputs(T, 6, 2, 64, "f16", "e4m3", 16, 2, rot, seed=rot)
    want = call(w, inter)
    assert call(w, inter, q_out=w["q"]) is w["q"]
    assert torch.equal(w["q"], want)
