"""The operators of a serving step together: plan, rotary append, attention, release, over several
steps of a ragged batch, against keys and values kept as plain lists."""

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_page_gb300 as pa
from oracle import serving as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HQ, HKV, D, PAGE, B, POOL, CAP = 8, 2, 64, 16, 4, 40, 96


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("e4m3", [True, False])
def test_serving_steps(e4m3):
    g = torch.Generator().manual_seed(5)
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    caches = [torch.zeros((POOL, PAGE, HKV, D), device=DEV).to(kind) for _ in range(2)]
    scale = [torch.full((HKV,), s, device=DEV) if e4m3 else None for s in (0.02, 0.01)]
    lens, table = i32([0] * B), i32([[-1] * 20] * B)
    pool, count, err = i32(list(range(POOL))), i32([POOL]), pa.new_err_word(DEV)
    length = 400
    ang = torch.arange(length).double()[:, None] * 100.0 ** (-torch.arange(0, D, 2).double() / D)
    cos, sin = ang.cos().float().to(DEV), ang.sin().float().to(DEV)
    keys, values = [[] for _ in range(B)], [[] for _ in range(B)]
    steps = [([30, 0, 1, 40], None), ([1, 20, 1, 1], None), ([1, 1, 50, 1], [32, 21, 0, 40]),
             ([1, 1, 0, 1], None), ([9, 60, 1, 3], [0, 22, 50, 43]), ([1, 1, 1, 1], None)]
    for new, keep in steps:
        if keep is not None:
            pa.pa_release_pages(lens, i32(keep), table, pool, count, PAGE, err=err)
            for b in range(B):
                del keys[b][keep[b]:], values[b][keep[b]:]
        cu, lk, slots, pos = pa.pa_plan_step(lens, i32(new), table, pool, count, PAGE,
                                             token_capacity=CAP, err=err)
        qkv = torch.randn((CAP, HQ + 2 * HKV, D), generator=g).to(torch.bfloat16).to(DEV)
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        q = pa.pa_rotary_append_varlen(q, k, v, *caches, slots, positions=pos, rotary_cos=cos,
                                       rotary_sin=sin, k_scale=scale[0], v_scale=scale[1], err=err)
        if e4m3:
            out, lse = pa.pa_fwd_varlen_e4m3(q, *caches, cu, lk, table, CAP, 320, k_scale=scale[0],
                                             v_scale=scale[1], err=err)
        else:
            out, lse = pa.pa_fwd_varlen_unified(q, *caches, cu, lk, table, CAP, 320, err=err)
        torch.cuda.synchronize()
        assert err[0].item() == 0, err.tolist()
        lens = lk
        # the same step on lists
        rows = np.concatenate([[0], np.cumsum(new)])
        assert cu.tolist() == rows.tolist()
        cd, sd = cos.double().cpu().numpy(), sin.double().cpu().numpy()
        at = [[len(keys[b]) + i for b in range(B) for i in range(new[b])]]
        turn = lambda x: sv.rotary_axes(x[:rows[-1]].double().cpu().numpy(), cd, sd, at,  # noqa: E731
                                        [0] * (D // 2), False)
        kt, vt = turn(qkv[:, HQ:HQ + HKV]), qkv[:rows[-1], HQ + HKV:].double().cpu().numpy()
        # what the cache holds of them: exactly the stored values, at most a rounding away
        for b in range(B):
            for i in range(rows[b], rows[b + 1]):
                s = slots[i].item()
                got = [c.view(-1, HKV, D)[s].double().cpu().numpy() *
                       (1.0 if x is None else x.double().cpu().numpy()[:, None])
                       for c, x in zip(caches, scale)]
                step = 2.0 ** -4 if e4m3 else 2.0 ** -8
                tiny = 2.0 ** -10 * 0.02 if e4m3 else 2.0 ** -20
                for x, y in zip(got, (kt[i], vt[i])):
                    assert (np.abs(x - y) <= step * 1.001 * np.abs(y) + tiny).all()
                keys[b].append(got[0])
                values[b].append(got[1])
        qt = q.double().cpu().numpy()
        for b in range(B):
            assert lens[b].item() == len(keys[b])
            if new[b] == 0:
                continue
            o, l = oracle.attend_rows(qt[rows[b]:rows[b + 1]], np.array(keys[b]),
                                      np.array(values[b]), D ** -0.5, True)
            assert np.abs(out[rows[b]:rows[b + 1]].double().cpu().numpy() - o).max() <= 1.6e-2
            assert np.abs(lse[:, rows[b]:rows[b + 1]].double().cpu().numpy() - l).max() <= 1e-3
    held = sum(sv.pages_of(len(x), PAGE) for x in keys)
    assert count.item() == POOL - held
