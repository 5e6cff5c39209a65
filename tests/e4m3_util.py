"""Inputs of ragged batches over a paged e4m3 cache, and the check of an attention result.

Tolerances, in 64 bits from each row's own values.  Let A = sum_t p_t |v_t| / l, the result for
|V|, and S = max_t scale |q| . |k_t|, the largest possible score.
  scores          fp32 sums of D exact products in D / 16 MMAs, each of which may cut 2^-22 of the
                  magnitudes it adds (17 sums for D = 128), and one fused operation: 2^-17 S; each
                  value of a bf16 row of q also loses what lies 2^-25 below the row's largest:
                  2^-24 Q, with Q = scale max|q| max_t sum|k_t|
  probabilities   e^score (2^-21), rounded to fp16: 2^-11; relative
  products        fp32 sums over the keys in MMAs of 16: n / 16 cuts of 2^-22 A; merges 2^-20 A
  result          one rounding to the type: half a step of |O| (fp16: 2^-25 below its range)
so |dO| <= (2 (2^-17 S + 2^-24 Q) + 2^-11 + n 2^-26 + 2^-19) A + half |O|, and
|dLSE| <= 2^-17 S + 2^-24 Q + n 2^-24 + 2^-20 + 2^-23 |LSE|.
"""

import numpy as np
import torch

import oracle
import paged_kv_cache_page_gb300 as pa

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
DEV = "cuda:0"


def batch(q_lens, k_lens, hq, hkv, d, dtype, page=16, seed=0, extra=3, peaky=1.0):
    g = torch.Generator().manual_seed(seed)
    held = [-(-k // page) for k in k_lens]
    pool = sum(held) + extra
    order = torch.randperm(pool, generator=g).to(torch.int32)
    width = max([1] + held) + 1
    table = torch.full((len(k_lens), width), -1, dtype=torch.int32)
    off = 0
    for b, n in enumerate(held):
        table[b, :n] = order[off:off + n]
        off += n
    cu = np.concatenate([[0], np.cumsum(q_lens)]).tolist()
    scale = [(0.5 + torch.rand(hkv, generator=g)) * (4.5 / 448) for _ in range(2)]
    kv = [(torch.randn((pool, page, hkv, d), generator=g) / s[:, None]).clamp(-448, 448)
          .to(torch.float8_e4m3fn).to(DEV) for s in scale]
    q = (torch.randn((cu[-1], hq, d), generator=g) * peaky).to(DT[dtype]).to(DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(q=q, k_cache=kv[0], v_cache=kv[1], k_scale=scale[0].to(DEV),
                v_scale=scale[1].to(DEV), cu_seqlens_q=i32(cu), seqlens_k=i32(k_lens),
                block_table=table.to(DEV), max_seqlen_q=max([0] + list(q_lens)),
                max_seqlen_k=max([0] + list(k_lens)), dtype=dtype, q_lens=list(q_lens),
                k_lens=list(k_lens))


def call(w, **kw):
    a = dict(k_scale=w["k_scale"], v_scale=w["v_scale"])
    a.update(kw)
    return pa.pa_fwd_varlen_e4m3(w["q"], w["k_cache"], w["v_cache"], w["cu_seqlens_q"],
                                 w["seqlens_k"], w["block_table"], w["max_seqlen_q"],
                                 w["max_seqlen_k"], **a)


def np64(t):
    return t.detach().cpu().double().numpy()


def dequantised(w, b, name):
    """The keys (or values) of sequence b: [length, Hkv, D] in 64 bits."""
    cache, scale = w[name + "_cache"], w[name + "_scale"]
    page, n = cache.shape[1], w["k_lens"][b]
    ids = w["block_table"][b, :-(-n // page)].long()
    x = np64(cache[ids].reshape(-1, *cache.shape[2:])[:n].view(torch.uint8)
             .view(torch.float8_e4m3fn))
    return x if scale is None else x * np64(scale)[:, None]


def check(w, out, lse, scale=None, causal=True, seqs=None):
    hq, d = w["q"].shape[1:]
    hkv = w["k_cache"].shape[2]
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    half = HALF[w["dtype"]]
    at = 0
    worst = 0.0
    for b, (m, n) in enumerate(zip(w["q_lens"], w["k_lens"])):
        rows = slice(at, at + m)
        at += m
        if m == 0 or (seqs is not None and b not in seqs):
            continue
        q, k, v = np64(w["q"][rows]), dequantised(w, b, "k"), dequantised(w, b, "v")
        o, l = oracle.attend_rows(q, k, v, scale, causal)
        a, _ = oracle.attend_rows(q, k, np.abs(v), scale, causal)
        got, got_l = np64(out[rows]), None if lse is None else np64(lse[:, rows])
        group = hq // hkv
        kabs = np.abs(k).repeat(group, axis=1)                      # [n, Hq, D]
        if n:
            S = scale * np.einsum("mhd,nhd->hmn", np.abs(q), kabs).max(-1)     # [Hq, m]
            Q = scale * np.abs(q).max(-1).T * kabs.sum(-1).max(0)[:, None]
        else:
            S = Q = np.zeros((hq, m))
        ds = 2.0 ** -17 * S + 2.0 ** -24 * Q
        room = (2 * ds + 2.0 ** -11 + n * 2.0 ** -26 + 2.0 ** -19).T[..., None] * a
        room = room + half * np.abs(o) + 2.0 ** -25
        bad = ~(np.abs(got - o) <= room)
        assert not bad.any(), (b, m, n, np.argwhere(bad)[:4].tolist(),
                               np.abs(got - o)[bad][:4], room[bad][:4])
        worst = max(worst, float(np.max(np.abs(got - o) / room)))
        if got_l is not None:
            fin = np.isfinite(l)
            assert np.array_equal(np.isfinite(got_l), fin) and (got_l[~fin] == -np.inf).all(), b
            lroom = ds + n * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * np.abs(np.where(fin, l, 0))
            assert (np.abs(got_l - l)[fin] <= lroom[fin]).all(), (b, np.abs(got_l - l)[fin].max())
    return worst
