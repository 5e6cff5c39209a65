"""pa_fwd_varlen_e4m3 where many long streams are dealt to the CTAs: equal shares that cut streams
anywhere or slots, one kv head a CTA or two to eight neighbouring ones side by side; against the oracle
on some of the sequences, and twice with the same bits."""

import pytest
import torch

import paged_kv_cache_page_gb300 as pa
from e4m3_util import DEV, DT, call, check

pytestmark = pytest.mark.gpu


def big_batch(q_lens, k_lens, hq, hkv, d, dtype, page, seed):
    """As e4m3_util.batch, made on the GPU."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    held = [-(-k // page) for k in k_lens]
    order = torch.randperm(sum(held) + 2, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(k_lens), max(held) + 1), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    scale = [(0.5 + torch.rand(hkv, generator=g, device=DEV)) * 0.01 for _ in range(2)]
    caches = [(torch.randn((at + 2, page, hkv, d), generator=g, device=DEV) / s[:, None])
              .clamp(-448, 448).to(torch.float8_e4m3fn) for s in scale]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    cu = [0]
    for m in q_lens:
        cu.append(cu[-1] + m)
    q = torch.randn((cu[-1], hq, d), generator=g, device=DEV).to(DT[dtype])
    return dict(q=q, k_cache=caches[0], v_cache=caches[1], k_scale=scale[0], v_scale=scale[1],
                cu_seqlens_q=i32(cu), seqlens_k=i32(k_lens), block_table=table,
                max_seqlen_q=max(q_lens), max_seqlen_k=max(k_lens), dtype=dtype, q_lens=list(q_lens),
                k_lens=list(k_lens))


# sequences, shortest, longest, hq, hkv, d, dtype, page, query rows in turn
CASES = [
    # one head a CTA, equal shares: an odd number of heads
    (60, 1030, 2507, 6, 3, 64, "f16", 16, (1,)),
    (23, 17, 3333, 28, 7, 128, "bf16", 32, (1, 3)),
    # two, four and eight heads side by side
    (40, 1501, 1999, 24, 6, 128, "bf16", 16, (1,)),
    (33, 1100, 3111, 12, 12, 64, "f16", 64, (1, 2)),
    (48, 2001, 4777, 32, 8, 128, "f16", 16, (1,)),
    (35, 1, 5003, 16, 16, 64, "bf16", 16, (1, 1, 5, 0)),
    (21, 1500, 2901, 32, 32, 64, "f16", 128, (1,)),
    (39, 1025, 2222, 32, 32, 128, "bf16", 16, (1,)),
    (37, 900, 4100, 64, 16, 128, "bf16", 32, (1, 4, 12)),
    # a few streams in slots, heads side by side
    (3, 20003, 61007, 32, 8, 64, "bf16", 64, (1,)),
    (4, 30011, 50021, 8, 4, 128, "f16", 16, (2, 1)),
    (9, 3001, 17003, 16, 2, 64, "f16", 256, (1, 3)),
]


# (a single row sees every key either way)
@pytest.mark.parametrize("case,causal", [(c, k) for c in CASES for k in (True, False)
                                         if k or max(c[-1]) > 1])
def test_many_long_streams(case, causal):
    n, lo, hi, hq, hkv, d, dtype, page, rows = case
    k_lens = [lo + (hi - lo) * ((7 * i) % n) // (n - 1) for i in range(n)]
    q_lens = [rows[i % len(rows)] for i in range(n)]
    w = big_batch(q_lens, k_lens, hq, hkv, d, dtype, page, seed=n)
    err = pa.new_err_word(DEV)
    out, lse = call(w, causal=causal, err=err)
    assert err.tolist() == [0] * 4
    check(w, out, lse, causal=causal, seqs={0, 1, 2, n // 3, n // 2, n - 2, n - 1})
    again, lse2 = call(w, causal=causal)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    # the sequences that no oracle looked at: the same as alone, up to what both may be off
    for b in range(n):
        if q_lens[b] == 0:
            continue
        r = slice(sum(q_lens[:b]), sum(q_lens[:b + 1]))
        one = dict(w, q=w["q"][r], cu_seqlens_q=torch.tensor([0, q_lens[b]], dtype=torch.int32, device=DEV),
                   seqlens_k=w["seqlens_k"][b:b + 1], block_table=w["block_table"][b:b + 1])
        o, l = call(one, causal=causal)
        none = l == -float("inf")
        assert torch.equal(lse[:, r] == -float("inf"), none)
        assert (lse[:, r] - l)[~none].abs().max() <= 1e-4
        # both roundings of the result, and of the probabilities (2^-11 each of the mean |v|)
        step = 2.0 ** -10 if dtype == "f16" else 2.0 ** -7
        assert (out[r].float() - o.float()).abs().max() <= step * o.float().abs().max() + 2.0 ** -10
