"""Beam search of an encoder-decoder model from the prompt to the last page given back: select, reorder, copy,
plan, append, self attention and cross attention, call by call against plain lists and as one captured
step that is replayed.

The model's projections are tables by token and position, so what every page has to hold is known bit for
bit.  A beam that has finished appends nothing: the batch is ragged in every step.

Scores.  ln of a sum of V = 50 exponentials in fp32, each 2^t with t <= 0 against the largest: t is rounded
once (2^-24 |t| ln 2 of the term; the mean of |t| under the terms' weights is at most log2(50) < 6), 2^t to
2^-22, and a term goes through fewer than 50 + 37 additions of 2^-24 each: (4.2 + 4 + 87) 2^-24 < 2^-17.
The fp32 score is off by 2^-24 of itself.
"""

import numpy as np
import pytest
import torch

import paged_kv_cache_page_gb300 as pa
from gpu_util import LSE_TOL, OUT_TOL, np64
from oracle import beam

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B, K, V, HQ, HKV, D, PAGE, LAYERS, END = 3, 4, 50, 8, 2, 64, 16, 2, 7
COLS, POOL, CAP, LONGEST, STEPS = 5, 60, 96, 80, 22
KEYS, HELD = [40, 7, 130], [40, 0, 113]  # encoder states, and how many of them count


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Model:
    def __init__(self):
        g = torch.Generator().manual_seed(11)
        heads = HQ + 2 * HKV
        self.qkv = [torch.randn((V, LONGEST, heads, D), generator=g).bfloat16().to(DEV) for _ in range(LAYERS)]
        self.xq = [torch.randn((V, LONGEST, HQ, D), generator=g).bfloat16().to(DEV) for _ in range(LAYERS)]
        self.kv = [torch.randn((sum(KEYS), 2 * HKV, D), generator=g).bfloat16().to(DEV) for _ in range(LAYERS)]
        self.mask = (torch.rand(sum(KEYS), generator=g) < 0.8).to(DEV)
        self.head = torch.randn((HQ * D, V), generator=g).to(DEV)
        self.bias = torch.zeros(V, device=DEV)
        self.bias[END] = 3.0
        self.cu_k, self.held = i32(np.cumsum([0] + KEYS).tolist()), i32(HELD)


class Search:
    """The state of one search on the GPU; `step` is the whole step, without a word from the host."""

    def __init__(self, model, prompts):
        self.m, rows = model, B * K
        self.caches = [torch.zeros((POOL, PAGE, HKV, D), dtype=torch.bfloat16, device=DEV)
                       for _ in range(2 * LAYERS)]
        self.table, self.lens = i32([[-1] * COLS] * rows), i32([0] * rows)
        self.pool, self.count = i32(list(range(POOL))), i32([POOL])
        self.scores = torch.full((B, K), float("-inf"), device=DEV)
        self.scores[:, 0] = 0
        self.finished = torch.zeros((B, K), dtype=torch.bool, device=DEV)
        self.cu, self.cu_x, self.pos = i32([0] * (rows + 1)), i32([0] * (B + 1)), i32([0] * CAP)
        self.slots = torch.zeros(CAP, dtype=torch.int64, device=DEV)
        self.tokens = torch.zeros(CAP + 1, dtype=torch.int64, device=DEV)
        self.out = [torch.zeros((CAP, HQ, D), dtype=torch.bfloat16, device=DEV) for _ in range(2 * LAYERS)]
        self.lse = [torch.zeros((HQ, CAP), device=DEV) for _ in range(2 * LAYERS)]
        self.logits = torch.zeros((B, K, V), device=DEV)
        size = pa.fwd_cross_workspace_size(CAP, CAP, HQ, HKV, D)
        self.workspace = torch.zeros(size, dtype=torch.uint8, device=DEV) if size else None
        self.err = pa.new_err_word(DEV)
        self.parents, self.picked, self.copies = i32([[0] * K] * B), i32([[0] * K] * B), i32([[0] * 3] * rows)
        flat = [t for p in prompts for t in p]
        self.tokens[:len(flat)] = torch.tensor(flat, device=DEV)
        new = torch.zeros((B, K), dtype=torch.int32)
        new[:, 0] = torch.tensor([len(p) for p in prompts])
        self.run(new.view(-1).to(DEV), None)

    def run(self, new, picked):
        """New tokens of each beam's row through the model, to the logits of each row's last token."""
        m = self.m
        pa.pa_plan_step(self.lens, new, self.table, self.pool, self.count, PAGE, self.cu, self.lens, self.slots,
                        self.pos, err=self.err)
        if picked is not None:
            at = torch.where(new > 0, self.cu[:-1], CAP).long()
            self.tokens.scatter_(0, at, picked.clamp(min=0).long().view(-1))
        self.cu_x.copy_(self.cu[::K])
        tokens, pos = self.tokens[:CAP], self.pos.long()
        for i in range(LAYERS):
            x = m.qkv[i][tokens, pos]
            kc, vc = self.caches[2 * i], self.caches[2 * i + 1]
            pa.pa_rotary_append_varlen(None, x[:, HQ:HQ + HKV], x[:, HQ + HKV:], kc, vc, self.slots, err=self.err)
            pa.pa_fwd_varlen_unified(x[:, :HQ].contiguous(), kc, vc, self.cu, self.lens, self.table, CAP,
                                     COLS * PAGE, causal=True, out=self.out[2 * i], lse=self.lse[2 * i])
            pa.pa_fwd_cross(m.xq[i][tokens, pos], m.kv[i][:, :HKV], m.kv[i][:, HKV:], self.cu_x, m.cu_k, CAP,
                            max(KEYS), seqlens_k=m.held, key_mask=m.mask, out=self.out[2 * i + 1],
                            lse=self.lse[2 * i + 1], workspace=self.workspace, err=self.err)
        last = (self.cu[1:].long() - 1).clamp(min=0)
        hidden = sum(o[last].float() for o in self.out).view(B * K, HQ * D)
        self.logits.copy_((hidden @ m.head / 8 + m.bias).view(B, K, V))

    def step(self):
        scores, parents, picked, finished = pa.pa_beam_select(self.logits, self.scores, K, self.finished, END,
                                                              err=self.err)
        pa.pa_beam_reorder(parents, self.lens, self.table, self.pool, self.count, PAGE, copies=self.copies,
                           err=self.err)
        pa.pa_copy_pages(self.copies, self.caches, err=self.err)
        self.scores.copy_(scores)
        self.finished.copy_(finished)
        self.parents.copy_(parents)
        self.picked.copy_(picked)
        self.run(((parents >= 0) & ~finished).int().view(-1), picked)


PROMPTS = [[3, 1, 4, 1, 5], [9, 2, 6] * 10 + [5, 3], [8] * 16]


def plain_rows(search, held, first):
    """What the attention calls had to return: the packed rows' self attention to their own tokens and
    cross attention to their request's states.  `first`: the first of its new tokens, by row."""
    m = search.m
    cu = search.cu.tolist()
    for i in range(LAYERS):
        qkv, xq = np64(m.qkv[i]), np64(m.xq[i])
        for r, tokens in enumerate(held):
            n = cu[r + 1] - cu[r]
            assert n == len(tokens) - first[r]
            kv = np.stack([qkv[t, p, HQ:] for p, t in enumerate(tokens)]) if tokens else None
            for j in range(n):
                p = first[r] + j
                o, l = beam.cross(qkv[tokens[p], p, :HQ][None], kv[:p + 1, :HKV], kv[:p + 1, HKV:], [0, 1],
                                         [0, p + 1])
                assert np.abs(np64(search.out[2 * i][cu[r] + j]) - o[0]).max() <= OUT_TOL["bf16"]
                assert np.abs(np64(search.lse[2 * i][:, cu[r] + j]) - l[:, 0]).max() <= LSE_TOL
        q = [xq[t, p] for r, tokens in enumerate(held) for p, t in enumerate(tokens) if p >= first[r]]
        if not q:
            continue
        kv = np64(m.kv[i])
        o, l = beam.cross(np.stack(q), kv[:, :HKV], kv[:, HKV:], cu[::K], np.cumsum([0] + KEYS), HELD, np64(m.mask))
        assert np.abs(np64(search.out[2 * i + 1][:len(q)]) - o).max() <= OUT_TOL["bf16"]
        got = np64(search.lse[2 * i + 1][:, :len(q)])
        assert (np.isinf(got) == np.isinf(l)).all()
        keys = np.isfinite(l)
        assert np.abs(got[keys] - l[keys]).max(initial=0) <= LSE_TOL


def check_pages(search, held):
    """Lengths, what the pages hold (bit for bit), and every page of the pool in its place."""
    lens, table = search.lens.tolist(), search.table.tolist()
    assert lens == [len(t) for t in held]
    used = set()
    for r, tokens in enumerate(held):
        pages = table[r][:-(-len(tokens) // PAGE)]
        used |= set(pages)
        for c, cache in enumerate(search.caches):
            side = slice(HQ, HQ + HKV) if c % 2 == 0 else slice(HQ + HKV, HQ + 2 * HKV)
            if not tokens:
                continue
            got = cache[torch.tensor(pages, device=DEV)].flatten(0, 1)[:len(tokens)]
            want = search.m.qkv[c // 2][torch.tensor(tokens), torch.arange(len(tokens))][:, side]
            assert torch.equal(got.view(torch.int16), want.contiguous().view(torch.int16)), (r, c)
    free = search.pool.tolist()[:search.count.item()]
    assert sorted(free + list(used)) == list(range(POOL))


def test_a_search_against_plain_lists():
    search = Search(Model(), PROMPTS)
    held = [list(PROMPTS[r // K]) if r % K == 0 else [] for r in range(B * K)]
    plain_rows(search, held, [0] * (B * K))
    check_pages(search, held)
    copied = 0
    for step in range(STEPS):
        if step == STEPS - 4:  # the second request has ended: its beams are dead
            search.scores[1] = float("-inf")
        if step == STEPS - 1:  # so have the others
            search.scores.fill_(float("-inf"))
        logits, before = np64(search.logits), np64(search.scores)
        finished = search.finished.tolist()
        search.step()
        assert search.err.tolist() == [0] * 4
        want = beam.select(logits, before, K, finished, END)
        assert search.parents.tolist() == want[1] and search.picked.tolist() == want[2]
        assert search.finished.tolist() == want[3]
        got, ref = np64(search.scores), np.array(want[0])
        dead = np.isinf(ref)
        assert (np.isinf(got) == dead).all()
        assert (np.abs(got[~dead] - ref[~dead]) <= 2.0**-17 + 2.0**-23 * np.abs(ref[~dead])).all()
        copied += int((search.copies[:, 2] > 0).sum())
        old, held, first = held, [], []
        for r in range(B * K):
            b, i = divmod(r, K)
            parent = want[1][b][i]
            tokens = list(old[b * K + parent]) if parent >= 0 else []
            first.append(len(tokens))
            held.append(tokens + [want[2][b][i]] if parent >= 0 and not want[3][b][i] else tokens)
        check_pages(search, held)
        plain_rows(search, held, first)
    assert copied > 0 and search.count.item() == POOL and held == [[]] * (B * K)


def test_a_captured_step_replayed():
    model = Model()
    eager, graphed = Search(model, PROMPTS), Search(model, PROMPTS)
    for s in (eager, graphed):
        s.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step()
    for step in range(STEPS):
        if step == STEPS - 1:
            for s in (eager, graphed):
                s.scores.fill_(float("-inf"))
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert eager.err.tolist() == graphed.err.tolist() == [0] * 4
        for name in ("parents", "picked", "finished", "lens", "table", "pool", "count", "cu", "copies"):
            assert torch.equal(getattr(eager, name), getattr(graphed, name)), name
        for a, b in zip(eager.caches + [eager.scores], graphed.caches + [graphed.scores]):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        rows = eager.cu[-1].item()
        for a, b in zip(eager.out, graphed.out):
            assert torch.equal(a[:rows], b[:rows])
    assert graphed.count.item() == POOL
