"""Beam search of an encoder-decoder model over a paged key/value cache, as measured cases.

A step of such a search is three operators, each named by a case's ``op``:

``select``   from the logits of every beam: the best continuations of each request over its
             beams and the vocabulary, with their scores, parents and tokens;
``reorder``  block tables, lengths and pool after the beams have been replaced by their
             continuations: full pages are shared, abandoned ones go back to the pool, and a
             partly filled page that several continuations would write to is copied, in the
             caches of all layers;
``cross``    attention of the decoder's rows to the encoder's states of their request: all
             beams of a request read one copy of its keys and values, of another length than
             the rows, packed behind one another or padded with masked places.

``run`` computes a case in elementary torch operations, or, where ``own`` is true, calls
the library's operators.  ``exact`` is the same from the definitions, in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def _select(name, seqs, beams, vocab, dtype, out, ends, first):
    """``out`` continuations of each of ``seqs`` requests; ``ends``: some beams have finished;
    ``first``: only the first beam of a request lives yet."""
    return dict(name=name, op="select", seqs=seqs, beams=beams, vocab=vocab, dtype=dtype, out=out,
                ends=ends, first=first)


def _reorder(name, seqs, beams, ctx, made, page, layers, heads, d, dtype, first):
    """Prompts of up to ``ctx`` tokens and up to ``made`` generated ones; caches of ``layers``
    layers with ``heads`` heads of ``d`` features; ``first``: the prompt's only row becomes
    ``beams`` beams."""
    return dict(name=name, op="reorder", seqs=seqs, beams=beams, ctx=ctx, made=made, page=page,
                layers=layers, heads=heads, d=d, dtype=dtype, first=first)


def _cross(name, seqs, rows_lo, rows_hi, keys_lo, keys_hi, hq, hkv, d, dtype, mask):
    """``seqs`` requests with rows_lo..rows_hi decoder rows (beams times new tokens) each and
    keys_lo..keys_hi encoder states; ``mask``: a tenth of the states is masked."""
    return dict(name=name, op="cross", seqs=seqs, rows_lo=rows_lo, rows_hi=rows_hi,
                keys_lo=keys_lo, keys_hi=keys_hi, hq=hq, hkv=hkv, d=d, dtype=dtype, mask=mask)


def listed():
    return [
        # one interactive request with four beams: the call after every token, latency
        _select("select_b1_k4", 1, 4, 32000, "bf16", 4, False, False),
        # a batch with fp32 logits of an odd vocabulary; some hypotheses have ended, and twice
        # as many candidates as beams are kept
        _select("select_b16_k5_odd", 16, 5, 50001, "f32", 10, True, False),
        # a full server batch over a large vocabulary: the largest read
        _select("select_b64_k8", 64, 8, 128000, "bf16", 16, False, False),
        # the tables of one short request: latency
        _reorder("reorder_b1_k4", 1, 4, 300, 60, 16, 2, 8, 64, "f16", False),
        # the first step after the prompts: every prompt's row becomes five beams
        _reorder("reorder_first_b32_k5", 32, 5, 1000, 0, 16, 12, 12, 64, "bf16", True),
        # a full batch with long prompts and a grouped-query cache: the most copies
        _reorder("reorder_b64_k8", 64, 8, 1024, 256, 64, 4, 8, 128, "bf16", False),
        # four beams of one request over a thousand states: latency
        _cross("cross_b1_k4", 1, 4, 4, 1000, 1000, 12, 12, 64, "f16", False),
        # five beams each of a batch whose inputs have very different lengths
        _cross("cross_beams_b32", 32, 5, 5, 100, 1500, 16, 16, 64, "bf16", False),
        # a padded batch with masked states, eight beams, grouped-query heads: the largest read
        _cross("cross_gqa_b64", 64, 8, 8, 4096, 4096, 32, 8, 128, "bf16", True),
        # a few proposed tokens of every beam checked at once
        _cross("cross_verify_b16", 16, 16, 40, 257, 2048, 12, 12, 64, "f16", False),
        # prompts of a ragged batch beside single rows
        _cross("cross_mixed_b12", 12, 1, 257, 33, 2048, 32, 8, 128, "bf16", True),
        # whole target sequences scored in one pass: the largest computation
        _cross("cross_score_b4", 4, 1024, 1024, 4096, 4096, 32, 32, 128, "bf16", False),
    ]


HEADS = ((4, 2, 64), (8, 1, 64), (12, 12, 64), (16, 16, 64), (16, 4, 128), (32, 8, 128),
         (32, 32, 128), (64, 8, 128), (20, 20, 64), (20, 4, 64))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("select", "reorder", "cross", "cross"))
    if op == "select":
        seqs, beams = _log(rng, 1, 128), rng.choice((1, 2, 3, 4, 5, 8, 12, 16))
        vocab = _log(rng, 500, 260000)
        dtype = rng.choice(("f16", "bf16", "f32"))
        while seqs * beams * vocab * (2 if dtype == "f32" else 1) > 64 * 8 * 128000:
            seqs, vocab = max(1, seqs * 2 // 3), vocab * 4 // 5
        c = _select("", seqs, beams, vocab, dtype, rng.choice((beams, beams, 2 * beams)),
                    rng.choice((False, True)), rng.choice((False, False, False, True)))
        if c["first"]:
            c["ends"] = False
    elif op == "reorder":
        first = rng.choice((False, False, False, True))
        seqs, beams = _log(rng, 1, 256), rng.choice((2, 3, 4, 5, 8, 12, 16))
        heads, d = rng.choice(((2, 64), (8, 64), (12, 64), (4, 128), (8, 128)))
        c = _reorder("", seqs, beams, _log(rng, 16, 4096), 0 if first else _log(rng, 4, 512),
                     rng.choice((16, 16, 32, 64, 128, 256)), rng.choice((1, 2, 3, 6, 12)), heads, d,
                     rng.choice(("f16", "bf16")), first)
        # at most the tokens of reorder_b64_k8's caches, and its copies
        size = lambda: c["seqs"] * c["layers"] * heads * d / (64 * 4 * 8 * 128)  # noqa: E731
        while (size() * (c["ctx"] + beams * (c["made"] + 2 * c["page"])) > 1024 + 8 * 384
               or size() * beams * c["page"] > 8 * 64):
            if c["seqs"] > 1:
                c["seqs"] = c["seqs"] * 2 // 3
            else:
                c["layers"], c["ctx"] = max(1, c["layers"] // 2), max(16, c["ctx"] // 2)
    else:
        hq, hkv, d = rng.choice(HEADS)
        keys = _log(rng, 1, 8192)
        rows = rng.choice((1, 4, 5, 8, _log(rng, 1, 64), _log(rng, 1, 1024)))
        seqs = _log(rng, 1, 128)
        while (seqs * keys * hkv * d > 2 ** 28 or seqs * hq * rows * keys * d > 2 ** 36
               or seqs * hq * rows * keys > 2 ** 29):
            if seqs > 1:
                seqs = seqs * 2 // 3
            else:
                rows, keys = max(1, rows * 2 // 3), max(1, keys * 3 // 4)
        c = _cross("", seqs, max(1, rows // rng.choice((1, 1, 4))), rows,
                   max(1, keys // rng.choice((1, 2, 8))), keys, hq, hkv, d,
                   rng.choice(("f16", "bf16")), rng.choice((False, False, True)))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g)


def _pages(x, page):
    return (x + page - 1) // page


def _i32(t):
    return t.to(torch.int32).to(DEV)


def _normal(g, shape, dtype):
    """N(0, 1) values, a part at a time (the fp32 values of a large tensor are many)."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    step = max(1, (1 << 27) // max(1, out[0].numel()))
    for i in range(0, shape[0], step):
        out[i:i + step] = torch.randn((min(step, shape[0] - i),) + tuple(shape[1:]), generator=g,
                                      device=DEV)
    return out


def prepare(case, seed):
    g = torch.Generator().manual_seed(int(seed))
    dg = torch.Generator(device=DEV).manual_seed(int(seed))
    return {"select": _prepare_select, "reorder": _prepare_reorder,
            "cross": _prepare_cross}[case["op"]](case, g, dg)


def _prepare_select(case, g, dg):
    seqs, beams, vocab, out = case["seqs"], case["beams"], case["vocab"], case["out"]
    x = torch.randn((seqs, beams, vocab), generator=dg, device=DEV) * 2.5
    # a few likely tokens, and some that may not be used
    likely = torch.randint(0, vocab, (seqs, beams, 8), generator=dg, device=DEV)
    x.scatter_add_(2, likely, 6 + 3 * torch.randn((seqs, beams, 8), generator=dg, device=DEV))
    x[..., torch.randint(0, vocab, (max(1, vocab // 200),), generator=dg, device=DEV)] = -math.inf
    scores = -torch.rand((seqs, beams), generator=dg, device=DEV) * 3
    scores = scores.cumsum(1) - 20 * torch.rand((seqs, 1), generator=dg, device=DEV)
    finished = None
    if case["ends"]:
        finished = torch.rand((seqs, beams), generator=dg, device=DEV) < 0.3
        finished[:, 0] = False
    if case["first"]:
        scores = torch.zeros((seqs, beams), device=DEV)
        scores[:, 1:] = -math.inf
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(op="select", logits=x.to(DTYPES[case["dtype"]]), scores=scores, finished=finished,
                end_token=2 % vocab, out=out, scores_out=torch.empty((seqs, out), device=DEV),
                parents=torch.empty((seqs, out), **i32), tokens=torch.empty((seqs, out), **i32),
                finished_out=torch.empty((seqs, out), dtype=torch.bool, device=DEV))


def _prepare_reorder(case, g, dg):
    seqs, beams, page = case["seqs"], case["beams"], case["page"]
    prompt = _ints(g, max(1, case["ctx"] // 2), case["ctx"], seqs)
    made = _ints(g, 1, case["made"], seqs) if case["made"] else torch.zeros(seqs, dtype=torch.int64)
    lens = (prompt + made)[:, None].repeat(1, beams)
    parents = _ints(g, 0, beams - 1, seqs * beams).view(seqs, beams)
    if case["first"]:
        lens[:, 1:] = 0
        parents.zero_()
    elif beams > 2:
        # a hypothesis that ended some tokens ago, kept beside the others
        ago = torch.minimum(_ints(g, 0, 2 * page, seqs), made - 1)
        lens[:, -1] -= torch.where(torch.rand(seqs, generator=g) < 0.25, ago, 0)
    width = (case["ctx"] + case["made"]) // page + 2
    # which beam of its column's time each beam descends from, from the last column backwards: a
    # page is shared by the beams with the same ancestor, the prompt's full pages by all
    ids = torch.zeros((seqs, beams, width), dtype=torch.int64)
    at = torch.arange(beams).repeat(seqs, 1)
    last = _pages(lens[:, 0], page) - 1
    for j in range(width - 1, -1, -1):
        older = _ints(g, 0, beams - 1, seqs * beams).view(seqs, beams)
        at = torch.where((last > j)[:, None], older.gather(1, at), at)
        inside = (prompt // page > j)[:, None]
        here = torch.where(inside, 0, at)
        ends = (lens // page == j) & (lens % page != 0) & (lens < lens[:, :1])
        here = torch.where(ends, beams + torch.arange(beams), here)
        ids[:, :, j] = here
    col = torch.arange(width)
    held = col < _pages(lens, page)[..., None]
    key = (torch.arange(seqs)[:, None, None] * width + col) * 2 * beams + ids
    names, page_of = key[held].unique(return_inverse=True)
    # a page more for each beam than they can hold, and a few besides
    pool = seqs * (case["ctx"] // page + beams * (-(-case["made"] // page) + 2)) + 8
    spare = pool - names.numel()
    order = torch.randperm(pool, generator=g)
    table = torch.full((seqs, beams, width), -1, dtype=torch.int64)
    table[held] = order[page_of]
    free = torch.zeros(pool, dtype=torch.int64)
    free[:spare] = order[names.numel():]
    # (one page more than the pool has, which the plain form uses for what is not copied)
    shape = (pool + 1, page, case["heads"], case["d"])
    whole = [_normal(dg, shape, DTYPES[case["dtype"]]) for _ in range(2 * case["layers"])]
    table = _i32(table.view(seqs * beams, width))
    return dict(op="reorder", page=page, parents=_i32(parents), seqlens=_i32(lens.view(-1)),
                block_table=table, free_pages=_i32(free), free_count=_i32(torch.tensor([spare])),
                block_table_out=torch.full_like(table, -1),
                seqlens_out=_i32(torch.zeros(seqs * beams)),
                copies=_i32(torch.zeros((seqs * beams, 3))), free_count_out=_i32(torch.zeros(1)),
                whole=whole, caches=[c[:pool] for c in whole])


def _prepare_cross(case, g, dg):
    seqs, hq, hkv, d = case["seqs"], case["hq"], case["hkv"], case["d"]
    dt = DTYPES[case["dtype"]]
    # lengths in equal steps, in an order of the seed's
    rows, keys = (torch.linspace(case[n + "_hi"], case[n + "_lo"], seqs).long()[
        torch.randperm(seqs, generator=g)] for n in ("rows", "keys"))
    zero = torch.zeros(1, dtype=torch.int64)
    cu_q, cu_k = torch.cat([zero, rows.cumsum(0)]), torch.cat([zero, keys.cumsum(0)])
    total_q, total_k = int(cu_q[-1]), int(cu_k[-1])
    # one projection of the encoder's states gives k and v as slices of the same rows
    kv = _normal(dg, (total_k, 2, hkv, d), dt)
    mask = None
    if case["mask"]:
        mask = torch.rand(total_k, generator=dg, device=DEV) < 0.9
        mask[cu_k[:-1].to(DEV)] = True
    return dict(op="cross", q=_normal(dg, (total_q, hq, d), dt), k=kv[:, 0], v=kv[:, 1],
                cu_seqlens_q=_i32(cu_q), cu_seqlens_k=_i32(cu_k), max_seqlen_q=case["rows_hi"],
                max_seqlen_k=case["keys_hi"], key_mask=mask,
                out=torch.empty((total_q, hq, d), dtype=dt, device=DEV),
                lse=torch.empty((hq, total_q), device=DEV))


# ------------------------------------------------------------------ one pass
def run(state):
    return {"select": _run_select, "reorder": _run_reorder, "cross": _run_cross}[state["op"]](state)


def _run_select(s):
    names = ("scores_out", "parents", "tokens", "finished_out")
    if own:
        import paged_kv_cache_page_gb300 as pa
        pa.pa_beam_select(s["logits"], s["scores"], s["out"], finished=s["finished"],
                          end_token=s["end_token"], scores_out=s["scores_out"],
                          parents=s["parents"], tokens=s["tokens"],
                          finished_out=s["finished_out"])
        return {n: s[n] for n in names}
    # scores in 64 bits: in 32 many candidates of different beams would be equal
    x = s["logits"].double()
    seqs, beams, vocab = x.shape
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top)
    norm = x.exp().sum(-1, keepdim=True).log_()
    cum = s["scores"].double()
    x = x.sub_(norm).add_(cum[..., None])
    if s["finished"] is not None:
        x.masked_fill_(s["finished"][..., None], -math.inf)
        x[..., s["end_token"]] = torch.where(s["finished"], cum, x[..., s["end_token"]])
    x = x.view(seqs, beams * vocab)
    best, at = [], []
    for _ in range(s["out"]):
        i = x.argmax(-1, keepdim=True)  # (the first of equal ones)
        best.append(x.gather(1, i))
        at.append(i)
        x.scatter_(1, i, -math.inf)
    best, at = torch.cat(best, 1), torch.cat(at, 1)
    parents, tokens = at // vocab, at % vocab
    done = tokens == s["end_token"]
    if s["finished"] is not None:
        done |= s["finished"].gather(1, parents)
    for n, value in zip(names, (best, parents, tokens, done)):
        s[n].copy_(value)
    return {n: s[n] for n in names}


def _run_reorder(s):
    names = ("block_table_out", "seqlens_out", "copies", "free_pages", "free_count_out", "caches")
    if own:
        import paged_kv_cache_page_gb300 as pa
        pa.pa_beam_reorder(s["parents"], s["seqlens"], s["block_table"], s["free_pages"],
                           s["free_count"], s["page"], block_table_out=s["block_table_out"],
                           seqlens_out=s["seqlens_out"], copies=s["copies"],
                           free_count_out=s["free_count_out"])
        pa.pa_copy_pages(s["copies"], s["caches"])
        return {n: s[n] for n in names}
    page, pool = s["page"], s["free_pages"].numel()
    seqs, beams = s["parents"].shape
    table = s["block_table"].view(seqs, beams, -1)
    width = table.shape[2]
    lens = s["seqlens"].view(seqs, beams).long()
    col = torch.arange(width, device=DEV)
    held = col < _pages(lens, page)[..., None]
    lives = s["parents"] >= 0
    par = s["parents"].long().clamp(min=0)
    new = torch.where(lives, lens.gather(1, par), 0)
    wide = par[..., None].expand(-1, -1, width)
    entry, has = table.gather(1, wide), held.gather(1, wide) & lives[..., None]
    partly = has & (col == (new // page)[..., None]) & (new % page != 0)[..., None]
    beam = torch.arange(beams, device=DEV)
    # pages that no child holds, each once
    same = (entry[:, None] == table[:, :, None]) & has[:, None]
    gone = held & ~same.any(2)
    twin = (table[:, None] == table[:, :, None]) & gone[:, None]
    gone &= ~(twin & (beam[:, None] > beam)[None, :, :, None]).any(2)
    # a partly filled page is the first child's that holds it and no other's
    clash = (entry[:, None] == entry[:, :, None]) & has[:, None]
    clash &= (beam[:, None] > beam)[None, :, :, None] | ~partly[:, None]
    copy = partly & clash.any(2)
    # groups in order, as far as the pool goes: pages given back first, then the copies
    free = s["free_count"].long()
    given, taken = gone.sum((1, 2)), copy.sum((1, 2))
    fits = (free + given.cumsum(0) - taken.cumsum(0) >= 0).long().cumprod(0).bool()
    gone, copy = gone & fits[:, None, None], copy & fits[:, None, None]
    order = gone.transpose(1, 2).reshape(-1)
    rank = order.long().cumsum(0)
    stack = torch.cat([s["free_pages"], s["free_pages"][:1]])
    stack[torch.where(order, free + rank - 1, pool)] = table.transpose(1, 2).reshape(-1)
    s["free_pages"].copy_(stack[:pool])
    filled = free + rank[-1:]
    wants = copy.transpose(1, 2).reshape(-1)
    rank = wants.long().cumsum(0)
    fresh = stack[torch.where(wants, filled - rank, 0)].view(seqs, width, beams).transpose(1, 2)
    s["free_count_out"].copy_(filled - rank[-1:])
    out = s["block_table_out"].view(seqs, beams, width)
    entry = torch.where(fits[:, None, None], torch.where(copy, fresh, entry), table)
    has = torch.where(fits[:, None, None], has, held)
    out.copy_(torch.where(has, entry, out))
    s["seqlens_out"].copy_(torch.where(fits[:, None], new, lens).view(-1))
    # where a child copies, it does so in one column
    any_copy = copy.any(2)
    src = (table.gather(1, wide) * copy).sum(2)
    dst = (fresh * copy).sum(2)
    triple = torch.stack([torch.where(any_copy, src, -1), torch.where(any_copy, dst, -1),
                          torch.where(any_copy, new % page, 0)], -1).view(-1, 3)
    s["copies"].copy_(triple)
    live = triple[:, 1] >= 0
    src, dst = torch.where(live, triple[:, 0], pool), torch.where(live, triple[:, 1], pool)
    part = (torch.arange(page, device=DEV) < triple[:, 2:])[..., None, None]
    for c in s["whole"]:
        c[dst] = torch.where(part, c[src], c[dst])
    return {n: s[n] for n in names}


def _run_cross(s):
    if own:
        import paged_kv_cache_page_gb300 as pa
        pa.pa_fwd_cross(s["q"], s["k"], s["v"], s["cu_seqlens_q"], s["cu_seqlens_k"],
                        s["max_seqlen_q"], s["max_seqlen_k"], key_mask=s["key_mask"],
                        out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    total, hq, d = s["q"].shape
    hkv, total_k = s["k"].shape[1], s["k"].shape[0]
    cu_q, cu_k = s["cu_seqlens_q"].long(), s["cu_seqlens_k"].long()
    seqs, most, far = cu_q.numel() - 1, s["max_seqlen_q"], s["max_seqlen_k"]
    t = torch.arange(far, device=DEV)
    at = cu_k[:-1, None] + t
    seen = at < cu_k[1:, None]
    at = at.clamp(max=total_k - 1)
    if s["key_mask"] is not None:
        seen &= s["key_mask"][at]
    rows = (cu_q[:-1, None] + torch.arange(most, device=DEV)).clamp(max=total - 1)
    q = s["q"][rows].float().reshape(seqs, most, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    score = q.reshape(seqs, hkv, -1, d) @ s["k"][at].float().permute(0, 2, 3, 1)
    score = score.mul_(1.0 / math.sqrt(d)).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    score = score.sub_(top).exp_()
    norm = score.sum(-1, keepdim=True)
    out = (score @ s["v"][at].float().transpose(1, 2)) / norm
    out = out.view(seqs, hkv, hq // hkv, most, d).permute(0, 3, 1, 2, 4)
    lse = (top + norm.log()).view(seqs, hq, most)
    row = torch.arange(total, device=DEV)
    seq = torch.searchsorted(cu_q[1:], row, right=True)
    at = row - cu_q[seq]
    s["out"].copy_(out.reshape(seqs, most, hq, d)[seq, at])
    s["lse"].copy_(lse[seq, :, at].T)
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ what a pass has to do
def work(case):
    op, seqs = case["op"], case["seqs"]
    if op == "select":
        beams, vocab, out = case["beams"], case["vocab"], case["out"]
        # every logit read once: its maximum, exponential and sum
        live = seqs if case["first"] else seqs * beams * (0.75 if case["ends"] else 1)
        n = live * vocab
        return dict(bytes=n * (4 if case["dtype"] == "f32" else 2) + seqs * (beams * 5 + out * 13),
                    flops=4 * n)
    if op == "reorder":
        beams, page = case["beams"], case["page"]
        columns = (case["ctx"] * 0.75 + case["made"] / 2) / page
        kept = 1 if case["first"] else beams * (1 - (1 - 1 / beams) ** beams)
        tokens = seqs * (beams - kept) * min(page / 2, case["ctx"] * 0.75 + case["made"] / 2)
        size = case["heads"] * case["d"] * 2
        # a table entry read and written for every page and beam; the copied tokens' k and v of
        # all layers read and written
        return dict(bytes=seqs * beams * (columns * 8 + 24) + tokens * size * 4 * case["layers"],
                    flops=0)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    rows = seqs * (case["rows_lo"] + case["rows_hi"]) / 2
    keys = seqs * (case["keys_lo"] + case["keys_hi"]) / 2
    return dict(bytes=keys * (hkv * d * 4 + (1 if case["mask"] else 0)) + rows * hq * (4 * d + 4),
                flops=4 * d * hq * rows * keys / seqs)


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    if case["op"] == "reorder":
        return None  # whole numbers and copied values
    s = prepare(case, seed)
    if case["op"] == "select":
        seqs, beams, vocab = s["logits"].shape
        out = {n: [] for n in ("scores_out", "parents", "tokens", "finished_out")}
        for b in range(seqs):
            lists = []
            for k in range(beams):
                x = s["logits"][b, k].double()
                base = s["scores"][b, k].double()
                if s["finished"] is not None and s["finished"][b, k]:
                    row = torch.full_like(x, -math.inf)
                    row[s["end_token"]] = base
                else:
                    row = base + torch.log_softmax(x, -1)
                lists.append(row)
            value, at = torch.cat(lists).sort(descending=True, stable=True)
            at = at[:case["out"]]
            out["scores_out"].append(value[:case["out"]])
            out["parents"].append((at // vocab).int())
            out["tokens"].append((at % vocab).int())
            done = at % vocab == s["end_token"]
            if s["finished"] is not None:
                done = done | s["finished"][b][at // vocab]
            out["finished_out"].append(done)
        return {n: torch.stack(v) for n, v in out.items()}
    total, hq, d = s["q"].shape
    group = hq // s["k"].shape[1]
    out = torch.zeros((total, hq, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((hq, total), dtype=torch.float64, device=DEV)
    cu_q, cu_k = s["cu_seqlens_q"].tolist(), s["cu_seqlens_k"].tolist()
    for b in range(case["seqs"]):
        here, there = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        k, v = s["k"][there], s["v"][there]
        if s["key_mask"] is not None:
            k, v = k[s["key_mask"][there]], v[s["key_mask"][there]]
        for h in range(hq):
            x = s["q"][here, h].double() @ k[:, h // group].double().T / math.sqrt(d)
            z = torch.logsumexp(x, -1)
            out[here, h] = (x - z[:, None]).exp() @ v[:, h // group].double()
            lse[h, here] = z
    return {"out": out, "lse": lse}
