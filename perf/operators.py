"""The operators of one serving step over a paged key/value cache, as measured cases.

A step of a serving program with a paged cache is four operators, each named by a
case's ``op``:

``plan``     from the requests' lengths: pages for the new tokens out of the pool of free
             pages, block tables, and the slot and position of every new token;
``release``  gives the pages of finished and of shortened requests back to the pool;
``append``   rotates q and k of the ragged batch's new tokens by positions with one or
             several axes and writes k and v into their slots, in 16 bits or as e4m3;
``attend``   attention of the new tokens (whole chunks, single tokens, both in one batch)
             over a paged e4m3 cache with a scale for each kv head.

``run`` computes a case in elementary torch operations, or, where ``own`` is true, calls
the library's operators.  ``exact`` is the same from the definitions, in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0


# ------------------------------------------------------------------ the cases
def _plan(name, seqs, ctx, chunks, chunk, page, spare):
    """``chunks`` of the ``seqs`` requests bring up to ``chunk`` new tokens, the others one;
    ``spare`` is how much of the needed pages the pool of free pages holds."""
    return dict(name=name, op="plan", seqs=seqs, ctx=ctx, chunks=chunks, chunk=chunk, page=page,
                spare=spare)


def _release(name, seqs, ctx, done, page):
    """Of ``seqs`` requests of up to ``ctx`` tokens ``done`` have finished; each fourth of the
    others takes back a few tokens."""
    return dict(name=name, op="release", seqs=seqs, ctx=ctx, done=done, page=page)


def _append(name, tokens, hq, hkv, d, dtype, cache, page, axes, rot, pairs):
    """``tokens`` new tokens; ``axes`` position axes; ``rot`` rotated features; ``pairs`` is
    "halves" or "even_odd"."""
    return dict(name=name, op="append", tokens=tokens, hq=hq, hkv=hkv, d=d, dtype=dtype,
                cache=cache, page=page, axes=axes, rot=rot, pairs=pairs)


def _attend(name, seqs, ctx_lo, ctx_hi, chunks, chunk_lo, chunk_hi, hq, hkv, d, dtype, page):
    """``seqs`` requests of ctx_lo..ctx_hi keys; ``chunks`` of them have chunk_lo to chunk_hi new
    tokens, in equal steps, the others one."""
    return dict(name=name, op="attend", seqs=seqs, ctx_lo=ctx_lo, ctx_hi=ctx_hi, chunks=chunks,
                chunk_lo=chunk_lo, chunk_hi=chunk_hi, hq=hq, hkv=hkv, d=d, dtype=dtype, page=page)


def listed():
    return [
        # one decode step of a batch of 64: the call that comes before every token
        _plan("plan_decode_b64", 64, 4096, 0, 1, 16, 1.25),
        # a full step of a large server: 1024 requests, 64 of them with prompt chunks
        _plan("plan_mixed_b1024", 1024, 4096, 64, 1000, 16, 1.25),
        # a few requests of a small batch have finished
        _release("release_b64", 64, 4096, 5, 16),
        # most of a large batch ends at once (a drained or cancelled batch)
        _release("release_b1024", 1024, 8192, 700, 16),
        # the new tokens of a decode step: latency
        _append("append_decode_b64", 64, 32, 8, 128, "bf16", "e4m3", 16, 1, 128, "halves"),
        # ragged image and video prompts with time, height and width positions, 64-wide heads,
        # half of the features rotated, into a 16-bit cache
        _append("append_axes_t1601", 1601, 12, 12, 64, "f16", "f16", 32, 3, 32, "even_odd"),
        # a full prefill step with three position axes into an e4m3 cache
        _append("append_axes_t8192", 8192, 32, 8, 128, "bf16", "e4m3", 16, 3, 128, "halves"),
        # two short sequences: latency
        _attend("attend_tiny", 2, 37, 100, 0, 1, 1, 4, 2, 64, "f16", 16),
        # grouped-query decode of a few long sequences of very different lengths
        _attend("attend_gqa_b8", 8, 1024, 8192, 0, 1, 1, 32, 8, 128, "bf16", 16),
        # decode of a full batch, a kv head for each query head: the largest read
        _attend("attend_mha_b256", 256, 4096, 4096, 0, 1, 1, 32, 32, 128, "f16", 16),
        # prompt chunks and single tokens in one ragged batch
        _attend("attend_mixed_b32", 32, 257, 4096, 3, 33, 257, 32, 8, 128, "bf16", 16),
        # long chunks over as long a cached prefix: the largest computation
        _attend("attend_chunk_b2", 2, 4096, 4096, 2, 2048, 2048, 32, 8, 128, "bf16", 64),
    ]


HEADS = ((4, 2, 64), (8, 1, 64), (12, 12, 64), (16, 4, 128), (32, 8, 128), (32, 32, 128),
         (64, 8, 128), (24, 8, 128), (20, 4, 64))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("plan", "release", "append", "append", "attend", "attend", "attend"))
    page = rng.choice((16, 16, 32, 64, 128, 256))
    if op == "plan":
        seqs = _log(rng, 1, 4096)
        chunks = rng.randint(0, min(seqs, 64))
        c = _plan("", seqs, _log(rng, 64, 8192), chunks, _log(rng, 2, 1000), page,
                  rng.choice((1.25, 2.0, 0.7)))
        if seqs > 1024:
            c["ctx"] = min(c["ctx"], 4096)
    elif op == "release":
        seqs = _log(rng, 1, 4096)
        c = _release("", seqs, _log(rng, 64, 8192 if seqs <= 1024 else 2048),
                     rng.randint(0, seqs), page)
    elif op == "append":
        hq, hkv, d = rng.choice(HEADS)
        dtype = rng.choice(("f16", "bf16"))
        c = _append("", _log(rng, 1, 8192), hq, hkv, d, dtype, rng.choice((dtype, "e4m3", "e4m3")),
                    page, rng.choice((1, 2, 3)), rng.choice((d, d, d // 2)),
                    rng.choice(("halves", "halves", "even_odd")))
        while c["tokens"] * (hq + 2 * hkv) * d > 8192 * 48 * 128:
            c["tokens"] = c["tokens"] * 2 // 3
    else:
        hq, hkv, d = rng.choice(HEADS)
        ctx = _log(rng, 1, 8192)
        kind = rng.choice(("single", "single", "chunk", "mixed"))
        chunk = 1 if kind == "single" else _log(rng, 2, min(2048, max(ctx, 2)))
        seqs = _log(rng, 1, 256)
        while (seqs * ctx * hkv * d > 2 ** 32 or seqs * hq * chunk * max(ctx, chunk) > 2 ** 29):
            seqs = max(1, seqs * 2 // 3)
            if seqs == 1:
                chunk = max(1, chunk * 2 // 3)
                ctx = max(1, ctx * 3 // 4)
        chunks = 0 if kind == "single" else seqs if kind == "chunk" else rng.randint(1, seqs)
        c = _attend("", seqs, max(1, ctx // rng.choice((1, 2, 8))), ctx, chunks,
                    max(1, chunk // 3), chunk, hq, hkv, d, rng.choice(("f16", "bf16")), page)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g)


def _pages(x, page):
    return (x + page - 1) // page


def _tables(g, held, width, pool):
    """Block tables whose row b holds held[b] pages of a random order of the pool (other entries
    -1), and that order."""
    order = torch.randperm(pool, generator=g).to(torch.int32)
    mask = torch.arange(width)[None, :] < held[:, None]
    table = torch.full((held.numel(), width), -1, dtype=torch.int32)
    table[mask] = order[:int(held.sum())]
    return table, order


def _i32(t):
    return t.to(torch.int32).to(DEV)


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _cache(g, shape, scale):
    """An e4m3 cache of N(0, 1) values under the scales of its kv heads."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for p in range(0, shape[0], step):
        x = torch.randn((min(step, shape[0] - p),) + shape[1:], generator=g, device=DEV)
        out[p:p + step] = (x / scale[:, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(out.dtype)
    return out


def prepare(case, seed):
    g = torch.Generator().manual_seed(int(seed))
    dg = torch.Generator(device=DEV).manual_seed(int(seed))
    op, page = case["op"], case["page"]
    s = dict(op=op, page=page)
    if op in ("plan", "release"):
        seqs, ctx = case["seqs"], case["ctx"]
        lens = _ints(g, 1, ctx, seqs)
        held = _pages(lens, page)
    if op == "plan":
        new = torch.ones(seqs, dtype=torch.int64)
        if case["chunks"]:
            new[:case["chunks"]] = _ints(g, 1, case["chunk"], case["chunks"])
            new = new[torch.randperm(seqs, generator=g)]
        if seqs >= 16:  # padding entries of a batch of a fixed size
            new[-2:] = 0
        need = int((_pages(lens + new, page) - held).sum())
        width = int(_pages(torch.tensor(ctx + case["chunk"]), page))
        pool = int(held.sum()) + max(1, int(need * case["spare"]))
        table, order = _tables(g, held, width, pool)
        free = torch.zeros(pool, dtype=torch.int32)
        rest = order[int(held.sum()):]
        free[:rest.numel()] = rest
        tokens = seqs + case["chunks"] * case["chunk"]
        s |= dict(cache_seqlens=_i32(lens), q_lens=_i32(new), block_table=table.to(DEV),
                  free_pages=free.to(DEV), free_count=_i32(torch.tensor([rest.numel()])),
                  free_count_out=_i32(torch.zeros(1)), cu_seqlens_q=_i32(torch.zeros(seqs + 1)),
                  seqlens_k=_i32(torch.zeros(seqs)),
                  slot_mapping=torch.zeros(tokens, dtype=torch.int64, device=DEV),
                  positions=_i32(torch.zeros(tokens)))
    elif op == "release":
        keep = lens.clone()
        few = torch.randperm(seqs, generator=g)
        keep[few[:case["done"]]] = 0
        some = few[case["done"]::4]
        keep[some] = (lens[some] - _ints(g, 1, 7, some.numel())).clamp(min=0)
        pool = seqs * int(_pages(torch.tensor(ctx), page)) + 100
        table, order = _tables(g, held, int(_pages(torch.tensor(ctx), page)), pool)
        free = torch.zeros(pool, dtype=torch.int32)
        free[:100] = order[-100:]
        s |= dict(cache_seqlens=_i32(lens), keep_lens=_i32(keep), block_table=table.to(DEV),
                  free_pages=free.to(DEV), free_count=_i32(torch.tensor([100])),
                  free_count_out=_i32(torch.zeros(1)), seqlens_out=_i32(torch.zeros(seqs)))
    elif op == "append":
        n, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        dt, rot = DTYPES[case["dtype"]], case["rot"]
        e4m3 = case["cache"] == "e4m3"
        pool = _pages(n, page) + 3
        # one projection gives q, k and v as slices of the same rows
        qkv = _normal(dg, (n, hq + 2 * hkv, d), dt)
        scale = [0.5 + torch.rand(hkv, generator=dg, device=DEV) for _ in range(2)]
        scale = [x * (4.5 / E4M3_MAX) for x in scale]
        shape = (pool, page, hkv, d)
        caches = [_cache(dg, shape, x) if e4m3 else _normal(dg, shape, dt) for x in scale]
        slots = torch.randperm(pool * page, generator=dg, device=DEV)[:n]
        if n >= 16:  # rows of padding
            slots[-2:] = -1
        length = 32768
        at = torch.randint(0, length - 8192, (case["axes"], 1), generator=dg, device=DEV)
        pos = (at + torch.randint(0, 8192, (case["axes"], n), generator=dg, device=DEV))
        freq = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
        angle = torch.arange(length, device=DEV, dtype=torch.float64)[:, None] * freq
        s |= dict(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], k_cache=caches[0],
                  v_cache=caches[1], k_scale=scale[0] if e4m3 else None,
                  v_scale=scale[1] if e4m3 else None, slot_mapping=slots.to(torch.int64),
                  positions=pos.to(torch.int32), cos=angle.cos().to(dt), sin=angle.sin().to(dt),
                  even_odd=case["pairs"] == "even_odd", axes=_pair_axes(case["axes"], rot // 2),
                  q_out=torch.empty((n, hq, d), dtype=dt, device=DEV))
    else:
        seqs, hq, hkv, d = case["seqs"], case["hq"], case["hkv"], case["d"]
        new = torch.ones(seqs, dtype=torch.int64)
        new[:case["chunks"]] = torch.linspace(case["chunk_lo"], case["chunk_hi"],
                                              case["chunks"]).long()
        lens = torch.maximum(_ints(g, case["ctx_lo"], case["ctx_hi"], seqs), new)
        order = torch.randperm(seqs, generator=g)
        new, lens = new[order], lens[order]
        held = _pages(lens, page)
        width, pool = int(held.max()), int(held.sum())
        table, _ = _tables(g, held, width, pool)
        cu = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)])
        scale = [(0.5 + torch.rand(hkv, generator=dg, device=DEV)) * (4.5 / E4M3_MAX)
                 for _ in range(2)]
        dt = DTYPES[case["dtype"]]
        shape = (pool, page, hkv, d)
        total = int(cu[-1])
        s |= dict(q=_normal(dg, (total, hq, d), dt), k_cache=_cache(dg, shape, scale[0]),
                  v_cache=_cache(dg, shape, scale[1]), k_scale=scale[0], v_scale=scale[1],
                  cu_seqlens_q=_i32(cu), seqlens_k=_i32(lens), block_table=table.to(DEV),
                  max_seqlen_q=int(new.max()), max_seqlen_k=int(lens.max()),
                  out=torch.empty((total, hq, d), dtype=dt, device=DEV),
                  lse=torch.empty((hq, total), device=DEV))
    return s


def _pair_axes(axes, pairs):
    """The axis of each rotated pair: sections of the pairs, as near to equal as they come."""
    return [p * axes // pairs for p in range(pairs)]


# ------------------------------------------------------------------ one pass
def run(state):
    return {"plan": _run_plan, "release": _run_release, "append": _run_append,
            "attend": _run_attend}[state["op"]](state)


def _run_plan(s):
    names = ("cu_seqlens_q", "seqlens_k", "slot_mapping", "positions", "block_table",
             "free_count_out")
    if own:
        import paged_kv_cache_page_gb300 as pa
        pa.pa_plan_step(s["cache_seqlens"], s["q_lens"], s["block_table"], s["free_pages"],
                        s["free_count"], s["page"], s["cu_seqlens_q"], s["seqlens_k"],
                        s["slot_mapping"], s["positions"], s["free_count_out"])
        return {n: s[n] for n in names}
    page, table = s["page"], s["block_table"]
    tokens, width = s["slot_mapping"].numel(), table.shape[1]
    old, new = s["cache_seqlens"].long(), s["q_lens"].long()
    free = s["free_count"].long()
    good = (old >= 0) & (new >= 0) & (old + new <= width * page)
    new = torch.where(good, new, 0)
    held = _pages(old, page)
    need = torch.where(good, _pages(old + new, page) - held, 0)
    # requests are taken in order up to the first that the free pages or the rows do not hold
    fits = (need.cumsum(0) <= free) & (new.cumsum(0) <= tokens)
    new, need = torch.where(fits, new, 0), torch.where(fits, need, 0)
    ends, after = new.cumsum(0), need.cumsum(0)
    col = torch.arange(width, device=DEV)[None, :] - held[:, None]
    fresh = (col >= 0) & (col < need[:, None])
    at = torch.where(fresh, free - 1 - (after - need)[:, None] - col, 0)
    s["block_table"].copy_(torch.where(fresh, s["free_pages"][at], table))
    row = torch.arange(tokens, device=DEV)
    live = row < ends[-1]
    seq = torch.searchsorted(ends, row, right=True).clamp(max=ends.numel() - 1)
    pos = torch.where(live, old[seq] + row - (ends - new)[seq], 0)
    slot = table[seq, pos // page].long() * page + pos % page
    s["cu_seqlens_q"][1:] = ends
    s["seqlens_k"].copy_(old + new)
    s["slot_mapping"].copy_(torch.where(live, slot, -1))
    s["positions"].copy_(pos)
    s["free_count_out"].copy_(free - after[-1:])
    return {n: s[n] for n in names}


def _run_release(s):
    if own:
        import paged_kv_cache_page_gb300 as pa
        pa.pa_release_pages(s["cache_seqlens"], s["keep_lens"], s["block_table"], s["free_pages"],
                            s["free_count"], s["page"], s["seqlens_out"], s["free_count_out"])
        return {n: s[n] for n in ("free_pages", "seqlens_out", "free_count_out")}
    page, pool = s["page"], s["free_pages"].numel()
    lens = s["cache_seqlens"].long()
    keep = torch.minimum(s["keep_lens"].long(), lens)
    col = torch.arange(s["block_table"].shape[1], device=DEV)[None, :]
    gone = ((col >= _pages(keep, page)[:, None]) & (col < _pages(lens, page)[:, None])).reshape(-1)
    rank = gone.long().cumsum(0)
    at = torch.where(gone, s["free_count"].long() + rank - 1, pool)
    grown = torch.cat([s["free_pages"], s["free_pages"][:1]])
    grown[at] = torch.where(gone, s["block_table"].reshape(-1), 0)
    s["free_pages"].copy_(grown[:pool])
    s["seqlens_out"].copy_(keep)
    s["free_count_out"].copy_(s["free_count"] + rank[-1:])
    return {n: s[n] for n in ("free_pages", "seqlens_out", "free_count_out")}


def _turned(x, cos, sin, rot, even_odd):
    """x [N, H, D] with its first rot features rotated, pairs under cos / sin [N, 1, rot / 2]."""
    if even_odd:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    y, z = a * cos - b * sin, a * sin + b * cos
    both = torch.stack([y, z], -1).flatten(-2) if even_odd else torch.cat([y, z], -1)
    return torch.cat([both, x[..., rot:]], -1)


def _stored(x, cache, scale):
    if scale is None:
        return x.to(cache.dtype)
    return (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype)


def _run_append(s):
    names = ("q_out", "k_cache", "v_cache")
    if own:
        import paged_kv_cache_page_gb300 as pa
        pa.pa_rotary_append_varlen(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                                   s["slot_mapping"], positions=s["positions"],
                                   rotary_cos=s["cos"], rotary_sin=s["sin"],
                                   rotary_interleaved=s["even_odd"], pair_axis=s["axes"],
                                   k_scale=s["k_scale"], v_scale=s["v_scale"], q_out=s["q_out"])
        return {n: s[n] for n in names}
    pairs = s["cos"].shape[1]
    pos = s["positions"][torch.tensor(s["axes"], device=DEV)].long().T  # [tokens, pairs]
    pair = torch.arange(pairs, device=DEV)
    cos, sin = s["cos"][pos, pair].float()[:, None], s["sin"][pos, pair].float()[:, None]
    turn = lambda x: _turned(x.float(), cos, sin, 2 * pairs, s["even_odd"])  # noqa: E731
    s["q_out"].copy_(turn(s["q"]))
    slots, page = s["slot_mapping"], s["page"]
    live = slots >= 0
    for name, x in (("k", turn(s["k"])), ("v", s["v"].float())):
        cache = s[name + "_cache"]
        rows = _stored(x, cache, s[name + "_scale"])
        at = torch.where(live, slots, 0)
        as_bits = torch.uint8 if cache.dtype == torch.float8_e4m3fn else torch.int16
        flat = cache.view(as_bits).view(-1, *cache.shape[2:])
        ahead = torch.cat([flat, flat[:1]])  # one more row takes what has no slot
        ahead[torch.where(live, at, flat.shape[0])] = rows.view(as_bits)
        flat.copy_(ahead[:-1])
    return {n: s[n] for n in names}


def _run_attend(s):
    if own:
        import paged_kv_cache_page_gb300 as pa
        pa.pa_fwd_varlen_e4m3(s["q"], s["k_cache"], s["v_cache"], s["cu_seqlens_q"],
                              s["seqlens_k"], s["block_table"], s["max_seqlen_q"],
                              s["max_seqlen_k"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                              causal=True, out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    q, kc, table = s["q"], s["k_cache"], s["block_table"].long().clamp(min=0)
    total, hq, d = q.shape
    hkv = kc.shape[2]
    seqs, most = table.shape[0], s["max_seqlen_q"]
    cu = s["cu_seqlens_q"].long()
    begin, new, lens = cu[:-1], cu[1:] - cu[:-1], s["seqlens_k"].long()

    def keys(cache, scale):  # [seqs, hkv, keys, d]
        x = cache[table].float() * scale[:, None]
        return x.flatten(1, 2).transpose(1, 2)

    i = torch.arange(most, device=DEV)
    rows = (begin[:, None] + i).clamp(max=total - 1)
    qq = q[rows].float().reshape(seqs, most, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    k = keys(kc, s["k_scale"])
    score = (qq.reshape(seqs, hkv, -1, d) * (1.0 / math.sqrt(d))) @ k.transpose(-1, -2)
    t = torch.arange(k.shape[2], device=DEV)
    seen = (t <= (i[None, :] + (lens - new)[:, None])[..., None]) & (t < lens[:, None, None])
    score = score.view(seqs, hkv, hq // hkv, most, -1)
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    score = score.sub_(top).exp_()
    norm = score.sum(-1, keepdim=True)
    del k
    o = score.view(seqs, hkv, -1, t.numel()) @ keys(s["v_cache"], s["v_scale"])
    o = o.view(seqs, hkv, hq // hkv, most, d) / norm
    lse = (top + norm.log()).squeeze(-1)
    row = torch.arange(total, device=DEV)
    seq = torch.searchsorted(cu[1:], row, right=True)
    at = row - begin[seq]
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(seqs, most, hq, d)[seq, at])
    s["lse"].copy_(lse.permute(0, 3, 1, 2).reshape(seqs, most, hq)[seq, at].T)
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ what a pass has to do
def work(case):
    op, page = case["op"], case["page"]
    if op == "plan":
        seqs, tokens = case["seqs"], case["seqs"] + case["chunks"] * case["chunk"]
        fresh = seqs // page + case["chunks"] * case["chunk"] // (2 * page)
        # lengths in; cumulative lengths, key counts, a slot and a position a row out; each new
        # page read from the pool and written to its table, each old one that gets tokens read
        return dict(bytes=seqs * 20 + tokens * 12 + fresh * 8, flops=0)
    if op == "release":
        seqs, gone = case["seqs"], case["done"] * (case["ctx"] // (2 * page) + 1)
        return dict(bytes=seqs * 12 + gone * 8, flops=0)
    if op == "append":
        n, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        held = 1 if case["cache"] == "e4m3" else 2
        bytes_ = n * d * ((hq + 2 * hkv) * 2 + hq * 2 + 2 * hkv * held)
        bytes_ += n * (8 + 4 * case["axes"] + 2 * case["rot"])
        return dict(bytes=bytes_, flops=n * (hq + hkv) * case["rot"] * 3)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    ctx = (case["ctx_lo"] + case["ctx_hi"]) / 2
    chunk = (case["chunk_lo"] + case["chunk_hi"]) / 2
    chunks, ones = case["chunks"], case["seqs"] - case["chunks"]
    rows = chunks * chunk + ones
    pairs = chunks * chunk * max(1.0, max(ctx, chunk) - chunk / 2) + ones * ctx
    bytes_ = (case["seqs"] * ctx * hkv * d * 2 + rows * hq * (4 * d + 4)
              + case["seqs"] * (8 + 4 * ctx / page))
    return dict(bytes=bytes_, flops=4 * d * hq * pairs)


# ------------------------------------------------------------------ the definitions, in 64 bits
def _e4m3(x):
    """x rounded to the nearest value of four exponent and three mantissa bits (ties to the even
    one), at most 448."""
    a = x.abs().clamp(max=E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign(torch.round(a / step) * step, x)


def exact(case, seed):
    if case["op"] in ("plan", "release"):
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        half = s["cos"].shape[1]
        first = [2 * p if s["even_odd"] else p for p in range(half)]
        second = [2 * p + 1 if s["even_odd"] else p + half for p in range(half)]
        angle = [torch.stack([s[n].double()[s["positions"][a].long(), p]
                              for p, a in enumerate(s["axes"])], 1)[:, None] for n in ("cos", "sin")]
        turned = {}
        for name in ("q", "k"):
            x = s[name].double()
            y = x.clone()
            y[..., first] = x[..., first] * angle[0] - x[..., second] * angle[1]
            y[..., second] = x[..., second] * angle[0] + x[..., first] * angle[1]
            turned[name] = y
        out = {"q_out": turned["q"]}
        slots = s["slot_mapping"]
        live = slots >= 0
        for name, x in (("k", turned["k"]), ("v", s["v"].double())):
            cache, scale = s[name + "_cache"].double(), s[name + "_scale"]
            if scale is not None:
                x = _e4m3(x / scale.double()[:, None])
            cache.view(-1, *cache.shape[2:])[slots[live]] = x[live]
            out[name + "_cache"] = cache
        return out
    total, hq, d = s["q"].shape
    hkv = s["k_cache"].shape[2]
    out = torch.zeros((total, hq, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((hq, total), dtype=torch.float64, device=DEV)
    cu, lens = s["cu_seqlens_q"].tolist(), s["seqlens_k"].tolist()
    for b, n in enumerate(lens):
        ids = s["block_table"][b, :_pages(n, s["page"])].long()
        k = s["k_cache"][ids].flatten(0, 1)[:n].double() * s["k_scale"].double()[:, None]
        v = s["v_cache"][ids].flatten(0, 1)[:n].double() * s["v_scale"].double()[:, None]
        rows = slice(cu[b], cu[b + 1])
        m = cu[b + 1] - cu[b]
        sees = torch.arange(n, device=DEV) <= torch.arange(m, device=DEV)[:, None] + n - m
        group = hq // hkv
        for h in range(hkv):
            q = s["q"][rows, h * group:(h + 1) * group].double()
            x = torch.einsum("mgd,nd->gmn", q, k[:, h]) / math.sqrt(d)
            x = x.masked_fill(~sees, -math.inf)
            z = torch.logsumexp(x, -1)
            out[rows, h * group:(h + 1) * group] = torch.einsum(
                "gmn,nd->mgd", (x - z[..., None]).exp(), v[:, h])
            lse[h * group:(h + 1) * group, rows] = z
    return {"out": out, "lse": lse}
