"""pa_fwd_varlen_e4m3 against the oracle in 64 bits on the dequantised cache (tolerances derived in
e4m3_util), and what must not change a result."""

import pytest
import torch

import paged_kv_cache_page_gb300 as pa
from e4m3_util import DEV, DT, batch, call, check

pytestmark = pytest.mark.gpu

HEADS = [(4, 2, 64), (8, 1, 64), (6, 6, 64), (8, 2, 128), (3, 3, 128), (20, 4, 128), (32, 1, 128)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", HEADS)
def test_single_tokens(heads, dtype):
    lens = [1, 2, 15, 16, 17, 31, 100, 513, 1000]
    w = batch([1] * len(lens), lens, *heads, dtype, seed=sum(heads))
    err = pa.new_err_word(DEV)
    out, lse = call(w, err=err)
    torch.cuda.synchronize()
    assert err[0].item() == 0
    check(w, out, lse)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 2, 128), (5, 5, 128), (12, 1, 64)])
def test_chunks_and_single_tokens(heads, causal, page):
    q_lens = [1, 5, 0, 33, 1, 17, 3, 130, 0]
    k_lens = [300, 5, 0, 70, 0, 40, 290, 131, 7]
    w = batch(q_lens, k_lens, *heads, "bf16" if page % 64 else "f16", page=page, seed=page)
    out, lse = call(w, causal=causal)
    check(w, out, lse, causal=causal)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [(8, 2, 64), (8, 8, 128), (16, 2, 128)])
def test_long_chunks(heads, dtype):
    q_lens, k_lens = [257, 1, 400, 64, 128], [600, 800, 400, 64, 1000]
    w = batch(q_lens, k_lens, *heads, dtype, page=32, seed=9)
    out, lse = call(w)
    check(w, out, lse)


@pytest.mark.parametrize("heads", [(32, 32, 64), (24, 24, 128), (7, 1, 64), (9, 3, 128), (96, 32, 128)])
def test_chunks_of_many_heads(heads):
    """More streams than CTAs (equal shares that cut streams), group sizes that divide no tile, rows
    that end inside a tile, and a chunk longer than its keys."""
    q_lens, k_lens = [300, 129, 1, 513, 200, 0], [700, 129, 50, 1300, 90, 0]
    w = batch(q_lens, k_lens, *heads, "bf16", page=32, seed=sum(heads))
    err = pa.new_err_word(DEV)
    out, lse = call(w, err=err)
    assert err.tolist() == [0] * 4
    check(w, out, lse)
    again, lse2 = call(w)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("b,q_len", [(2, 16), (2, 17), (63, 16), (64, 12), (64, 13), (64, 16), (65, 1)])
def test_around_the_limits_between_the_kernels(b, q_len):
    """48 and 64 rows per kv head, with few and with many streams; single tokens beside them."""
    q_lens = [q_len if i % 3 else 1 for i in range(b)]
    w = batch(q_lens, [(37 * i) % 190 + 18 for i in range(b)], 4, 1, 64, "bf16", seed=b + q_len)
    out, lse = call(w)
    check(w, out, lse)


@pytest.mark.parametrize("heads,dtype", [((4, 1, 128), "f16"), ((8, 2, 64), "bf16"), ((1, 1, 128), "bf16")])
@pytest.mark.parametrize("causal", [True, False])
def test_a_chunk_over_a_long_prefix_is_split_and_joined(heads, dtype, causal):
    w = batch([150], [9001], *heads, dtype, page=128, seed=17, peaky=4.0)
    out, lse = call(w, causal=causal)
    check(w, out, lse, causal=causal)


@pytest.mark.parametrize("d", [64, 128])
def test_chunks_with_shifting_maxima_and_odd_scales(d):
    """Rising maxima inside a tile and from tile to tile (probabilities already written are scaled
    again), a negative and a zero scale, rows of zeros and of large magnitude."""
    w = batch([200, 90], [900, 400], 6, 3, d, "bf16", seed=18)
    k = w["k_cache"]
    for b in range(2):
        for j, page in enumerate(w["block_table"][b].tolist()):
            if page >= 0:
                step = torch.arange(16, device=DEV)[:, None, None] * 0.3
                k[page] = (k[page].float() * 0.01 + j * 3.0 + step).clamp(-448, 448).to(k.dtype)
    w["q"] = w["q"].abs()
    w["q"][7] = 0
    w["q"][9] *= 64
    check(w, *call(w))
    w["k_scale"] = w["k_scale"] * torch.tensor([-1.0, 0.0, 1.0], device=DEV)
    check(w, *call(w))


@pytest.mark.parametrize("heads", [(1, 1, 128), (1, 1, 64), (64, 1, 128), (8, 8, 128)])
@pytest.mark.parametrize("q_len", [1, 4])
def test_one_long_sequence_is_split_and_joined(heads, q_len):
    w = batch([q_len], [20011], *heads, "f16", page=64, seed=3, peaky=3.0)
    out, lse = call(w)
    check(w, out, lse)
    again, lse2 = call(w)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_rows_that_see_no_key():
    # more query rows than keys: the first ones are empty
    w = batch([20, 3, 40], [5, 0, 39], 4, 2, 64, "f16", seed=1)
    out, lse = call(w)
    check(w, out, lse)
    assert (out[:15] == 0).all() and (lse[:, :15] == -float("inf")).all()
    assert (out[20:24] == 0).all() and (lse[:, 20:24] == -float("inf")).all()


def test_many_short_and_empty_sequences():
    import random
    rng = random.Random(2)
    q = [rng.choice((0, 1, 1, 2)) for _ in range(4096)]
    k = [rng.choice((0, 1, 16, 17, 40)) for _ in range(4096)]
    w = batch(q, k, 4, 2, 64, "bf16", seed=2)
    out, lse = call(w)
    check(w, out, lse, seqs=set(range(0, 4096, 7)) | set(range(4080, 4096)))


@pytest.mark.parametrize("d,every", [(64, 50), (128, 3)])
def test_chunks_among_the_most_sequences(d, every):
    """4096 entries of which some are chunks for the tcgen05 kernel, the last one among them."""
    q = [40 if i % every == 0 or i == 4095 else i % 2 for i in range(4096)]
    k = [90 if m == 40 and i % 4 else m + i % 30 for i, m in enumerate(q)]
    w = batch(q, k, 2, 1, d, "f16" if d == 64 else "bf16", seed=d)
    err = pa.new_err_word(DEV)
    out, lse = call(w, err=err)
    assert err.tolist() == [0] * 4
    check(w, out, lse, seqs=set(range(0, 4096, 37)) | set(range(4090, 4096)))


def test_rows_behind_the_last_sequence_stay():
    w = batch([2, 0, 3], [50, 0, 20], 4, 2, 128, "f16", seed=4)
    w["q"] = torch.cat([w["q"], torch.randn(6, 4, 128, device=DEV).half()])
    out = torch.full((11, 4, 128), 7.0, dtype=torch.float16, device=DEV)
    lse = torch.full((4, 11), 7.0, device=DEV)
    call(w, out=out, lse=lse)
    check(w, out, lse)
    assert (out[5:] == 7).all() and (lse[:, 5:] == 7).all()
    out2, none = call(w, return_lse=False)
    assert none is None and torch.equal(out2[:5], out[:5])


def test_strided_views():
    w = batch([3, 1, 40], [60, 500, 40], 8, 2, 128, "bf16", page=32, seed=5)
    out, lse = call(w)
    qkv = torch.randn((44, 12, 128), device=DEV).bfloat16()
    qkv[:, 2:10] = w["q"]
    wide = torch.zeros((w["k_cache"].shape[0], 32, 6, 128), device=DEV).to(torch.float8_e4m3fn)
    wide[:, :, 1:3].view(torch.uint8).copy_(w["k_cache"].view(torch.uint8))
    wide[:, :, 3:5].view(torch.uint8).copy_(w["v_cache"].view(torch.uint8))
    table = torch.full((3, w["block_table"].shape[1] + 5), -3, dtype=torch.int32, device=DEV)
    table[:, :-5] = w["block_table"]
    w2 = dict(w, q=qkv[:, 2:10], k_cache=wide[:, :, 1:3], v_cache=wide[:, :, 3:5],
              block_table=table[:, :-5])
    out2, lse2 = call(w2)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d", [64, 128])
def test_scales(d):
    w = batch([1, 9], [100, 50], 4, 2, d, "f16", seed=6)
    w["k_scale"] = torch.tensor([-0.01, 0.02], device=DEV)
    w["v_scale"] = torch.tensor([0.0, -0.01], device=DEV)
    check(w, *call(w))
    w["k_scale"] = torch.tensor([0.0, 0.01], device=DEV)  # every key weighs the same
    check(w, *call(w))
    w["k_scale"] = w["v_scale"] = None
    check(w, *call(w, scale=1.0 / 4096), scale=1.0 / 4096)


@pytest.mark.parametrize("power", [-100, 60, 120])
def test_query_rows_far_from_one(power):
    """bf16 rows of magnitudes that fp16 does not have."""
    w = batch([1, 18], [90, 200], 4, 2, 128, "bf16", seed=7)
    w["q"] = (w["q"].float() * 2.0 ** power).bfloat16()
    w["q"][3, 1] = 0
    scale = 2.0 ** -power / 128 ** 0.5
    check(w, *call(w, scale=scale), scale=scale)


def test_sharp_and_shifting_maxima():
    """Scores whose maximum grows along the keys, far past what a reference may be passed by."""
    w = batch([1, 30], [800, 300], 2, 1, 64, "f16", seed=8)
    k = w["k_cache"]
    for b in range(2):
        for j, page in enumerate(w["block_table"][b].tolist()):
            if page >= 0:
                k[page] = (k[page].float() * 0.01 + j * 2.0).clamp(-448, 448).to(k.dtype)
    w["q"] = w["q"].abs()
    check(w, *call(w))
    w["q"] = -w["q"]
    check(w, *call(w))


@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 2, 128)])
def test_nan_where_nobody_looks(heads):
    """NaN behind the last key of a page, in pages of nobody, and at keys that a row does not see."""
    q_lens, k_lens = [1, 40, 17, 200], [37, 100, 17, 333]
    w = batch(q_lens, k_lens, *heads, "bf16", seed=10)
    out, lse = call(w)
    clean = (out.clone(), lse.clone())
    nan = 0x7f
    used = {}
    for b, n in enumerate(k_lens):
        for j, page in enumerate(w["block_table"][b].tolist()):
            if page >= 0:
                used[page] = min(16, n - 16 * j)
    for name in ("k_cache", "v_cache"):
        raw = w[name].view(torch.uint8)
        for page in range(raw.shape[0]):
            raw[page, used.get(page, 0):] = nan
    out, lse = call(w)
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])
    # V at the last key of each chunk: only its last row sees it; K at the last key of the third
    starts = [0, 1, 41, 58]
    for b in (1, 2, 3):
        n = k_lens[b]
        page = w["block_table"][b, (n - 1) // 16].item()
        w["v_cache"].view(torch.uint8)[page, (n - 1) % 16, 0, 3] = nan | 0x80
        if b == 2:
            w["k_cache"].view(torch.uint8)[page, (n - 1) % 16, 1, 5] = nan
    out, lse = call(w)
    group = heads[0] // heads[1]
    for b in (1, 2, 3):
        last = starts[b] + q_lens[b] - 1
        assert torch.equal(out[starts[b]:last], clean[0][starts[b]:last])
        assert torch.isnan(out[last, :group, 3]).all()
        rest = torch.ones(heads[2], dtype=torch.bool, device=DEV)
        rest[3] = False
        assert torch.equal(out[last, :group][:, rest], clean[0][last, :group][:, rest])
        assert torch.isnan(out[last, group:]).all().item() == (b == 2)
        assert torch.isnan(lse[group:, last]).all().item() == (b == 2)


def test_bad_tables_and_lengths_are_reported():
    w = batch([1, 2], [100, 60], 4, 2, 64, "f16", seed=11)
    good, _ = call(w)
    table = w["block_table"].clone()
    for bad in (-1, w["k_cache"].shape[0], 2 ** 31 - 1):
        w["block_table"][0, 2] = bad
        err = pa.new_err_word(DEV)
        out, lse = call(w, err=err)
        assert err.tolist()[:2] == [pa.PA_DEVERR_PAGE_OOB, 0]
        assert torch.equal(out[1:], good[1:]) and torch.isfinite(lse).all()
    w["block_table"].copy_(table)
    for bad in (-5, 10 ** 6, 101):
        w["seqlens_k"][0] = bad
        err = pa.new_err_word(DEV)
        out, lse = call(w, err=err)
        assert err.tolist()[:3] == [pa.PA_DEVERR_LENGTH, 0, bad]
        assert torch.equal(out[1:], good[1:]) and (out[0] == 0).all()
    w["seqlens_k"][0] = 100
    # query offsets that go backwards or past the rows stay within them
    for cu in ([0, 5, 3], [-4, 1, 99], [2, 2, 2]):
        w["cu_seqlens_q"].copy_(torch.tensor(cu, dtype=torch.int32))
        out, lse = call(w)
        torch.cuda.synchronize()
        assert out.shape == (3, 4, 64)


def test_empty_calls():
    w = batch([1], [5], 4, 2, 64, "f16")
    w0 = dict(w, q=w["q"][:0])
    out, lse = call(w0)
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)


def test_graphs_share_a_workspace_and_replay_with_new_lengths():
    """Two captured calls with one workspace, replayed in turn after the lengths change."""
    wa = batch([1] * 6, [900, 5, 300, 1, 77, 4000], 8, 2, 128, "bf16", page=32, seed=12)
    wb = batch([3, 50], [2000, 50], 4, 4, 64, "f16", seed=13)
    ws = torch.full((max(pa.fwd_varlen_e4m3_workspace_size(6, 53, 50, 8, 2, 128, 4000),
                         pa.fwd_varlen_e4m3_workspace_size(2, 53, 50, 4, 4, 64, 2000)),), 0xff,
                    dtype=torch.uint8, device=DEV)
    outs, graphs = [], []
    for w in (wa, wb):
        o = torch.empty_like(w["q"])
        l = torch.empty((w["q"].shape[1], w["q"].shape[0]), device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(w, out=o, lse=l, workspace=ws)
        outs.append((o, l))
        graphs.append(g)
    for lens in ([900, 5, 300, 1, 77, 4000], [1, 0, 4000, 640, 3, 16]):
        wa["seqlens_k"].copy_(torch.tensor(lens, dtype=torch.int32))
        wa["k_lens"] = lens
        wa["block_table"].copy_(torch.randint(0, wa["k_cache"].shape[0], wa["block_table"].shape,
                                              dtype=torch.int32))
        for _ in range(3):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for w, (o, l) in zip((wa, wb), outs):
            check(w, o, l)
            eager, eager_l = call(w)
            assert torch.equal(o, eager) and torch.equal(l, eager_l)


def test_two_streams_at_once():
    ws = [batch([1] * 4, [3000, 200, 1500, 8], 8, 2, 128, "f16", seed=s) for s in (20, 21)]
    want = [call(w) for w in ws]
    streams = [torch.cuda.Stream() for _ in ws]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = []
        for w, s in zip(ws, streams):
            with torch.cuda.stream(s):
                got.append(call(w))
    torch.cuda.synchronize()
    for (o, l), (o2, l2) in zip(want, got):
        assert torch.equal(o, o2) and torch.equal(l, l2)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements, its last pages in use."""
    page, hkv, d = 256, 8, 128
    w = batch([1, 20], [700, 600], 8, hkv, d, "bf16", page=page, seed=30)
    small = w["k_cache"].shape[0]
    pages = (1 << 32) // (page * hkv * d) + small
    big = [torch.empty((pages, page, hkv, d), dtype=torch.float8_e4m3fn, device=DEV)
           for _ in range(2)]
    for x, name in zip(big, ("k_cache", "v_cache")):
        x.view(torch.uint8)[pages - small:].copy_(w[name].view(torch.uint8))
    table = torch.where(w["block_table"] >= 0, w["block_table"] + (pages - small), -1)
    out, lse = call(w)
    out2, lse2 = call(dict(w, k_cache=big[0], v_cache=big[1], block_table=table))
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_agrees_with_the_16_bit_call():
    """The same values in a 16-bit cache through pa_fwd_varlen_unified."""
    w = batch([1, 40, 1, 300], [500, 900, 33, 300], 8, 2, 128, "f16", page=16, seed=14)
    w["k_scale"] = torch.full((2,), 2.0 ** -7, device=DEV)
    w["v_scale"] = torch.full((2,), 2.0 ** -7, device=DEV)
    k16, v16 = [(w[n].float() * 2.0 ** -7).to(DT["f16"]) for n in ("k_cache", "v_cache")]
    out, lse = call(w)
    ref, ref_l = pa.pa_fwd_varlen_unified(w["q"], k16, v16, w["cu_seqlens_q"], w["seqlens_k"],
                                          w["block_table"], 300, 900)
    check(w, out, lse)
    assert (out.float() - ref.float()).abs().max() <= 2e-3
    assert (lse - ref_l).abs().max() <= 1e-3
