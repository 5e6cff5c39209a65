"""What the host does around the beam search calls: threads that call at the same time, two streams,
two captured graphs."""

import ctypes
import threading

import pytest
import torch

import paged_kv_cache_page_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_the_interpreter_lock_is_not_held_over_a_launch():
    """In the place of the library's entry the interpreter's own question whether the calling thread
    holds the lock."""
    native = pa._native or pa._load_native()
    lib = pa.load_library()
    entries = [ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.pa_beam_select, lib.pa_beam_reorder, lib.pa_copy_pages, lib.pa_fwd_cross,
        lib.pa_fwd_cross_workspace_size)]
    ask = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    x = torch.zeros((3, 2, 64), dtype=torch.float16, device=DEV)
    try:
        native.bind_beam(ask, ask, ask, ask, entries[4])
        held = [
            native.beam_select(torch.zeros((1, 2, 9), device=DEV), torch.zeros((1, 2), device=DEV), None, -1,
                               torch.zeros((1, 2), device=DEV), i32([[0, 0]]), i32([[0, 0]]), None, None),
            native.beam_reorder(i32([[0, 0]]), i32([1, 1]), i32([[0], [1]]), i32([0, 0]), i32([0]), 16,
                                i32([[0], [1]]), i32([1, 1]), i32([[0] * 3] * 2), i32([0]), None),
            native.copy_pages(i32([[0, 1, 2]]), [torch.zeros((4, 16, 2, 64), device=DEV)], None),
            native.fwd_cross(x, x, x, i32([0, 3]), i32([0, 3]), 3, 3, None, None, None, torch.empty_like(x),
                             None, None, None)]
    finally:
        native.bind_beam(*entries)
    assert held == [0] * 4


def work_of(seed):
    """A call of each kind on tensors of its own, and its results."""
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((7, 4, 9001), generator=g).bfloat16().to(DEV)
    scores = -torch.rand((7, 4), generator=g).to(DEV)
    q = torch.randn((300, 8, 64), generator=g).half().to(DEV)
    kv = torch.randn((500, 2, 2, 64), generator=g).half().to(DEV)
    cu_q, cu_k = i32([0, 260, 300]), i32([0, 400, 500])
    rows = torch.randperm(64, generator=g).int().view(8, 8)
    table, pool = rows.to(DEV), torch.arange(64, 96).int().to(DEV)
    parents = torch.randint(0, 4, (2, 4), generator=g).int().to(DEV)
    lens, count = i32([100] * 8), i32([32])

    def call():
        a = pa.pa_beam_select(logits, scores, 6, end_token=3)
        b = pa.pa_fwd_cross(q, kv[:, 0], kv[:, 1], cu_q, cu_k, 260, 400)
        c = pa.pa_fwd_cross(q[:8], kv[:, 0], kv[:, 1], i32_8, cu_k, 4, 400)
        out, left = torch.zeros_like(table), torch.zeros_like(count)
        d = pa.pa_beam_reorder(parents, lens, table, free, count, 16, block_table_out=out,
                               seqlens_out=torch.zeros_like(lens), free_count_out=left)
        return [*a, *b, *c, *d, left]

    i32_8 = i32([0, 4, 8])
    free = torch.cat([pool, torch.zeros(64, dtype=torch.int32, device=DEV)])
    return call


def test_calls_from_several_threads_and_streams():
    calls = [work_of(s) for s in range(3)]
    want = [[t.clone() for t in c()] for c in calls]
    got = [None] * 3

    def run(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(30):
                got[i] = calls[i]()
        stream.synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for w, x in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, x))


def test_two_captured_graphs_side_by_side():
    calls, graphs, got = [work_of(s) for s in (5, 6)], [], []
    want = [[t.clone() for t in c()] for c in calls]
    for c in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(c())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for w, x in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, x))
