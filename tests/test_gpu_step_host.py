"""What the host does around the serving-step calls: threads that call at the same time."""

import ctypes
import threading

import pytest
import torch

import paged_kv_cache_page_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_batches_of_different_sizes_from_two_threads():
    """Launches whose shared memory differs, by way of the C ABI, which leaves the threads free to run."""
    lib = pa.load_library()
    codes = {}

    def work(B, calls):
        z = lambda n, t=torch.int32: torch.zeros(n, dtype=t, device=DEV)  # noqa: E731
        cached, new, table, free, count = z(B), z(B), z((B, 2)), z(8), z(1)
        cu, lens, slots, pos, left = z(B + 1), z(B), z(4, torch.int64), z(4), z(1)
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        got = set()
        for _ in range(calls):
            got.add(lib.pa_plan_step(
                cached.data_ptr(), new.data_ptr(), B, table.data_ptr(), 2, 2, 16, free.data_ptr(),
                count.data_ptr(), 8, cu.data_ptr(), lens.data_ptr(), slots.data_ptr(), pos.data_ptr(), 4,
                left.data_ptr(), None, ctypes.c_void_p(stream.cuda_stream)))
        stream.synchronize()
        codes[B] = got, lib.pa_last_error_string()

    threads = [threading.Thread(target=work, args=(B, 20000)) for B in (4096, 3500)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(c[0] == {pa.PA_OK} for c in codes.values()), codes


def test_the_interpreter_lock_is_not_held_over_a_launch():
    """In the place of the library's entry the interpreter's own question whether the calling thread
    holds the lock."""
    native = pa._native or pa._load_native()
    lib = pa.load_library()
    entries = [ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.pa_plan_step, lib.pa_release_pages, lib.pa_rotary_append_varlen, lib.pa_fwd_varlen_e4m3,
        lib.pa_fwd_varlen_e4m3_workspace_size)]
    ask = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    x = torch.zeros((3, 2, 64), dtype=torch.float16, device=DEV)
    c = torch.zeros((4, 16, 2, 64), dtype=torch.float8_e4m3fn, device=DEV)
    try:
        native.bind(ask, ask, ask, ask, entries[4])
        held = [
            native.plan_step(i32([1]), i32([1]), i32([[0]]), i32([0]), i32([0]), 16, i32([0, 0]), i32([0]),
                             torch.zeros(2, dtype=torch.int64, device=DEV), i32([0, 0]), i32([0]), None),
            native.release_pages(i32([1]), i32([1]), i32([[0]]), i32([0]), i32([0]), 16, i32([0]), i32([0]),
                                 None),
            native.rotary_append_varlen(x, x, x, c, c, torch.zeros(3, dtype=torch.int64, device=DEV), None,
                                        None, None, False, None, None, None, x, None),
            native.fwd_varlen_e4m3(x, c, c, i32([0, 3]), i32([3]), i32([[0]]), 3, 3, None, None, None, True,
                                   torch.empty_like(x), None, None, None)]
    finally:
        native.bind(*entries)
    assert held == [0] * 4
