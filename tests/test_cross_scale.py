"""Scales that pa_fwd_cross refuses: scores are taken times scale log2(e) in fp32 (CPU)."""

import pytest

import paged_kv_cache_page_gb300 as pa
from paged_kv_cache_page_gb300 import build as pabuild

P = 4096  # stands for an aligned device pointer; never read by a refused call


@pytest.mark.parametrize("scale,ok", [(0.125, True), (1e-30, True), (2.3e38, True), (2.4e38, False), (3.4e38, False)])
def test_scale_times_log2_e_is_finite(scale, ok):
    pabuild.build()
    lib = pa.load_library()
    # (a misaligned q is refused behind the scale)
    rc = lib.pa_fwd_cross(P + 2, 256, 64, P, 256, 64, P, 256, 64, P, P, None, None, 1, 4, 50, 4, 50, 4, 2, 64, scale, P,
                          None, None, 0, None, pa.PA_F16, None)
    assert rc == pa.PA_ERR_INVALID_ARG
    assert (b"scale" in lib.pa_last_error_string()) != ok
