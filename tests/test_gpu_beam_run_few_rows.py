"""The searches of test_gpu_beam_run with the bound of a step's rows: K tokens of G heads a request, the cross
attention kernel for few rows."""

import pytest

import paged_kv_cache_page_gb300 as pa
import test_gpu_beam_run as search

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("run,searches", [("test_a_search_against_plain_lists", 1),
                                          ("test_a_captured_step_replayed", 2)])
def test_with_the_bound_of_a_step(run, searches, monkeypatch):
    assert search.K * search.HQ // search.HKV <= 16
    real, bounds = pa.pa_fwd_cross, []

    def call(q, k, v, cu_q, cu_k, max_q, max_k, **kw):
        if len(bounds) >= searches * search.LAYERS:  # behind the prompts
            max_q = search.K
        bounds.append(max_q)
        return real(q, k, v, cu_q, cu_k, max_q, max_k, **kw)

    monkeypatch.setattr(pa, "pa_fwd_cross", call)
    getattr(search, run)()
    assert search.K in bounds

