"""What pa_beam_reorder may be given: no page in the tables of two requests (CPU)."""

import os

from oracle import beam

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_page_of_two_requests_would_be_given_back_under_its_other_owner():
    # requests 0 and 1 hold page 5, a common prompt's: 0 ends, then 1 does
    rows, lens = [[5, 6], [5, 7]], [20, 20]
    first = beam.reorder([[-1], [0]], lens, rows, [], 16, 8)
    assert 5 in first["free"] and 5 in first["rows"][1]
    second = beam.reorder([[0], [-1]], first["lens"], first["rows"], first["free"], 16, 8)
    assert second["free"].count(5) == 2


def test_the_contract_excludes_it():
    text = open(os.path.join(ROOT, "include", "pagedattn.h")).read()
    text = " ".join(text[text.index("* pa_beam_reorder --"):text.index("PA_API int pa_beam_reorder")].split(" * "))
    text = " ".join(text.split())
    assert "No page is in the tables of two requests" in text.replace(" * ", " ")
    assert "such as all of the request's beams hold" not in text.replace(" * ", " ")
