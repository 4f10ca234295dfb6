"""Host-side checks of the paged cache's later fields and sizes; no GPU is used (fake pointers, nothing is launched)."""
import pytest
import torch

from test_paged_host import FAKE, cache, desc, extend, pa  # noqa: F401  (pa: the fixture)


def test_place_for_extended_counts(pa):
    n = pa.path_pages_workspace_size(cache(pa))
    for ok in (None, FAKE, FAKE + 4):
        assert extend(pa, cache(pa, extended=ok), desc(pa, total_tokens=0)) == 0
    c = cache(pa, extended=FAKE + 2)
    assert extend(pa, c, desc(pa)) == 1 and pa.path_pages_compact(c, FAKE, n, None) == 1
    assert pa.path_paged_advance(c, None, None) == 1


def test_place_for_the_sums_rest(pa):
    for ok in (None, FAKE, FAKE + 16):
        assert extend(pa, cache(pa, a_pool=FAKE, a_rest=ok), desc(pa, total_tokens=0), log_f=FAKE) == 0
    assert extend(pa, cache(pa, a_pool=FAKE, a_rest=FAKE + 8), desc(pa), log_f=FAKE) == 1
