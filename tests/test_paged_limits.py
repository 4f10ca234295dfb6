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


GB = 1 << 30


def big(pa, dtype, d=128, heads=8, slots=1024):
    return cache(pa, slots=slots, heads=heads, head_dim=d, page_size=64, table_width=512, k_pages=30000, v_pages=30000, cache_dtype=dtype)


@pytest.mark.parametrize("slots", [64, 256, 1024, 4096])
def test_workspace_of_a_prompt_among_single_tokens(pa, slots):
    """512 tokens of a prompt beside a token of every other slot: not a chunk's workspace for every slot."""
    c = big(pa, pa.PATH_BF16, slots=slots)
    n = pa.path_paged_workspace_size(c, desc(pa, heads_q=32, total_tokens=512 + slots - 1, max_new=512))
    singles = pa.path_paged_workspace_size(c, desc(pa, heads_q=32, total_tokens=slots, max_new=1))
    assert 0 < n <= 4 * GB + singles


def test_workspace_of_stated_prompts(pa):
    """One slot with several tokens, stated: the prompt's own workspace, whatever the slots."""
    c = big(pa, pa.PATH_BF16, slots=4096)
    n = pa.path_paged_workspace_size(c, desc(pa, heads_q=32, total_tokens=512 + 4095, max_new=512, max_multi=1))
    alone = pa.path_paged_workspace_size(c, desc(pa, heads_q=32, total_tokens=512, max_new=512, max_multi=1))
    assert alone <= n <= alone + 4 * 8 * 4096 * 8  # (the plan's numbers of each slot stay)
    assert n < 0.12 * GB
    assert extend(pa, c, desc(pa, heads_q=32, max_multi=-1), nbytes=1 << 40) == 1


@pytest.mark.parametrize("total,max_new,heads_q", [(16 * 4096, 4096, 32), (64 * 4096, 4096, 32), (1 << 20, 1 << 20, 8), (2048, 2, 128)])
def test_workspace_of_many_prompts(pa, total, max_new, heads_q):
    """Rounds of slots: four gigabytes, or what one slot's pass needs."""
    c = big(pa, pa.PATH_BF16)
    n = pa.path_paged_workspace_size(c, desc(pa, heads_q=heads_q, total_tokens=total, max_new=max_new))
    one = pa.path_paged_workspace_size(c, desc(pa, heads_q=heads_q, total_tokens=max_new, max_new=max_new))
    singles = pa.path_paged_workspace_size(c, desc(pa, heads_q=heads_q, total_tokens=1024, max_new=1))
    assert 0 < n <= max(one, 4 * GB) + singles


def test_workspace_grows_with_the_call(pa):
    """A workspace for the largest call holds every smaller one, across the step to several rounds."""
    c = big(pa, pa.PATH_BF16)
    size = lambda total, most: pa.path_paged_workspace_size(c, desc(pa, heads_q=32, total_tokens=total, max_new=most))  # noqa: E731
    sizes = [size(total, 2048) for total in range(2048, 65536, 1700)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    sizes = [size(40000, most) for most in range(20, 20000, 517)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("slots,total,max_new,heads_q", [(4096, 512 + 4095, 512, 32), (16384, 512 + 16383, 512, 32), (1024, 64 * 4096, 4096, 32)])
def test_workspace_of_fp32_calls(pa, slots, total, max_new, heads_q):
    c = big(pa, pa.PATH_FP32, slots=slots)
    size = lambda **kw: pa.path_paged_workspace_size(c, desc(pa, heads_q=heads_q, **kw))  # noqa: E731
    one, singles = size(total_tokens=max_new, max_new=max_new, max_multi=1), size(total_tokens=slots, max_new=1)
    assert 0 < size(total_tokens=total, max_new=max_new) <= max(one, 4 * GB) + singles
    assert size(total_tokens=total, max_new=max_new, max_multi=1) < 0.3 * GB
