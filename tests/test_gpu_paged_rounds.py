"""Calls whose slots with several new tokens are taken in several rounds of the chunk kernels."""
import pytest
import torch

import paged_ref as R
from test_gpu_paged import DEV, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fox", [False, True])
def test_many_short_prompts(cuda_lib, fox):
    """700 slots of 0 to 5 new tokens in a call that allows 20: more than four gigabytes of chunks hold, so several rounds;
    slots without tokens, with one, left out and empty lie between them."""
    t = [(7 * b) % 40 if b % 23 else -1 for b in range(700)]
    n = [0 if x < 0 else b % 6 for b, x in enumerate(t)]
    n[5] = 20
    c = R.make_case("bf16", 128, 8, 8, 16, t, n, fox, seed=11)
    c["k_table"][10, -(-t[10] // 16) :] = -1  # no page for its new tokens (t[10] = 30, n[10] = 4)
    assert n[10] == 4 and t[10] == 30
    c["k_table"][10, 1] = -1
    ref = R.extend_ref(dict(c, n=n[:10] + [0] + n[11:]), 0.125)
    out = torch.full_like(c["q"], 3.0).to(DEV)
    got, cache = run(c, 0.125, out=out)
    with pytest.raises(RuntimeError, match="page-table"):
        cache.check()
    a, b = int(c["q_start"][10]), int(c["q_start"][11])
    assert (got["o"][a:b] == 3).all()
    R.check_extend(c, got, ref, 0.125, tokens=[i for i in range(sum(n)) if not a <= i < b])
    cache.advance(c["q_start"].to(DEV))
    cache.check()
    assert cache.seq_len.tolist() == [x if x < 0 or i == 10 else x + m for i, (x, m) in enumerate(zip(t, n))]


def test_stated_number_of_prompts(cuda_lib):
    """max_multi holds the first slots with several tokens; the others are left out, single tokens are not."""
    t, n = [40, 5, 100, 0, 64, 33], [30, 1, 20, 17, 1, 40]
    c = R.make_case("bf16", 64, 4, 2, 16, t, n, seed=12)
    got, cache = run(c, 0.125, max_multi=4)
    R.check_extend(c, got, R.extend_ref(c, 0.125), 0.125)
    cache.check()
    out = torch.full_like(c["q"], 3.0).to(DEV)
    got, cache = run(c, 0.125, max_multi=2, out=out)
    cache.advance(c["q_start"].to(DEV))
    with pytest.raises(RuntimeError, match="q_start"):
        cache.check()
    few = dict(c, n=[30, 1, 20, 0, 1, 0])
    kept = [i for b in (0, 1, 2, 4) for i in range(int(c["q_start"][b]), int(c["q_start"][b + 1]))]
    R.check_extend(few, got, R.extend_ref(few, 0.125), 0.125, tokens=kept)
    assert (got["o"][[i for i in range(sum(n)) if i not in kept]] == 3).all()
    assert cache.seq_len.tolist() == [70, 6, 120, 0, 65, 33]


def test_many_short_fp32_prompts(cuda_lib):
    """1300 slots of up to 3 new tokens and 128 heads: several rounds of the fp32 kernels."""
    t = [(7 * b) % 37 if b % 29 else -1 for b in range(1300)]
    n = [0 if x < 0 else b % 4 for b, x in enumerate(t)]
    c = R.make_case("fp32", 128, 128, 8, 16, t, n, seed=13)
    got, cache = run(c, 0.1)
    R.check_extend(c, got, R.extend_ref(c, 0.1), 0.1)
    cache.check()


def test_stated_number_of_fp32_prompts(cuda_lib):
    t, n = [40, 5, 100, 0, 64], [30, 1, 20, 17, 1]
    c = R.make_case("fp32", 64, 4, 2, 16, t, n, seed=14)
    out = torch.full_like(c["q"], 3.0).to(DEV)
    got, cache = run(c, 0.125, max_multi=2, out=out)
    cache.advance(c["q_start"].to(DEV))
    with pytest.raises(RuntimeError, match="q_start"):
        cache.check()
    few = dict(c, n=[30, 1, 20, 0, 1])
    kept = [i for b in (0, 1, 2, 4) for i in range(int(c["q_start"][b]), int(c["q_start"][b + 1]))]
    R.check_extend(few, got, R.extend_ref(few, 0.125), 0.125, tokens=kept)
    assert cache.seq_len.tolist() == [70, 6, 120, 0, 65]
