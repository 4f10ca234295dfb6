"""LinearCache.extend with starts that fall: a slot whose row is bad, or begins before an earlier good row's tokens end, is left out
whole and reported; the others get what they get alone."""
import pytest
import torch

from linear_ref import check
from test_gpu_linear_serving import DEV, check_state, expect, make

pytestmark = pytest.mark.gpu


def taken(start, total, max_new):
    """Slots that are not left out, by the rule above."""
    out, end = [], 0
    for b, (lo, hi) in enumerate(zip(start, start[1:])):
        if lo < 0 or hi < lo or hi > total or hi - lo > max_new or hi == lo:
            continue
        if lo >= end:
            out.append(b)
        end = max(end, hi)
    return out


STARTS = [
    [0, 3000, 0, 3000],                            # twice all tokens, in several segments
    [0, 3000, 1000, 2000, 0, 2900],
    [0, 40, 0, 40, 0, 40, 0, 40],                  # one segment each
    [0, 5, 0, 5, 3, 8],                            # tokens and drafts
    [0, 20, 5, 45, 50, 60],                        # begins inside an earlier slot's tokens; the next ones are good
    [0, 1, 900, 1, 17, 950, 5, 1000, 1001, 1040],
    [0, 900000, 3, 9, 600],                        # an end that is none
    [100, 2900, 0, 90, 2900, 3000],                # before all others, but later
    [0] + [7] * 40 + [30, 600, 8, 20] + [25] * 30 + [500, 900, 901],  # over more slots than a warp has lanes
    [5 * i for i in range(300)] + [0, 17, 1495, 1500],                # than a block has threads
]


@pytest.mark.parametrize("dtype,d,hq,hkv", [("bf16", 64, 2, 2), ("bf16", 128, 4, 1), ("fp32", 64, 2, 1)])
@pytest.mark.parametrize("start", STARTS)
def test_slots_that_begin_before_an_earlier_one_ends(cuda_lib, dtype, d, hq, hkv, start):
    total, slots = 3000, len(start) - 1
    max_new = max([hi - lo for lo, hi in zip(start, start[1:]) if hi <= total] + [1])
    cache, q, k, v, ld = make(dtype, d, hq, hkv, [total] + [0] * (slots - 1), seed=20)
    before, out = cache.state.clone(), torch.full_like(q, 7.0)
    s = torch.tensor(start, dtype=torch.int32, device=DEV)
    for update in (False, True):
        cache.extend(q, k, v, ld, q_start=s, max_new=max_new, scale=0.2, out=out, update=update)
        with pytest.raises(RuntimeError, match="q_start"):
            cache.check()
        cache.check()
        assert update or torch.equal(cache.state, before)
    good, written = taken(start, total, max_new), torch.zeros(total, dtype=torch.bool)
    for b in range(slots):
        if b not in good:
            assert torch.equal(cache.state[b], before[b]), b
            continue
        rows = slice(start[b], start[b + 1])
        written[rows] = True
        n = start[b + 1] - start[b]
        for _, _, (want, A), (state, SA) in expect(before[b : b + 1], q[rows], k[rows], v[rows], ld, [n], 0.2):
            check("o", out[rows], want, A, dtype, terms=n + 2 * d + 64)
            check_state(cache.state[b], state, SA, dtype, terms=n + 64)
    assert bool((out[~written.to(DEV)] == 7.0).all()), "rows of no slot"


@pytest.mark.parametrize("slots", [257, 5000])
def test_many_slots_after_an_error_that_nobody_has_read(cuda_lib, slots):
    """More slots than a block has threads: a code that still stands makes blocks look closer, good rows stay good."""
    n = [1 + b % 3 for b in range(slots)]
    cache, q, k, v, ld = make("bf16", 64, 1, 1, n, seed=22)
    before = cache.state.clone()
    good = torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    want = cache.extend(q, k, v, ld, q_start=good, max_new=3).clone()
    cache.check()
    state = cache.state.clone()
    cache.state.copy_(before)
    bad = good.clone()
    bad[slots - 3] = 0  # the slot before it falls, the one after it begins in the first one's tokens and has too many
    bad[slots - 2] = 2  # now it has two, which are others' tokens
    cache.extend(q, k, v, ld, q_start=bad, max_new=3, update=False)
    got = cache.extend(q, k, v, ld, q_start=good, max_new=3)
    assert torch.equal(got, want) and torch.equal(cache.state, state)
    with pytest.raises(RuntimeError, match="q_start"):
        cache.check()
    cache.extend(q, k, v, ld, q_start=bad, max_new=3)
    with pytest.raises(RuntimeError, match="q_start"):
        cache.check()
    left_out = [b for b in range(slots) if b not in taken(bad.tolist(), len(q), 3)]
    assert left_out == [slots - 4, slots - 3, slots - 2]
    assert torch.equal(cache.state[left_out], state[left_out])
