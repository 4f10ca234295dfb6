"""Slots that a call of the paged attention leaves out: nothing of theirs changes, their lengths do not grow, and the
next call goes on from there as the definition says."""
import pytest
import torch

import paged_ref as R
from test_gpu_paged import DEV, run, to_cache

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def now(c, cache, t, n, seed):
    """The case of a next call on the cache as it stands: t cached tokens, n new ones per slot."""
    new = R.make_case(c["dtype"], c["d"], c["hq"], c["hkv"], c["page"], [-1] * len(n), n, c["fox"], seed=seed)
    for x in ("k_pool", "v_pool", "k_table", "v_table", "seq_len"):
        new[x] = getattr(cache, x).cpu()
    if c["fox"]:
        new["a_pool"] = cache.a_pool.cpu()
    return dict(new, t=list(t))


# the streaming pass, drafts, prompt chunks beside one token and beside several, and the fp32 kernels
@pytest.mark.parametrize("dtype,d,n", [("bf16", 64, [1, 1]), ("bf16", 128, [5, 2]), ("bf16", 64, [40, 1]), ("bf16", 128, [300, 20]),
                                       ("fp32", 64, [1, 1]), ("fp32", 128, [5, 1]), ("fp32", 64, [40, 20])])
@pytest.mark.parametrize("fox", [False, True])
def test_a_refused_reserve_leaves_no_hole(cuda_lib, dtype, d, n, fox):
    """Slot 0 needs a page that the pool has not.  The call that follows leaves it out whole (its cached keys too), advance
    does not count its tokens, and once there are pages it goes on with nothing lost."""
    t = [32, 25, 300]
    c = R.make_case(dtype, d, 4, 2, 32, t, n + [0], fox, seed=sum(n) + d)
    free_k, free_v = c["k_table"][0, 1:].clone(), c["v_table"][0, 1:].clone()
    c["k_table"][0, 1:] = -1
    c["v_table"][0, 1:] = -1
    cache = to_cache(c)
    cache.k_ref.fill_(1)  # nothing is free
    cache.v_ref.fill_(1)
    cache.reserve(i32(n + [0]))
    out = torch.full_like(c["q"], 3.0).to(DEV)
    got, _ = run(c, 0.125, cache=cache, out=out)
    cache.advance(c["q_start"].to(DEV))
    with pytest.raises(RuntimeError, match="not enough free pages"):
        cache.check()
    assert cache.seq_len.tolist() == [32, 25 + n[1], 300]
    assert (got["o"][: n[0]] == 3).all()
    alone = dict(c, n=[0, n[1], 0])
    R.check_extend(alone, got, R.extend_ref(alone, 0.125), 0.125, tokens=torch.arange(n[0], n[0] + n[1]))
    cache.k_ref[free_k[free_k >= 0].long().to(DEV)] = 0
    cache.v_ref[free_v[free_v >= 0].long().to(DEV)] = 0
    cache.reserve(i32([n[0], 0, 0]))
    c = now(c, cache, [32, 25 + n[1], 300], [n[0], 0, 0], seed=7)
    got, _ = run(c, 0.125, cache=cache)
    cache.advance(c["q_start"].to(DEV))
    R.check_extend(c, got, R.extend_ref(c, 0.125), 0.125)
    cache.check()
    assert cache.seq_len.tolist() == [32 + n[0], 25 + n[1], 300]


@pytest.mark.parametrize("dtype,n,max_new", [("bf16", [3, 1, 2], 2), ("bf16", [30, 1, 20], 20), ("bf16", [3, 1, 1], 1),
                                             ("fp32", [9, 1, 4], 4)])
def test_more_tokens_than_max_new_are_not_counted(cuda_lib, dtype, n, max_new):
    c = R.make_case(dtype, 64, 4, 2, 16, [40, 90, 16], n, seed=sum(n))
    out = torch.full_like(c["q"], 3.0).to(DEV)
    got, cache = run(c, 0.125, max_new=max_new, out=out)
    cache.advance(c["q_start"].to(DEV))
    with pytest.raises(RuntimeError, match="q_start"):
        cache.check()
    assert cache.seq_len.tolist() == [40, 90 + n[1], 16 + n[2]]
    assert (got["o"][: n[0]] == 3).all()
    rest = dict(c, n=[0] + n[1:])
    R.check_extend(rest, got, R.extend_ref(rest, 0.125), 0.125, tokens=torch.arange(n[0], sum(n)))
    c = now(c, cache, cache.seq_len.tolist(), [1, 1, 1], seed=3)  # (each last page has room)
    got, _ = run(c, 0.125, cache=cache)
    cache.advance(c["q_start"].to(DEV))
    R.check_extend(c, got, R.extend_ref(c, 0.125), 0.125)
    cache.check()
    assert cache.seq_len.tolist() == [41, 91 + n[1], 17 + n[2]]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_overlapping_ranges_are_not_counted(cuda_lib, dtype):
    c = R.make_case(dtype, 64, 4, 2, 16, [40] * 5, [30] * 5, seed=61, width_slack=30)
    s = torch.tensor([0, 150, 0, 150, 0, 1], dtype=torch.int32)  # the last slot has one token
    need = torch.arange(5 * 15).view(5, 15).int()
    c.update(k_table=need, v_table=need.clone(), k_pool=torch.randn(75, 2, 16, 64).to(R.DT[dtype]),
             v_pool=torch.randn(75, 2, 16, 64).to(R.DT[dtype]), k_ref=torch.ones(75).int(), v_ref=torch.ones(75).int())
    _, cache = run(dict(c, q_start=s), 0.125, max_new=150)
    cache.advance(s.to(DEV))
    with pytest.raises(RuntimeError, match="q_start"):
        cache.check()
    assert cache.seq_len.tolist() == [40, 40, 40, 40, 41]


@pytest.mark.parametrize("dtype,n", [("bf16", 5), ("bf16", 30), ("fp32", 5)])
def test_advance_by_part_of_a_call_is_refused(cuda_lib, dtype, n):
    """The cached keys have passed all tokens of the call: fewer (rejected draft tokens) cannot be counted."""
    c = R.make_case(dtype, 64, 4, 2, 16, [40, 90], [n, n], seed=n)
    _, cache = run(c, 0.125)
    cache.advance(i32([0, n - 2, 2 * n - 2]))
    with pytest.raises(RuntimeError, match="q_start"):
        cache.check()
    assert cache.seq_len.tolist() == [40, 90 + n]
    cache.advance(i32([0, n, n]))
    cache.check()
    assert cache.seq_len.tolist() == [40 + n, 90 + n]
    cache.advance(i32([0, 0, 0]))
    cache.check()
    assert cache.seq_len.tolist() == [40 + n, 90 + n]


def test_two_calls_and_their_advances(cuda_lib):
    """Calls on different slots may be followed by their advances in any order; a slot that is freed forgets what a
    call gave it."""
    c = R.make_case("bf16", 64, 4, 2, 16, [40, 90], [3, 1], seed=5)
    cache = to_cache(c)
    a, b = i32([0, 3, 3]), i32([3, 3, 4])
    for s in (a, b):
        run(dict(c, q_start=s.cpu()), 0.125, cache=cache, max_new=3)
    cache.advance(b)
    assert cache.seq_len.tolist() == [40, 91]
    cache.advance(a)
    assert cache.seq_len.tolist() == [43, 91]
    run(dict(c, q_start=a.cpu()), 0.125, cache=cache, max_new=3)
    cache.free(i32([0]))
    cache.reserve(i32([7, 0]))
    cache.advance(i32([0, 7, 7]))
    assert cache.seq_len.tolist() == [7, 91]
    cache.check()


@pytest.mark.parametrize("fox", [False, True])
def test_advance_needs_the_pages_of_its_rows(cuda_lib, fox):
    """Rows that the caller wrote itself: advance stops a length at a page that is not there."""
    c = R.make_case("bf16", 64, 4, 2, 16, [16, 20], [16, 12], fox, seed=1, width_slack=3)
    cache = to_cache(c)
    cache.advance(i32([0, 17, 29]))
    with pytest.raises(RuntimeError, match="page-table"):
        cache.check()
    assert cache.seq_len.tolist() == [16, 32]
    cache.advance(i32([0, 16, 16]))
    cache.check()
    assert cache.seq_len.tolist() == [32, 32]


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
def test_drafts_are_checked_on_a_fork(cuda_lib, dtype, d):
    """5 draft tokens checked on a fork of their sequence; 3 are accepted, so the fork goes and the sequence takes the 3."""
    c = R.make_case(dtype, d, 4, 2, 16, [45, -1], [5, 0], seed=d, slack=20, width_slack=3)
    cache = to_cache(c)
    cache.fork(i32([0]), i32([1]))
    cache.reserve(i32([0, 5]))
    got, _ = run(dict(c, q_start=torch.tensor([0, 0, 5], dtype=torch.int32)), 0.125, cache=cache)
    cache.advance(i32([0, 0, 5]))
    cache.check()
    ref = R.extend_ref(c, 0.125)
    R.check_extend(c, dict(got, k=ref[2].to(R.DT[dtype]), v=ref[3].to(R.DT[dtype])), ref, 0.125)  # o only
    cache.free(i32([1]))
    part = dict(c, n=[3, 0], q_start=torch.tensor([0, 3, 3], dtype=torch.int32), k_pool=cache.k_pool.cpu(),
                v_pool=cache.v_pool.cpu(), **{x: c[x][:3] for x in ("q", "k", "v", "w", "beta")})
    got, _ = run(part, 0.125, cache=cache)
    cache.advance(i32([0, 3, 3]))
    cache.check()
    R.check_extend(part, got, R.extend_ref(part, 0.125), 0.125)
    assert cache.seq_len.tolist() == [48, -1]


def test_captured_steps_run_on_past_a_full_pool(cuda_lib):
    """reserve, extend and advance as one captured step, replayed without a look at the status while the pool runs full:
    sequences stand still at a page that is not there and go on when one is freed, with every counted token in place."""
    from softmax_attention_chunk_gb300.paged import PagedCache

    P, pages = 16, 7
    cache = PagedCache(3, 2, 64, P, pages, table_width=12)
    g = torch.Generator(device=DEV).manual_seed(2)
    bf = lambda *s: torch.randn(*s, device=DEV, generator=g).to(torch.bfloat16)  # noqa: E731
    q, k, v, w, beta = bf(3, 4, 64), bf(3, 2, 64), bf(3, 2, 64), bf(3, 2, 64), torch.zeros(3, 2, device=DEV)
    lens, own, free = [20, 28, 5], [2, 2, 1], pages - 5
    cache.reserve(i32(lens))
    cache.k_pool.copy_(bf(*cache.k_pool.shape))
    cache.v_pool.copy_(bf(*cache.v_pool.shape))
    cache.advance(i32([0, 20, 48, 53]))
    cache.check()
    first = [(cache.k_table[b].clone(), cache.v_table[b].clone()) for b in range(3)]
    k0, v0 = cache.k_pool.clone(), cache.v_pool.clone()
    out = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=DEV)

    def step():
        cache.reserve()
        cache.extend(q, k, v, w, beta, scale=0.125, out=out)
        cache.advance()

    step_graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(step_graph):
        step()
    live = [True] * 3
    start = list(lens)
    for i in range(60):
        if i == 40:  # one sequence ends
            cache.free(i32([2]))
            free += own[2]
            live[2] = False
        step_graph.replay()
        need = [b for b in range(3) if live[b] and lens[b] % P == 0 and own[b] * P == lens[b]]
        if len(need) <= free:
            free -= len(need)
            for b in need:
                own[b] += 1
        for b in range(3):
            if live[b] and lens[b] < own[b] * P:
                lens[b] += 1
    torch.cuda.synchronize()
    assert cache.seq_len.tolist() == [lens[0], lens[1], -1]
    assert any(x < s + 60 for x, s in zip(lens[:2], start))  # (some stood still)
    with pytest.raises(RuntimeError, match="not enough free pages"):
        cache.check()
    for b in range(2):
        pos = torch.arange(start[b], device=DEV)
        table = [x[b].cpu().long() for x in (cache.k_table, cache.v_table)]
        made = torch.arange(start[b], lens[b])
        for pool, new, t, (old, was) in ((cache.k_pool, k, table[0], (k0, first[b][0])), (cache.v_pool, v, table[1], (v0, first[b][1]))):
            x = pool.cpu()
            assert torch.equal(x[t[made // P], :, made % P], new[b].cpu().expand(len(made), 2, 64))
            assert torch.equal(x[t[pos.cpu() // P], :, pos.cpu() % P], old.cpu()[was.cpu().long()[pos.cpu() // P], :, pos.cpu() % P])


@pytest.mark.parametrize("n", [[1, 1, 1, 1], [6, 3, 2, 8], [90, 40, 200, 1]])
def test_two_calls_at_once_on_one_cache(cuda_lib, n):
    """Calls on different slots of a cache, on two streams and with a workspace each."""
    c = R.make_case("bf16", 64, 4, 2, 16, [3000, 64, 2000, 500], n, seed=sum(n))
    cache = to_cache(c)
    cut = int(c["q_start"][2])
    parts = []
    for sl, start in ((slice(0, cut), [0, n[0], cut, cut, cut]), (slice(cut, None), [0, 0, 0, n[2], n[2] + n[3]])):
        parts.append(([c[x][sl].clone().to(DEV) for x in ("q", "k", "v", "w", "beta")], i32(start)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for s, (x, start) in zip(streams, parts):
        with torch.cuda.stream(s):
            outs.append(cache.extend(*x, q_start=start, max_new=max(n), scale=0.125))
    torch.cuda.synchronize()
    got = dict(o=torch.cat([o.cpu() for o in outs]), k=cache.k_pool.cpu(), v=cache.v_pool.cpu())
    R.check_extend(c, got, R.extend_ref(c, 0.125), 0.125)
    for _, start in parts:
        cache.advance(start)
    cache.check()
    assert cache.seq_len.tolist() == [a + b for a, b in zip(c["t"], n)]
