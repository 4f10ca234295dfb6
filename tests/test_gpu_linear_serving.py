"""Linear attention over a cache of states (LinearCache): prompts, drafts and single tokens against the definition in 64 bits."""
import math

import pytest
import torch

from linear_ref import DT, U, check, final_state, walk

pytestmark = pytest.mark.gpu
DEV = "cuda"


def starts(n):
    return torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32, device=DEV)


def make(dtype, d, hq, hkv, n, seed=0, extra=0):
    from softmax_attention_chunk_gb300.linear import LinearCache

    g = torch.Generator(device=DEV).manual_seed(200 + seed)
    N = sum(n) + extra
    r = lambda h: torch.randn(N, h, d, generator=g, device=DEV).to(DT[dtype])  # noqa: E731
    state = 3.0 * torch.randn(len(n), hkv, d, d, generator=g, device=DEV)
    ld = torch.tensor([[-0.3, -0.01, 0.0, -math.inf, -2.0][i % 5] for i in range(hkv)], device=DEV)
    return LinearCache.from_tensors(state, dtype=DT[dtype]), r(hq), r(hkv), r(hkv), ld


def expect(state, q, k, v, ld, n, scale):
    """Per slot with tokens: (slot, rows, (o, A), (state, its A))."""
    H = k.shape[1]
    at = 0
    for b, m in enumerate(n):
        if m:
            s = slice(at, at + m)
            heads = lambda t: t[s].permute(1, 0, 2)  # noqa: E731
            kh, vh = heads(k), heads(v)
            qh = heads(q).reshape(H, -1, m, q.shape[-1])
            o, A = walk(qh, kh[:, None].expand_as(qh), vh[:, None].expand_as(qh), ld[:, None].expand(qh.shape[:2]), scale, state=state[b][:, None])
            back = lambda t: t.reshape(-1, m, q.shape[-1]).permute(1, 0, 2)  # noqa: E731
            yield b, s, (back(o), back(A)), final_state(kh, vh, ld, state[b])
        at += m


def check_state(got, want, A, dtype, terms):
    bound = (U["bf16"] ** 2 if dtype == "bf16" else 0) * A + terms * 2.0 ** -24 * A + 1e-30
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


CASES = [[1], [1, 1, 1], [0, 3, 1, 0, 16], [17], [2, 130, 0, 1, 64, 15], [1, 1, 700, 1], [128, 129, 127], [5, 0, 2600, 31]]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("d,hq,hkv", [(64, 2, 2), (64, 6, 2), (128, 5, 5), (128, 16, 1)])
@pytest.mark.parametrize("n", CASES)
def test_new_tokens(cuda_lib, dtype, d, hq, hkv, n):
    cache, q, k, v, ld = make(dtype, d, hq, hkv, n, extra=3)
    before = cache.state.clone()
    out = torch.full_like(q, 7.0)
    o = cache.extend(q, k, v, ld, q_start=starts(n), max_new=max(n), scale=0.2, out=out, update=False)
    assert o is out and torch.equal(cache.state, before)
    kept = o.clone()
    o = cache.extend(q, k, v, ld, q_start=starts(n), max_new=max(n), scale=0.2, out=out)
    cache.check()
    assert torch.equal(o, kept)
    assert bool((o[sum(n):] == 7.0).all()), "rows behind the last token"
    seen = set()
    for b, rows, (want, A), (state, SA) in expect(before, q, k, v, ld, n, 0.2):
        check("o", o[rows], want, A, dtype, terms=n[b] + 2 * d + 64)
        check_state(cache.state[b], state, SA, dtype, terms=n[b] + 64)
        seen.add(b)
    for b in set(range(len(n))) - seen:
        assert torch.equal(cache.state[b], before[b])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_prompt_in_parts_and_token_by_token(cuda_lib, dtype):
    """One prompt, in chunks and as single tokens: the same states."""
    n = [300, 1]
    cache, q, k, v, ld = make(dtype, 64, 2, 2, n, seed=1)
    from softmax_attention_chunk_gb300.linear import LinearCache

    other = LinearCache.from_tensors(cache.state.clone(), dtype=DT[dtype])
    whole = cache.extend(q, k, v, ld, q_start=starts(n), max_new=300)
    at = 0
    for m in (37, 1, 16, 100, 146):
        part = other.extend(q[at : at + m], k[at : at + m], v[at : at + m], ld, q_start=starts([m, 0]))
        tol = 2 * U[dtype] if dtype == "bf16" else 2e-5
        assert float((part.double() - whole[at : at + m].double()).norm()) <= tol * float(whole[at : at + m].double().norm())
        at += m
    assert float((other.state[0] - cache.state[0]).norm()) <= 2e-5 * float(cache.state[0].norm())


def test_one_token_per_slot_without_starts(cuda_lib):
    cache, q, k, v, ld = make("bf16", 128, 4, 2, [1] * 37, seed=2)
    before = cache.state.clone()
    o = cache.extend(q, k, v, ld, scale=0.5)
    for b, rows, (want, A), (state, SA) in expect(before, q, k, v, ld, [1] * 37, 0.5):
        check("o", o[rows], want, A, "bf16", terms=400)
        check_state(cache.state[b], state, SA, "fp32", terms=8)


def test_bad_rows_of_q_start_are_left_out_and_reported(cuda_lib):
    n = [3, 40, 2]
    for bad in ([0, 3, 2, 45], [0, 3, 43, 99], [-1, 3, 43, 45], [0, 3, 44, 45]):
        cache, q, k, v, ld = make("bf16", 64, 2, 2, n, seed=3)
        before = cache.state.clone()
        s = torch.tensor(bad, dtype=torch.int32, device=DEV)
        cache.extend(q, k, v, ld, q_start=s, max_new=40)
        with pytest.raises(RuntimeError, match="q_start"):
            cache.check()
        cache.check()
        for b in range(3):
            m = bad[b + 1] - bad[b]
            if bad[b] < 0 or m < 0 or m > 40 or bad[b + 1] > 45:
                assert torch.equal(cache.state[b], before[b]), (bad, b)


def test_fork_and_reset(cuda_lib):
    from softmax_attention_chunk_gb300.linear import LinearCache

    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    state = torch.randn(6, 3, 64, 64, device=DEV)
    cache = LinearCache.from_tensors(state.clone())
    cache.fork(i32([0, 0, 2]), i32([1, 5, 3]))
    cache.check()
    want = state.clone()
    want[1], want[5], want[3] = state[0], state[0], state[2]
    assert torch.equal(cache.state, want)
    cache.reset(i32([4, 0]))
    cache.check()
    want[4] = want[0] = 0
    assert torch.equal(cache.state, want)
    # no slot, listed twice, a child that is a parent too: left out, the others are not
    for parents, children, done in (([1, 2], [6, 0], [1]), ([1, 2, 3], [0, 0, 4], [2]), ([1, 2, 3], [2, 4, 0], [2]), ([-1, 3], [0, 4], [1])):
        before = cache.state.clone()
        cache.fork(i32(parents), i32(children))
        with pytest.raises(RuntimeError, match="slot"):
            cache.check()
        for j in done:
            before[children[j]] = before[parents[j]]
        assert torch.equal(cache.state, before), (parents, children)
    with pytest.raises(RuntimeError, match="slot"):
        cache.reset(i32([7]))
        cache.check()


def test_nan_stays_in_its_slot(cuda_lib):
    n = [2, 200, 1, 90]
    cache, q, k, v, ld = make("bf16", 64, 4, 2, n, seed=4)
    from softmax_attention_chunk_gb300.linear import LinearCache

    other = LinearCache.from_tensors(cache.state.clone())
    want = cache.extend(q, k, v, ld, q_start=starts(n), max_new=200)
    k2 = k.clone()
    k2[20:30] = math.nan
    other.state[2] = math.inf
    got = other.extend(q, k2, v, ld, q_start=starts(n), max_new=200)
    for b, rows in ((0, slice(0, 2)), (3, slice(203, 293))):
        assert torch.equal(got[rows], want[rows]) and torch.equal(other.state[b], cache.state[b])
    assert bool(got[30:202].isnan().any())


def test_captured_step_replays_with_new_lengths(cuda_lib):
    n = [[1, 60, 0, 5], [200, 1, 17, 16], [0, 0, 0, 234]]
    N = 234
    cache, q, k, v, ld = make("bf16", 64, 4, 2, [N, 0, 0, 0], seed=5)
    from softmax_attention_chunk_gb300.linear import LinearCache

    other = LinearCache.from_tensors(cache.state.clone())
    s = starts(n[0])
    cache.extend(q, k, v, ld, q_start=s, max_new=N, update=False)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        o = cache.extend(q, k, v, ld, q_start=s, max_new=N)
    for m in n:
        s.copy_(starts(m))
        graph.replay()
        want = other.extend(q, k, v, ld, q_start=starts(m), max_new=N)
        assert torch.equal(o[: sum(m)], want[: sum(m)]) and torch.equal(cache.state, other.state)
    cache.check()


def test_two_caches_at_once(cuda_lib):
    n = [900, 1, 40]
    made = [make("bf16", 128, 4, 2, n, seed=6 + i) for i in range(2)]
    from softmax_attention_chunk_gb300.linear import LinearCache

    want = []
    for c, q, k, v, ld in made:
        twin = LinearCache.from_tensors(c.state.clone())
        want.append((twin.extend(q, k, v, ld, q_start=starts(n), max_new=900), twin.state))
    s = starts(n)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for (c, q, k, v, ld), st in zip(made, streams):
        with torch.cuda.stream(st):
            got.append(c.extend(q, k, v, ld, q_start=s, max_new=900))
    torch.cuda.synchronize()
    for g, (c, *_), (wo, ws) in zip(got, made, want):
        assert torch.equal(g, wo) and torch.equal(c.state, ws)


def test_many_slots(cuda_lib):
    n = [(i * 7) % 23 for i in range(1500)]
    cache, q, k, v, ld = make("bf16", 64, 1, 1, n, seed=8)
    before = cache.state.clone()
    o = cache.extend(q, k, v, ld, q_start=starts(n), max_new=22)
    cache.check()
    for b, rows, (want, A), (state, SA) in list(expect(before, q, k, v, ld, n, 1.0))[::97]:
        check("o", o[rows], want, A, "bf16", terms=n[b] + 200)
        check_state(cache.state[b], state, SA, "bf16", terms=n[b] + 64)


@pytest.mark.parametrize("d,hq,hkv,n", [(64, 2, 2, [3000]), (128, 4, 1, [700, 1, 30])])
def test_many_calls_in_a_row(cuda_lib, d, hq, hkv, n):
    """Thousands of calls behind one another: the kernels' warps meet in every order, and no bounded wait gives up."""
    cache, q, k, v, ld = make("bf16", d, hq, hkv, n, seed=9)
    s = starts(n)
    want = cache.extend(q, k, v, ld, q_start=s, max_new=max(n), update=False).clone()
    out = torch.empty_like(q)
    for _ in range(3000):
        cache.extend(q, k, v, ld, q_start=s, max_new=max(n), update=False, out=out)
    cache.check()
    assert torch.equal(out, want)
