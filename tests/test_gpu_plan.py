"""A step's plan (PagedCache.plan) against a plain model on the CPU, and whole steps of speculative serving: plan, attention
over forks and over the states of linear attention, verification, the accepted tokens taken in."""
import pytest
import torch

from test_gpu_pages import Model

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make_cache(slots, page=16, pages=400, width=40, **kw):
    from softmax_attention_chunk_gb300.paged import PagedCache

    return PagedCache(slots=slots, heads=1, head_dim=64, page_size=page, k_pages=pages, table_width=width, **kw)


def expect(model, n, tokens, from_start):
    """The maps, from the model's tables after its reserve."""
    rows = []
    start = [0]
    for b, m in enumerate(n):
        m = max(m, 0)
        for i in range(m):
            pos = int(model.seq_len[b]) + i
            row = lambda t: int(t[b, pos // model.P]) * model.P + pos % model.P  # noqa: E731
            rows.append((b, pos, row(model.k_table), row(model.v_table), None if from_start is None else from_start[b] + i))
        start.append(start[-1] + m)
    blank = (-1, -1, -1, -1, None if from_start is None else -1)
    cols = list(zip(*(rows + [blank] * (tokens - len(rows))))) if tokens else [()] * 5
    return start, cols


def compare(plan, want):
    start, cols = want
    assert plan.q_start.tolist() == start
    for name, col in zip(("slot", "position", "k_row", "v_row"), cols):
        assert getattr(plan, name).tolist() == list(col), name
    assert (plan.source is None) if not cols[4] or cols[4][0] is None else plan.source.tolist() == list(cols[4])


@pytest.mark.parametrize("page,slots,steps", [(16, 1, [[1], [15], [1], [40], [0]]),
                                              (16, 5, [[3, 0, 17, 1, 0], [1, 1, 1, 1, 1], [-2, 40, 16, 0, 300], [0, 0, 0, 0, 0]]),
                                              (256, 3, [[256, 1, 255], [1, 255, 2]]), (32, 300, [[i % 3 for i in range(300)], [1] * 300])])
@pytest.mark.parametrize("slack,source", [(0, False), (7, True)])
def test_steps(cuda_lib, page, slots, steps, slack, source):
    cache = make_cache(slots, page=page, pages=1000)
    model = Model(cache)
    for n in steps:
        tokens = sum(max(x, 0) for x in n) + slack
        old = [sum(max(x, 0) + 2 for x in n[:b]) for b in range(slots + 1)] if source else None
        plan = cache.plan(i32(n), tokens, from_start=i32(old) if source else None)
        model.reserve(n)
        compare(plan, expect(model, n, tokens, old))
        for name in ("k_table", "v_table", "seq_len", "k_ref", "v_ref"):
            assert torch.equal(getattr(cache, name).cpu(), getattr(model, name)), name
        cache.advance(plan.q_start)
        model.seq_len += torch.tensor([max(x, 0) if model.seq_len[b] >= 0 else 0 for b, x in enumerate(n)], dtype=torch.int32)
        cache.check()
        assert torch.equal(cache.seq_len.cpu(), model.seq_len)


def test_one_token_for_every_slot_in_use(cuda_lib):
    cache = make_cache(4)
    cache.plan(i32([5, 0, 16, 1]), 22)
    cache.advance(i32([0, 5, 5, 21, 22]))
    plan = cache.plan(None, 3)
    cache.check()
    assert plan.q_start.tolist() == [0, 1, 1, 2, 3] and plan.slot.tolist() == [0, 2, 3] and plan.position.tolist() == [5, 16, 1]


def test_refused_plans_are_empty_and_change_nothing(cuda_lib):
    def state(c):
        return [t.clone() for t in (c.k_table, c.v_table, c.seq_len, c.k_ref, c.v_ref)]

    for kw, n, tokens, why in ((dict(), [5, 6, 0], 10, "q_start"), (dict(pages=3), [40, 16, 0], 100, "free pages"), (dict(width=2), [3, 33, 0], 100, "outgrow"),
                               (dict(), [2 ** 31 - 1, 2 ** 31 - 1, 2], 64, None), (dict(), [1, 0, 0], 0, "q_start")):
        cache = make_cache(3, **kw)
        cache.plan(i32([0, 2, 0]), 2)
        cache.advance(i32([0, 0, 2, 2]))
        cache.check()
        before = state(cache)
        plan = cache.plan(i32(n), tokens, from_start=i32([0, 0, 0, 0]))
        with pytest.raises(RuntimeError, match=why):
            cache.check()
        assert all(torch.equal(a, b) for a, b in zip(before, state(cache)))
        assert plan.q_start.tolist() == [0] * 4
        assert all((getattr(plan, f) == -1).all() for f in ("slot", "position", "k_row", "v_row", "source"))


def test_more_slots_than_shared_memory_holds_starts_of(cuda_lib):
    slots = 5000
    n = [(i * 13) % 3 for i in range(slots)]
    cache = make_cache(slots, pages=slots, width=2)
    plan = cache.plan(i32(n), sum(n) + 1)
    cache.check()
    slot = [b for b, m in enumerate(n) for _ in range(m)]
    assert plan.slot.tolist() == slot + [-1]
    assert plan.position.tolist()[:-1] == [i for m in n for i in range(m)]


def test_captured_plan(cuda_lib):
    cache, twin = make_cache(3), make_cache(3)
    n = i32([1, 2, 3])
    cache.plan(n, 12)
    cache.free(i32([0, 1, 2]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = cache.plan(n, 12)
        cache.advance(plan.q_start)
    for step in ([1, 2, 3], [0, 12, 0], [4, 4, 4], [30, 0, 0], [5, 0, 1]):
        n.copy_(i32(step))
        graph.replay()
        want = twin.plan(i32(step), 12)
        twin.advance(want.q_start)
        assert all(torch.equal(a, b) for a, b in zip(plan[:5], want[:5]))
        assert torch.equal(cache.k_table, twin.k_table) and torch.equal(cache.seq_len, twin.seq_len)


def test_refusals(cuda_lib):
    cache = make_cache(3)
    for args in ((i32([1, 2]), 9), (torch.ones(3, device=DEV), 9), (i32([1, 1, 1]), -1), (i32([1, 1, 1]), (1 << 22) + 1), (i32([1, 1, 1]).cpu(), 9),
                 (i32([1, 1, 1]), 9, i32([0, 1, 2]))):
        with pytest.raises(ValueError):
            cache.plan(*args)


def test_speculative_serving(cuda_lib):
    """Three sequences of a model with one PaTH layer and one linear layer: steps with drafts that are partly rejected leave
    the caches, and give the accepted tokens the outputs, of sequences that were given the accepted tokens alone."""
    from softmax_attention_chunk_gb300.linear import LinearCache
    from softmax_attention_chunk_gb300.paged import PagedCache

    g = torch.Generator(device=DEV).manual_seed(11)
    B, H, d, V = 3, 2, 64, 500
    kw = dict(heads=H, head_dim=d, page_size=16, k_pages=80, table_width=20)
    paged, alone = PagedCache(slots=2 * B, **kw), PagedCache(slots=2 * B, **kw)
    linear, linear_alone = LinearCache(2 * B, H, d), LinearCache(2 * B, H, d)
    ld = torch.tensor([-0.1, -0.01], device=DEV)
    emb = {n: torch.randn(V, H, d, generator=g, device=DEV).bfloat16() for n in ("q", "k", "v", "w")}
    emb["w"] = (emb["w"].float() / emb["w"].float().norm(dim=-1, keepdim=True)).bfloat16()
    beta_of = 2 * torch.rand(V, H, generator=g, device=DEV)
    head = torch.randn(2 * H * d, V, generator=g, device=DEV) * 0.3

    def layer(cache, lin, tok, start, n, update):
        x = {name: t[tok.long()].contiguous() for name, t in emb.items()}
        a = cache.extend(x["q"], x["k"], x["v"], x["w"], beta_of[tok.long()], q_start=start, max_new=n, scale=0.125)
        b = lin.extend(x["q"], x["k"], x["v"], ld, q_start=start, max_new=n, scale=0.125, update=update)
        return a, b

    prompt = [37, 5, 20]
    tok = torch.randint(0, V, (sum(prompt),), generator=g, device=DEV).int()
    n = i32(prompt + [0] * B)
    for c, lin in ((paged, linear), (alone, linear_alone)):
        plan = c.plan(n, sum(prompt))
        layer(c, lin, tok, plan.q_start, 37, True)
        c.advance(plan.q_start)
    last = torch.randint(0, V, (B,), generator=g, device=DEV).int()
    parents, children = i32([0, 1, 2]), i32([3, 4, 5])
    D = 5  # tokens of a step: the known one and four drafts
    kept = 0
    for step in range(6):
        # drafts, checked on a fork; the linear layer's states stay
        draft_probs = torch.softmax(0.3 * torch.randn(B * D, V, generator=g, device=DEV), -1)
        drafts = torch.multinomial(draft_probs, 1, generator=g)[:, 0].int().view(B, D)
        drafts[:, 0] = last
        tok = drafts.reshape(-1).contiguous()
        paged.fork(parents, children)
        plan = paged.plan(i32([0] * B + [D] * B), B * D)
        before = linear.state.clone()
        linear.fork(parents, children)
        a, b = layer(paged, linear, tok, plan.q_start, D, False)
        assert torch.equal(linear.state[:B], before[:B])
        target = torch.softmax(torch.cat([a, b], -1).reshape(B * D, -1).float() @ head * 0.02, -1)
        uniform = torch.rand(B * D, generator=g, device=DEV)
        keep, after = paged.verify(target, tok, uniform, draft=draft_probs, q_start=plan.q_start, max_new=D)
        # the children's counts are the parents' new tokens
        paged.free(children)
        n_new = torch.cat([keep[B:], torch.zeros_like(keep[:B])])
        from_start = torch.cat([plan.q_start[B:], plan.q_start[-1:].expand(B)])
        taken = paged.plan(n_new, B * D, from_start=from_start)
        rows = taken.source.clamp(min=0).long()
        layer(paged, linear, tok[rows], taken.q_start, D, True)
        paged.advance(taken.q_start)
        paged.check(), linear.check()
        # the same sequences with the accepted tokens alone
        ks = keep[B:].tolist()
        assert keep[:B].tolist() == [0] * B and all(1 <= k <= D for k in ks)
        kept += sum(ks) - B
        only = torch.cat([drafts[i, :k] for i, k in enumerate(ks)])
        p2 = alone.plan(i32(ks + [0] * B), len(only))
        a2, b2 = layer(alone, linear_alone, only, p2.q_start, D, True)
        alone.advance(p2.q_start)
        assert torch.equal(tok[taken.source[: len(only)].long()], only)
        assert torch.equal(alone.seq_len[:B], paged.seq_len[:B])
        for i, k in enumerate(ks):
            at = sum(ks[:i])
            for got, want in ((a, a2), (b, b2)):  # (drafts behind a token change nothing before it)
                x, y = got[i * D : i * D + k].double(), want[at : at + k].double()
                assert float((x - y).norm()) <= 2.0 ** -7 * float(y.norm())
        assert float((linear.state[:B] - linear_alone.state[:B]).norm()) <= 2e-5 * float(linear_alone.state[:B].norm())
        last = after[B:].clone()
        assert bool(((last >= 0) & (last < V)).all())
    assert 0 < kept < 6 * B * (D - 1), "some drafts are kept, some are not"
