"""Verification of drafted tokens (PagedCache.verify) against its definition on the CPU: products, differences and running
sums in 64 bits (numpy), a slot at a time.  Indices have to be equal: the uniform numbers' goals are then further from the
borders than the sums are off (2^-40), which the reference checks."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def make_cache(slots):
    from softmax_attention_chunk_gb300.paged import PagedCache

    return PagedCache(slots=slots, heads=1, head_dim=64, page_size=16, k_pages=slots)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def positive(x):
    x = x.double().cpu().numpy()
    return np.where(x > 0, x, 0.0)


def reference(target, draft, tokens, uniform, start):
    keep, after = [], []
    p, u, tok = positive(target), uniform.double().cpu().numpy(), tokens.tolist()
    V = p.shape[1]
    for b in range(len(start) - 1):
        lo, hi = start[b], start[b + 1]
        if hi <= lo:
            keep.append(0), after.append(-1)
            continue
        k = 1
        while lo + k < hi:
            i, x = lo + k, tok[lo + k]
            if not (0 <= x < V):
                break
            q = 1.0 if draft is None else positive(draft[i])[x]
            if not u[i] * q < p[i - 1][x]:
                break
            k += 1
        row = p[lo + k - 1]
        rest = row.copy()
        if lo + k < hi:
            if draft is not None:
                rest = np.maximum(row - positive(draft[lo + k]), 0.0)
            elif 0 <= tok[lo + k] < V:
                rest[tok[lo + k]] = 0.0
            if not rest.sum() > 0:
                rest = row
        keep.append(k)
        c = np.cumsum(rest)
        if not c[-1] > 0:
            after.append(-1)
            continue
        goal = u[lo] * c[-1]
        assert np.abs(c - goal)[rest > 0].min() > 2.0 ** -40 * c[-1] or u[lo] in (0.0, 0.25, 0.5), "a goal on a border says nothing"
        after.append(min(int((c <= goal).sum()), int(np.nonzero(rest)[0].max())))
    return keep, after


def case(dtype, V, n, seed, noise=0.7, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    N = sum(n)
    logits = 2.0 * torch.randn(N, V, generator=g, device=DEV)
    near = torch.roll(logits, 1, 0) + noise * torch.randn(N, V, generator=g, device=DEV)
    rows = lambda x: torch.nn.functional.pad(torch.softmax(x, -1).to(DT[dtype]), (0, pad), value=float("nan"))[:, :V]  # noqa: E731
    target, draft = rows(logits), rows(near)
    tokens = torch.multinomial(draft.float() + 1e-30, 1, generator=g)[:, 0].to(torch.int32)
    return target, draft, tokens, torch.rand(N, generator=g, device=DEV)


def starts(n):
    return [0] + torch.tensor(n).cumsum(0).tolist()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V,pad", [(1, 0), (2, 0), (7, 0), (33, 2), (64, 64), (511, 0), (513, 3), (4096, 0), (32000, 0), (50001, 0), (131072, 8), (262144, 0)])
@pytest.mark.parametrize("with_draft", [True, False])
def test_kept_and_next(cuda_lib, dtype, V, pad, with_draft):
    n = [1, 5, 0, 2, 40, 9]
    target, draft, tokens, uniform = case(dtype, V, n, seed=V + pad, pad=pad)
    s = starts(n)
    cache = make_cache(len(n))
    keep, after = cache.verify(target, tokens, uniform, draft=draft if with_draft else None, q_start=i32(s), max_new=40)
    cache.check()
    want = reference(target, draft if with_draft else None, tokens, uniform, s)
    assert (keep.tolist(), after.tolist()) == want


@pytest.mark.parametrize("slots", [1, 3, 64, 700])
def test_numbers_of_slots(cuda_lib, slots):
    n = [1 + (i * 5) % 4 for i in range(slots)]
    target, draft, tokens, uniform = case("fp32", 5000, n, seed=slots, noise=0.2)
    cache = make_cache(slots)
    keep, after = cache.verify(target, tokens, uniform, draft=draft, q_start=i32(starts(n)))
    assert (keep.tolist(), after.tolist()) == reference(target, draft, tokens, uniform, starts(n))
    assert slots < 64 or 1 < len(set(keep.tolist()))


def test_same_models_keep_every_draft(cuda_lib):
    """draft row i equal to target row i - 1: u < 1 keeps it, whatever it is."""
    n = [9, 17, 3]
    target, _, _, uniform = case("bf16", 1000, n, seed=1)
    draft = torch.roll(target, 1, 0)
    tokens = torch.multinomial(draft.float(), 1)[:, 0].to(torch.int32)
    cache = make_cache(3)
    keep, after = cache.verify(target, tokens, torch.full_like(uniform, 1 - 2.0 ** -24), draft=draft, q_start=i32(starts(n)))
    assert keep.tolist() == n
    last = [int(torch.nonzero(target[e - 1])[-1]) for e in starts(n)[1:]]
    assert all(0 <= a <= b for a, b in zip(after.tolist(), last))


def test_borders(cuda_lib):
    """Zero probabilities are neither kept nor drawn; u 0 draws the first positive entry; sums that fall on a border exactly
    pass at the next entry; a residual of nothing leaves the target; a row of nothing draws none."""
    V = 2048
    t = torch.zeros(12, V, device=DEV)
    q = torch.zeros(12, V, device=DEV)
    u = torch.zeros(12, device=DEV)
    t[0, 100], t[0, 900] = 0.5, 0.5          # slot 0: u = 0.5 falls on the border after 100
    u[0] = 0.5
    t[1, 5:9] = 0.25                         # slot 1: u = 0: entry 5
    t[2, 7] = 1.0                            # slot 2: a draft of probability 0 under the target, kept not
    q[3, 3] = 1.0
    t[4, 7], q[5, 7] = 0.5, 0.75             # slot 3: rejected, nothing is left of the target: its own row
    u[5] = 0.999
    # slot 4: a target of zeros
    t[7, 11], q[8, 11] = 1.0, 0.0            # slot 5: a draft that could not have been drawn, but the target would: kept
    t[8, V - 1] = 1e-30
    t[9, 3], t[9, 4] = 0.25, 0.75            # slot 6: u = 0.25: entry 4
    u[9] = 0.25
    tokens = torch.zeros(12, dtype=torch.int32, device=DEV)
    tokens[3], tokens[5], tokens[8] = 3, 7, 11
    s = [0, 1, 2, 4, 6, 7, 9, 10]
    cache = make_cache(7)
    keep, after = cache.verify(t, tokens, u, draft=q, q_start=i32(s))
    assert keep.tolist() == [1, 1, 1, 1, 1, 2, 1]
    assert after.tolist() == [900, 5, 7, 7, -1, V - 1, 4]
    assert (keep.tolist(), after.tolist()) == reference(t, q, tokens, u, s)
    cache.check()


def test_equal_probabilities(cuda_lib):
    """Sums of equal powers of two are exact: entry floor(u V)."""
    V = 32768
    u = torch.rand(32, device=DEV)
    cache = make_cache(32)
    keep, after = cache.verify(torch.full((32, V), 1.0 / V, device=DEV), torch.zeros(32, dtype=torch.int32, device=DEV), u, q_start=i32(list(range(33))))
    assert after.tolist() == (u.double() * V).long().tolist() and keep.tolist() == [1] * 32


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("power", [-100, -70, -62, 100])
@pytest.mark.parametrize("V", [1000, 1001, 32768])
def test_rows_of_tiny_and_huge_numbers(cuda_lib, dtype, power, V):
    """Probabilities need not add up to 1 (at 2^-100 some are denormal: the reference gets the same)."""
    n = [4, 1, 3, 6, 2, 5]
    target, draft, tokens, uniform = case(dtype, V, n, seed=V + power + 200)
    target, draft = target * 2.0 ** power, draft * 2.0 ** power
    keep, after = make_cache(len(n)).verify(target, tokens, uniform, draft=draft, q_start=i32(starts(n)))
    assert (keep.tolist(), after.tolist()) == reference(target, draft, tokens, uniform, starts(n))


def test_infinity_in_both_rows(cuda_lib):
    n = [3, 3, 1]
    target, draft, tokens, uniform = case("fp32", 6000, n, seed=5)
    want = reference(target, draft, tokens, uniform, starts(n))
    target[4, 9], draft[5, 9] = float("inf"), float("inf")
    keep, after = make_cache(3).verify(target, tokens, uniform, draft=draft, q_start=i32(starts(n)))
    assert [keep.tolist()[b] for b in (0, 2)] == [want[0][b] for b in (0, 2)] and [after.tolist()[b] for b in (0, 2)] == [want[1][b] for b in (0, 2)]
    assert 1 <= int(keep[1]) <= 3 and -1 <= int(after[1]) < 6000


def test_nan_and_infinity(cuda_lib):
    n = [3, 3, 1]
    target, draft, tokens, uniform = case("fp32", 6000, n, seed=5)
    target[:, 17], draft[:, 40] = float("nan"), float("nan")
    target[1, 50] = -1.0
    cache = make_cache(3)
    got = cache.verify(target, tokens, uniform, draft=draft, q_start=i32(starts(n)))
    assert (got[0].tolist(), got[1].tolist()) == reference(target, draft, tokens, uniform, starts(n))
    clean = got[1].tolist()
    target[6, 99] = float("inf")
    got = cache.verify(target, tokens, uniform, draft=draft, q_start=i32(starts(n)))
    assert got[1].tolist()[:2] == clean[:2] and -1 <= int(got[1][2]) < 6000
    for bad in (float("nan"), -1.0, 2.0, float("inf")):
        got = cache.verify(target, tokens, torch.full_like(uniform, bad), draft=draft, q_start=i32(starts(n)))
        assert all(-1 <= x < 6000 for x in got[1].tolist())


def test_bad_rows_and_tokens_are_reported(cuda_lib):
    n = [3, 4, 2]
    target, draft, tokens, uniform = case("bf16", 300, n, seed=6)
    cache = make_cache(3)
    good = cache.verify(target, tokens, uniform, draft=draft, q_start=i32(starts(n)))
    for bad in ([0, 3, 2, 9], [-1, 3, 7, 9], [0, 3, 7, 10]):
        keep, after = cache.verify(target, tokens, uniform, draft=draft, q_start=i32(bad))
        with pytest.raises(RuntimeError, match="q_start"):
            cache.check()
        for b in range(3):
            if bad[b] < 0 or bad[b + 1] < bad[b] or bad[b + 1] > 9:
                assert (int(keep[b]), int(after[b])) == (0, -1)
            elif bad[b : b + 2] == starts(n)[b : b + 2]:
                assert (int(keep[b]), int(after[b])) == (int(good[0][b]), int(good[1][b]))
    keep, after = cache.verify(target, tokens, uniform, draft=draft, q_start=i32(starts(n)), max_new=3)
    assert (int(keep[1]), int(after[1])) == (0, -1)
    with pytest.raises(RuntimeError, match="q_start"):
        cache.check()
    for x in (-1, 300, 2 ** 31 - 1):
        t = tokens.clone()
        t[4] = x
        for dr in (draft, None):
            keep, after = cache.verify(target, t, uniform, draft=dr, q_start=i32(starts(n)))
            with pytest.raises(RuntimeError, match="vocabulary"):
                cache.check()
            assert (keep.tolist(), after.tolist()) == reference(target, dr, t, uniform, starts(n))


def test_refusals(cuda_lib):
    target, draft, tokens, uniform = case("fp32", 100, [4], seed=7)
    cache = make_cache(1)
    s = i32([0, 4])
    for kw in (dict(target=target.half()), dict(target=target[0]), dict(target=target.t().contiguous().t()), dict(target=target.cpu()),
               dict(draft=draft[:3]), dict(draft=draft.bfloat16()), dict(tokens=tokens.long()), dict(tokens=tokens[:3]),
               dict(uniform=uniform.double()), dict(uniform=uniform[:2]), dict(q_start=None), dict(q_start=i32([0])), dict(max_new=-1),
               dict(target=target[:1].expand(4, 100))):
        a = dict(target=target, tokens=tokens, uniform=uniform, draft=draft, q_start=s)
        a.update(kw)
        with pytest.raises(ValueError):
            cache.verify(**a)


def test_no_tokens(cuda_lib):
    cache = make_cache(4)
    e = torch.empty(0, 50, device=DEV)
    keep, after = cache.verify(e, i32([]), torch.empty(0, device=DEV), q_start=i32([0] * 5))
    assert keep.tolist() == [0] * 4 and after.tolist() == [-1] * 4


def test_large_offsets_and_captured_calls(cuda_lib):
    """Rows behind 2^31 entries; a captured call replays with new tokens and starts."""
    N, V = 9000, 250000
    target = torch.zeros(N, V, dtype=torch.bfloat16, device=DEV)
    tokens = torch.zeros(N, dtype=torch.int32, device=DEV)
    uniform = torch.full((N,), 0.4, device=DEV)
    rows = [8997, 8998, 8999]
    for i, r in enumerate(rows):
        target[r, 249999 - i] = 1.0
    tokens[8998] = 249999
    cache = make_cache(2)
    s = i32([0, 1, 2])
    cache.verify(target, tokens, uniform, q_start=s, max_new=8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        keep, after = cache.verify(target, tokens, uniform, q_start=s, max_new=8)
    s.copy_(i32([8996, 8997, 9000]))
    graph.replay()
    assert keep.tolist() == [1, 2] and after.tolist() == [-1, 249998]
    tokens[8999] = 249998
    graph.replay()
    assert keep.tolist() == [1, 3] and after.tolist() == [-1, 249997]
