"""Attention of new tokens over a paged cache against the plain 64-bit form: types, head layouts, lengths,
odd sizes, windows, bad pages, captured graphs, and a served run with forks, trims and compaction."""
import math

import pytest
import torch

import paged_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def to_cache(c):
    from softmax_attention_chunk_gb300.paged import PagedCache

    t = {k: c[k].to(DEV) for k in ("k_pool", "v_pool", "k_table", "v_table", "seq_len", "k_ref", "v_ref")}
    return PagedCache.from_tensors(**t, a_pool=c["a_pool"].to(DEV) if c["fox"] else None)


def run(c, scale, window=0, sinks=0, q_start=True, cache=None, out=None, **kw):
    cache = cache or to_cache(c)
    dev = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    kw.setdefault("max_new", max(c["n"]) if q_start else None)
    o = cache.extend(dev(c["q"]), dev(c["k"]), dev(c["v"]), dev(c["w"]), dev(c["beta"]), log_f=dev(c["log_f"]),
                     q_start=dev(c["q_start"]) if q_start else None, scale=scale, window=window, sinks=sinks, out=out, **kw)
    torch.cuda.synchronize()
    got = dict(o=o.cpu(), k=cache.k_pool.cpu(), v=cache.v_pool.cpu())
    if c["fox"]:
        got["a"] = cache.a_pool.cpu()
    return got, cache


CASES = [
    # dtype, d, hq, hkv, page, cached, new, fox, window, sinks
    ("fp32", 64, 2, 2, 16, [0], [1], False, 0, 0),
    ("fp32", 64, 4, 2, 16, [5, 0, 33, 64, 1], [1, 1, 1, 1, 1], False, 0, 0),
    ("fp32", 64, 2, 1, 32, [70, 0, 129], [40, 65, 3], True, 0, 0),
    ("fp32", 128, 3, 1, 64, [100, 31], [33, 64], False, 0, 0),
    ("fp32", 128, 2, 2, 16, [200, 0], [1, 17], True, 40, 3),
    ("bf16", 64, 1, 1, 64, [0], [1], False, 0, 0),
    ("bf16", 64, 1, 1, 64, [1], [1], False, 0, 0),
    ("bf16", 64, 16, 16, 64, [515], [1], False, 0, 0),
    ("bf16", 64, 8, 2, 16, [15, 16, 17, 0, 300], [1, 1, 1, 1, 1], False, 0, 0),
    ("bf16", 64, 16, 1, 128, [260, 3], [1, 1], True, 0, 0),
    ("bf16", 64, 10, 2, 32, [77, 128], [1, 1], False, 0, 0),
    ("bf16", 128, 8, 2, 64, [64, 1000, 1, 0], [1, 1, 1, 1], False, 0, 0),
    ("bf16", 128, 16, 1, 256, [700], [1], True, 0, 0),
    ("bf16", 64, 4, 4, 16, [500, 90, 30], [1, 1, 1], True, 64, 4),
    ("bf16", 64, 4, 4, 16, [500, 90, 30], [1, 1, 1], False, 1, 0),
    ("bf16", 128, 4, 2, 32, [600, 10], [1, 1], False, 100, 70),
    ("bf16", 64, 4, 2, 32, [200, 0, 65], [8, 8, 8], False, 0, 0),
    ("bf16", 64, 4, 4, 32, [130, 7, 64, 0], [2, 16, 1, 9], True, 0, 0),
    ("bf16", 128, 4, 2, 64, [333, 64], [5, 7], True, 0, 0),
    ("bf16", 128, 16, 2, 64, [333, 64], [3, 16], False, 50, 2),
    ("bf16", 64, 2, 2, 64, [300, 0], [64, 65], False, 0, 0),
    ("bf16", 64, 8, 2, 16, [200, 129, 0, 40], [130, 1, 200, 31], True, 0, 0),
    ("bf16", 64, 4, 4, 64, [700], [257], False, 90, 4),
    ("bf16", 64, 2, 1, 128, [1100], [300], True, 256, 0),
    ("bf16", 128, 8, 2, 64, [500, 3, 64], [192, 33, 1], False, 0, 0),
    ("bf16", 128, 2, 2, 256, [300], [140], True, 33, 1),
    ("bf16", 128, 6, 2, 32, [0, 90], [300, 0], False, 0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_extend_matches_the_definition(cuda_lib, case):
    dtype, d, hq, hkv, page, t, n, fox, window, sinks = case
    c = R.make_case(dtype, d, hq, hkv, page, t, n, fox, seed=sum(t) + 7 * sum(n) + d)
    scale = 1.0 / math.sqrt(d)
    ref = R.extend_ref(c, scale, window, sinks)
    got, cache = run(c, scale, window, sinks)
    R.check_extend(c, got, ref, scale)
    cache.check()


@pytest.mark.parametrize("dtype,d,hq,hkv,fox", [("bf16", 64, 4, 2, False), ("bf16", 128, 8, 1, True), ("fp32", 64, 2, 2, True)])
def test_one_token_per_slot_without_q_start(cuda_lib, dtype, d, hq, hkv, fox):
    """Empty slots are left out: their rows of o keep what they held."""
    t = [40, -1, 0, 129, -1]
    c = R.make_case(dtype, d, hq, hkv, 32, t, [1] * 5, fox, seed=5)
    ref = R.extend_ref(c, 0.2)
    out = torch.full((5, hq, d), 7.0, dtype=R.DT[dtype], device=DEV)
    got, cache = run(c, 0.2, q_start=False, out=out)
    R.check_extend(c, got, ref, 0.2, tokens=[0, 2, 3])
    assert (got["o"][[1, 4]] == 7).all()
    cache.check()
    cache.advance()
    torch.cuda.synchronize()
    assert cache.seq_len.tolist() == [41, -1, 1, 130, -1]


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
@pytest.mark.parametrize("n", [[1, 1], [70, 20]])
def test_scales(cuda_lib, n, scale):
    """Score scale 0, negative, and large (peaked softmax, many changes of the running maximum)."""
    c = R.make_case("bf16", 64, 4, 2, 32, [300, 64], n, seed=9)
    got, _ = run(c, scale)
    o, A, *_ = ref = R.extend_ref(c, scale)
    if abs(scale) <= 0.3:
        R.check_extend(c, got, ref, abs(scale))
    else:
        # scores of up to 2 * 64 off by (u + 4 u_t) relative: probabilities may shift by about one; the
        # values stay a mean of v, and most rows (one clear maximum) agree
        assert torch.isfinite(got["o"]).all()
        assert ((got["o"].double() - o).abs().amax(-1) < 0.25).double().mean() > 0.8


@pytest.mark.parametrize("n", [[1, 1, 1], [8, 8, 8], [70, 70, 70]])
def test_bad_pages_and_rows_are_reported_and_touch_nothing_else(cuda_lib, n):
    """A table entry outside the pool hides its rows; a slot that would outgrow its table, or whose row of q_start is
    bad, is left out whole.  The other slots' results are those of a clean call."""
    c = R.make_case("bf16", 64, 4, 2, 16, [100, 100, 100], n, seed=3)
    ref = R.extend_ref(c, 0.125)
    first, second, third = (torch.arange(int(c["q_start"][b]), int(c["q_start"][b + 1])) for b in range(3))
    bad = dict(c, k_table=c["k_table"].clone())
    bad["k_table"][1, 2] = 10 ** 9
    got, cache = run(bad, 0.125)
    assert torch.isfinite(got["o"]).all()
    with pytest.raises(RuntimeError, match="page-table"):
        cache.check()
    cache.check()  # cleared
    for sel in (first, third):
        assert float((got["o"].double() - ref[0])[sel].norm() / ref[0][sel].norm()) < 2 * R.U["bf16"]
    # too long for the table row
    long = dict(c, seq_len=torch.tensor([100, 16 * c["k_table"].shape[1] - n[1] + 1, 100], dtype=torch.int32))
    out = torch.full_like(c["q"], 3.0).to(DEV)
    got, cache = run(long, 0.125, out=out)
    assert (got["o"][second] == 3).all()
    with pytest.raises(RuntimeError, match="outgrow"):
        cache.check()
    for sel in (first, third):
        assert float((got["o"].double() - ref[0])[sel].norm() / ref[0][sel].norm()) < 2 * R.U["bf16"]
    # a falling q_start: slot 1 would have a negative count, slot 2 too many
    s = c["q_start"].clone()
    s[2] = s[1] - 1
    out = torch.full_like(c["q"], 3.0).to(DEV)
    got, cache = run(dict(c, q_start=s), 0.125, out=out)
    assert (got["o"][torch.cat([second, third])] == 3).all()
    with pytest.raises(RuntimeError, match="q_start"):
        cache.check()
    assert float((got["o"].double() - ref[0])[first].norm() / ref[0][first].norm()) < 2 * R.U["bf16"]


@pytest.mark.parametrize("n", [[1, 1, 1], [8, 3, 5], [70, 1, 33]])
def test_captured_step_replays_with_new_lengths(cuda_lib, n):
    """A captured call reads lengths and tables at every replay."""
    a = R.make_case("bf16", 64, 4, 2, 32, [90, 33, 200], n, seed=21)
    b = R.make_case("bf16", 64, 4, 2, 32, [10, 200, 64], n, seed=22)
    width, total = max(a["k_table"].shape[1], b["k_table"].shape[1]), max(a["k_pool"].shape[0], b["k_pool"].shape[0])

    def pad(c):
        c = dict(c)
        for x in ("k_table", "v_table"):
            c[x] = torch.nn.functional.pad(c[x], (0, width - c[x].shape[1]), value=-1)
        for x in ("k_pool", "v_pool"):
            c[x] = torch.cat([c[x], torch.zeros(total - c[x].shape[0], *c[x].shape[1:], dtype=c[x].dtype)])
        for x in ("k_ref", "v_ref"):
            c[x] = torch.nn.functional.pad(c[x], (0, total - c[x].shape[0]))
        return c

    a, b = pad(a), pad(b)
    cache = to_cache(a)
    ins = {x: a[x].to(DEV) for x in ("q", "k", "v", "w", "beta", "q_start")}
    call = lambda: cache.extend(ins["q"], ins["k"], ins["v"], ins["w"], ins["beta"], q_start=ins["q_start"],  # noqa: E731
                                max_new=max(n), scale=0.125)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = call()
    for c in (a, b, a):
        for x in ("q", "k", "v", "w", "beta", "q_start"):
            ins[x].copy_(c[x])
        for x in ("k_pool", "v_pool", "k_table", "v_table", "seq_len"):
            getattr(cache, x).copy_(c[x])
        g.replay()
        torch.cuda.synchronize()
        R.check_extend(c, dict(o=o.cpu(), k=cache.k_pool.cpu(), v=cache.v_pool.cpu()), R.extend_ref(c, 0.125), 0.125)
    cache.check()


def test_same_call_gives_the_same_bits(cuda_lib):
    for n in ([1, 1, 1], [8, 2, 16], [140, 1, 70]):
        c = R.make_case("bf16", 64, 8, 4, 64, [3000, 100, 900], n, seed=31)
        x, _ = run(c, 0.125)
        y, _ = run(c, 0.125)
        assert torch.equal(x["o"], y["o"]) and torch.equal(torch.nan_to_num(x["k"]), torch.nan_to_num(y["k"]))


def test_on_another_stream(cuda_lib):
    c = R.make_case("bf16", 64, 4, 2, 32, [300, 64], [9, 1], seed=41)
    s = torch.cuda.Stream()
    cache = to_cache(c)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, _ = run(c, 0.125, cache=cache)
    R.check_extend(c, got, R.extend_ref(c, 0.125), 0.125)


@pytest.mark.parametrize("dtype,d,fox", [("bf16", 64, False), ("bf16", 128, True), ("fp32", 64, True)])
def test_served_run(cuda_lib, dtype, d, fox):
    """Prompts in chunks, single tokens, a fork, a beam dropped, compaction, a window trimmed: the outputs of
    every step against the definition over the whole token history of each sequence."""
    from softmax_attention_chunk_gb300.paged import PagedCache

    H, G, P, slots, window, sinks = 2, 2, 16, 5, 48, 3
    scale = 1 / math.sqrt(d)
    dt = R.DT[dtype]
    cache = PagedCache(slots, H, d, P, k_pages=80, v_pages=60, table_width=20, dtype=dt, fox=fox)
    g = torch.Generator().manual_seed(d)
    hist = {b: None for b in range(slots)}  # (q, k, v, w, beta, log_f) of each live slot
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731

    def new_tok(m):
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        return (rnd(m, H * G, d).to(dt), rnd(m, H, d).to(dt), rnd(m, H, d).to(dt),
                torch.nn.functional.normalize(rnd(m, H, d), dim=-1).to(dt), 2 * torch.sigmoid(rnd(m, H)),
                torch.log(torch.sigmoid(rnd(m, H) + 2)))

    def step(counts, win=0):
        toks = [new_tok(m) for m in counts]
        packed = [torch.cat(x).to(DEV) for x in zip(*toks)]
        start = i32([0] + torch.tensor(counts).cumsum(0).tolist())
        cache.reserve(i32(counts))
        o = cache.extend(*packed[:5], log_f=packed[5] if fox else None, q_start=start, max_new=max(counts), scale=scale,
                         window=win, sinks=sinks if win else 0)
        cache.advance(start)
        cache.check()
        for b, m in enumerate(counts):
            if not m:
                continue
            old = hist[b]
            hist[b] = toks[b] if old is None else tuple(torch.cat(x) for x in zip(old, toks[b]))
            L = hist[b][0].shape[0]
            c = dict(dtype=dtype, d=d, hq=H * G, hkv=H, page=P, t=[0], n=[L], fox=fox,
                     q_start=torch.tensor([0, L]), k_table=torch.arange(64)[None].int(), v_table=torch.arange(64)[None].int(),
                     k_pool=torch.zeros(64, H, P, d, dtype=dt), v_pool=torch.zeros(64, H, P, d, dtype=dt),
                     a_pool=torch.zeros(64, H, P), **dict(zip(("q", "k", "v", "w", "beta", "log_f"), hist[b])))
            ref = R.extend_ref(c, scale, win, sinks if win else 0)[0][L - m :]
            got = o[int(start[b]) : int(start[b + 1])].cpu().double()
            # cached keys were rounded once per earlier call (at most 14 here) on top of one call's bound
            tol = (2 + math.sqrt(14)) * R.U["bf16"] if dtype == "bf16" else 1024 * R.U["fp32"]
            assert float((got - ref).norm() / ref.norm()) < tol, (b, m)

    step([37, 20, 0, 0, 0])
    step([30, 1, 0, 0, 0])
    step([1, 1, 0, 0, 0])
    cache.fork(i32([0, 0, 1]), i32([2, 3, 4]))
    for child, parent in ((2, 0), (3, 0), (4, 1)):
        hist[child] = hist[parent]
    cache.check()
    step([1, 1, 1, 1, 1])
    cache.free(i32([0, 4]))
    hist[0] = hist[4] = None
    step([0, 1, 5, 1, 0])
    cache.compact()
    cache.check()
    used = int((cache.k_ref > 0).sum())
    assert (cache.k_ref[:used] > 0).all() and (cache.k_ref[used:] == 0).all()
    step([33, 1, 1, 1, 0])
    for _ in range(5):  # slot 2 grows to 80 tokens: its rows 16..31 leave the window of 48
        step([1, 1, 1, 1, 0], win=window)
    before = int((cache.k_ref > 0).sum())
    cache.trim(window, sinks)
    cache.check()
    assert int((cache.k_ref > 0).sum()) < before
    step([1, 1, 9, 1, 0], win=window)
    cache.compact()
    step([1, 1, 1, 1, 0], win=window)
    cache.free(i32([0, 1, 2, 3]))
    cache.check()
    assert int(cache.k_ref.abs().sum()) == 0 and int(cache.v_ref.abs().sum()) == 0
    assert (cache.k_table == -1).all() and (cache.seq_len == -1).all()
