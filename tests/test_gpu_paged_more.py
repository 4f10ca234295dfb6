"""More calls of the paged attention against the plain 64-bit form: odd head groups, draft widths, windows across key
tiles, several passes over a long prompt, many slots, padded packs, pools above 2^31 elements, two streams."""
import math

import pytest
import torch

import paged_ref as R
from test_gpu_paged import DEV, run, to_cache

pytestmark = pytest.mark.gpu

CASES = [
    # dtype, d, hq, hkv, page, cached, new, fox, window, sinks
    # fp32: every number of heads per key head the single-token pass pairs, and odd ones
    ("fp32", 64, 4, 1, 16, [200, 31], [1, 1], True, 0, 0),
    ("fp32", 128, 16, 2, 32, [64, 257], [1, 1], False, 0, 0),
    ("fp32", 64, 16, 1, 64, [100], [1], False, 30, 2),
    ("fp32", 128, 5, 1, 16, [129, 0], [1, 1], True, 0, 0),
    ("fp32", 64, 12, 2, 16, [90, 16], [1, 70], True, 0, 0),
    ("fp32", 128, 8, 1, 128, [300, 128], [129, 1], False, 64, 5),
    # single tokens: 3, 6, 12 heads per key head, gates, 128 wide rows on every page size
    ("bf16", 64, 3, 1, 16, [300, 16], [1, 1], False, 0, 0),
    ("bf16", 128, 12, 2, 16, [300, 15], [1, 1], True, 0, 0),
    ("bf16", 128, 12, 1, 32, [513, 0], [1, 1], False, 0, 0),
    ("bf16", 64, 64, 4, 256, [1025], [1], True, 200, 0),
    ("bf16", 128, 2, 2, 128, [1025, 255], [1, 1], True, 7, 9),
    # drafts: 9 to 16 columns and 17 to 32, one token beside eight, widths at the edge of the streaming pass
    ("bf16", 64, 3, 1, 16, [190, 16], [3, 5], True, 0, 0),
    ("bf16", 64, 4, 1, 32, [400, 0], [8, 1], False, 0, 0),
    ("bf16", 64, 6, 2, 64, [128, 127], [8, 6], True, 30, 1),
    ("bf16", 64, 1, 1, 64, [600, 63], [16, 11], False, 0, 0),
    ("bf16", 64, 2, 1, 16, [100, 48], [9, 16], True, 0, 0),
    ("bf16", 128, 2, 2, 32, [200, 1], [16, 9], False, 0, 0),
    ("bf16", 128, 8, 2, 16, [500, 64], [4, 2], True, 100, 0),
    ("bf16", 128, 8, 2, 16, [500, 64], [5, 2], True, 100, 0),
    ("bf16", 128, 16, 1, 256, [300], [2], False, 0, 0),
    ("bf16", 64, 2, 2, 16, [500], [13], False, 5, 2),
    # prompt chunks: several blocks with 3, 5 and 6 heads per key head, gates, windows that start inside a block
    ("bf16", 64, 3, 1, 16, [0, 33], [600, 290], False, 0, 0),
    ("bf16", 64, 5, 1, 32, [700], [513], True, 0, 0),
    ("bf16", 128, 6, 1, 16, [129], [520], True, 0, 0),
    ("bf16", 128, 3, 1, 128, [0], [770], False, 300, 2),
    ("bf16", 64, 6, 2, 64, [400, 0], [300, 257], True, 129, 130),
    ("bf16", 64, 2, 2, 16, [1000], [530], False, 1, 0),
    ("bf16", 128, 2, 1, 64, [1000], [270], True, 1000, 1),
    ("bf16", 64, 16, 1, 64, [65], [66], False, 0, 0),
    # one token, drafts and a prompt in one call; empty and fresh slots between them
    ("bf16", 64, 4, 2, 16, [300, 20, -1, 0, 64, 5], [1, 5, 0, 300, 0, 64], True, 0, 0),
    ("bf16", 128, 8, 2, 32, [300, 20, 700, 0], [1, 1, 70, 1], False, 33, 1),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_extend_matches_the_definition(cuda_lib, case):
    dtype, d, hq, hkv, page, t, n, fox, window, sinks = case
    c = R.make_case(dtype, d, hq, hkv, page, t, n, fox, seed=sum(t) + 11 * sum(n) + d + 1)
    scale = 1.0 / math.sqrt(d)
    got, cache = run(c, scale, window, sinks)
    R.check_extend(c, got, R.extend_ref(c, scale, window, sinks), scale)
    cache.check()


@pytest.mark.parametrize("fox,window", [(False, 0), (True, 500)])
def test_a_prompt_of_more_than_one_pass(cuda_lib, fox, window):
    """4200 new tokens beside 70 and one: the keys are carried on over 4096 tokens, then over the rest."""
    c = R.make_case("bf16", 64, 2, 1, 64, [100, 40, 200], [4200, 70, 1], fox, seed=3)
    got, cache = run(c, 0.125, window, 3 if window else 0)
    ref = R.extend_ref(c, 0.125, window, 3 if window else 0)
    if window:  # new keys that the window hides before the second pass are left as the first stored them
        pos = torch.arange(100 + 3, 100 + 4200 - window + 1)
        page, row = c["k_table"][0, pos // 64].long(), pos % 64
        assert torch.isfinite(got["k"][page, :, row]).all()
        got["k"][page, :, row] = ref[2][page, :, row].to(got["k"].dtype)
    R.check_extend(c, got, ref, 0.125, passes=2)
    cache.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_more_slots_than_one_block_scans(cuda_lib, dtype):
    """1500 slots, most of them with one token, a few empty, idle or with a chunk."""
    t = [(7 * b) % 50 if b % 11 else -1 for b in range(1500)]
    n = [0 if x < 0 or b % 13 == 0 else (20 if b % 97 == 1 else 1) for b, x in enumerate(t)]
    c = R.make_case(dtype, 64, 2, 1, 16, t, n, seed=4, slack=0, width_slack=0)
    got, cache = run(c, 0.125)
    R.check_extend(c, got, R.extend_ref(c, 0.125), 0.125)
    cache.check()
    c = R.make_case(dtype, 64, 2, 1, 16, [x if x >= 0 else 5 for x in t], [1] * 1500, seed=5, slack=0, width_slack=0)
    got, cache = run(c, 0.125, q_start=False)
    R.check_extend(c, got, R.extend_ref(c, 0.125), 0.125)
    cache.check()


@pytest.mark.parametrize("n", [[1, 1, 1], [6, 1, 4], [70, 1, 260]])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_padded_pack_and_generous_max_new(cuda_lib, dtype, n):
    """Rows of the packed tensors behind the last sequence are neither read (NaN) nor written, and a max_new larger
    than every count changes no result beyond the bound."""
    c = R.make_case(dtype, 64, 4, 2, 32, [90, 33, 200], n, seed=6)
    ref = R.extend_ref(c, 0.125)
    N = sum(n)
    pad = dict(c)
    for x in ("q", "k", "v", "w", "beta"):
        pad[x] = torch.cat([c[x], torch.full((40,) + c[x].shape[1:], float("nan"), dtype=c[x].dtype)])
    for max_new in (max(n), max(n) + 30):
        out = torch.full_like(pad["q"], 5.0).to(DEV)
        got, cache = run(pad, 0.125, out=out, max_new=max_new)
        assert (got["o"][N:] == 5).all()
        got["o"] = got["o"][:N]
        R.check_extend(c, got, ref, 0.125)
        cache.check()


@pytest.mark.parametrize("n", [[1, 1], [7, 3], [100, 90]])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_nan_in_one_slot_stays_there(cuda_lib, dtype, n):
    c = R.make_case(dtype, 64, 4, 2, 16, [150, 77], n, seed=8)
    ref = R.extend_ref(c, 0.125)
    bad = {x: c[x].clone() for x in ("q", "k", "v", "w", "beta")}
    for x in bad.values():
        x[: n[0]] = float("nan")
    got, _ = run(dict(c, **bad), 0.125)
    o, r = got["o"][n[0] :].double(), ref[0][n[0] :]
    fro = (2 if dtype == "bf16" else 256) * R.U[dtype]
    assert float((o - r).norm() / r.norm()) <= fro
    pages = c["k_table"][1][c["k_table"][1] >= 0].long()
    k, kr = got["k"][pages].double(), ref[2][pages]
    assert torch.equal(torch.isnan(k), torch.isnan(kr))
    kfro = R.U["bf16"] + 2 * 2.0 ** -11 if dtype == "bf16" else 64 * R.U["fp32"]
    assert float(torch.nan_to_num(k - kr).norm() / torch.nan_to_num(kr).norm()) <= kfro


@pytest.mark.parametrize("dtype,d,n", [("bf16", 128, [1, 1]), ("bf16", 128, [6, 3]), ("bf16", 128, [130, 300]), ("fp32", 64, [1, 40])])
def test_pools_above_two_to_the_31_elements(cuda_lib, dtype, d, n):
    """The used pages lie at the far end of pools whose offsets pass 32 bits."""
    from softmax_attention_chunk_gb300.paged import PagedCache

    c = R.make_case(dtype, d, 4, 2, 64, [200, 31], n, seed=9, nan_fill=False)
    few = c["k_pool"].shape[0]
    pages = 2 ** 31 // (2 * 64 * d) + 64 + few
    lift = pages - few
    pools = [torch.zeros(pages, 2, 64, d, dtype=R.DT[dtype], device=DEV) for _ in range(2)]
    assert pools[0].numel() > 2 ** 31
    for pool, x in zip(pools, ("k_pool", "v_pool")):
        pool[lift:].copy_(c[x])
    tables = [torch.where(c[x] >= 0, c[x] + lift, c[x]).to(DEV) for x in ("k_table", "v_table")]
    refs = [torch.nn.functional.pad(c[x], (lift, 0)).to(DEV) for x in ("k_ref", "v_ref")]
    cache = PagedCache.from_tensors(pools[0], pools[1], tables[0], tables[1], c["seq_len"].to(DEV), refs[0], refs[1])
    got, _ = run(c, 0.1, cache=cache)
    got["k"], got["v"] = got["k"][lift:], got["v"][lift:]
    R.check_extend(c, got, R.extend_ref(c, 0.1), 0.1)
    cache.check()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    before = [int(x) for x in cache.k_table[0][: -(-200 // 64)]]
    cache.free(i32([1]))
    cache.fork(i32([0]), i32([1]))  # the copies go to the lowest free pages
    cache.check()
    for b, page in enumerate(before):
        copy = int(cache.k_table[1, b])
        rows = min(64, 200 - 64 * b)
        assert copy < few and torch.equal(cache.k_pool[copy, :, :rows], cache.k_pool[page, :, :rows])
    cache.compact()
    cache.check()
    assert int(cache.k_table.max()) < few and int(cache.v_table.max()) < few


def test_two_caches_on_two_streams(cuda_lib):
    """Calls in flight at once share nothing."""
    a = R.make_case("bf16", 64, 4, 2, 32, [3000, 64], [9, 1], seed=41)
    b = R.make_case("bf16", 64, 4, 2, 32, [2000, 500], [200, 90], seed=42)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    ca, cb = to_cache(a), to_cache(b)
    ins = [{x: c[x].to(DEV) for x in ("q", "k", "v", "w", "beta", "q_start")} for c in (a, b)]
    torch.cuda.synchronize()
    outs = []
    for stream, cache, i, m in ((s, ca, ins[0], 9), (t, cb, ins[1], 200)):
        with torch.cuda.stream(stream):
            outs.append(cache.extend(i["q"], i["k"], i["v"], i["w"], i["beta"], q_start=i["q_start"], max_new=m, scale=0.125))
    torch.cuda.synchronize()
    for c, cache, o in ((a, ca, outs[0]), (b, cb, outs[1])):
        R.check_extend(c, dict(o=o.cpu(), k=cache.k_pool.cpu(), v=cache.v_pool.cpu()), R.extend_ref(c, 0.125), 0.125)


def test_two_captured_steps_of_one_cache(cuda_lib):
    """Two graphs of the same cache, replayed in turn: each has its own workspace, and the second reads the keys the
    first wrote."""
    n = [1, 1, 1]
    c = R.make_case("bf16", 64, 4, 2, 32, [90, 33, 200], n, seed=51, slack=4, width_slack=2)
    cache = to_cache(c)
    ins = {x: c[x].to(DEV) for x in ("q", "k", "v", "w", "beta")}
    keep = {x: getattr(cache, x).clone() for x in ("k_pool", "v_pool", "seq_len")}

    def step():
        o = cache.extend(ins["q"], ins["k"], ins["v"], ins["w"], ins["beta"], scale=0.125)
        cache.advance()
        return o

    graphs = []
    step()
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = step()
        graphs.append((g, o))
    for x, y in keep.items():
        getattr(cache, x).copy_(y)
    cache.reserve(torch.full((3,), 2, dtype=torch.int32, device=DEV))
    t = list(c["t"])
    for g, o in graphs:
        now = dict(c, t=t, seq_len=torch.tensor(t, dtype=torch.int32), k_pool=cache.k_pool.cpu(), v_pool=cache.v_pool.cpu(),
                   k_table=cache.k_table.cpu(), v_table=cache.v_table.cpu())
        g.replay()
        torch.cuda.synchronize()
        R.check_extend(now, dict(o=o.cpu(), k=cache.k_pool.cpu(), v=cache.v_pool.cpu()), R.extend_ref(now, 0.125), 0.125)
        t = [x + 1 for x in t]
    assert cache.seq_len.tolist() == t
    cache.check()


@pytest.mark.parametrize("dtype,fox", [("bf16", False), ("bf16", True), ("fp32", True)])
def test_overlapping_ranges_stay_in_bounds(cuda_lib, dtype, fox):
    """q_start rows that each look right but name more tokens together than there are: these slots are left out."""
    c = R.make_case(dtype, 64, 4, 2, 16, [40] * 9, [30] * 9, fox, seed=61, width_slack=30)
    N = 270
    bad = dict(c, q_start=torch.tensor([0, N, 0, N, 0, N, 0, N, 0, N], dtype=torch.int32))
    out = torch.full((N, 4, 64), 3.0, dtype=R.DT[dtype], device=DEV)
    got, cache = run(bad, 0.125, out=out, max_new=N)
    assert (got["o"] == 3).all()
    assert torch.equal(torch.nan_to_num(got["k"]), torch.nan_to_num(c["k_pool"]))
    with pytest.raises(RuntimeError, match="q_start"):
        cache.check()
    got, cache = run(c, 0.125)
    R.check_extend(c, got, R.extend_ref(c, 0.125), 0.125)
    cache.check()


def test_long_fp32_prompt_with_the_gate(cuda_lib):
    c = R.make_case("fp32", 64, 2, 1, 16, [70, 5], [600, 300], True, seed=62)
    got, cache = run(c, 0.125)
    R.check_extend(c, got, R.extend_ref(c, 0.125), 0.125)
    cache.check()


@pytest.mark.parametrize("dtype,max_new", [("bf16", 5), ("bf16", 40), ("fp32", 5)])
def test_one_token_per_slot_with_a_generous_max_new(cuda_lib, dtype, max_new):
    c = R.make_case(dtype, 64, 4, 2, 32, [40, 0, 129, 64, 7, 300], [1] * 6, seed=63)
    cache = to_cache(c)
    ins = [c[x].to(DEV) for x in ("q", "k", "v", "w", "beta")]
    o = cache.extend(*ins, max_new=max_new, scale=0.125)
    torch.cuda.synchronize()
    R.check_extend(c, dict(o=o.cpu(), k=cache.k_pool.cpu(), v=cache.v_pool.cpu()), R.extend_ref(c, 0.125), 0.125)
    cache.check()
