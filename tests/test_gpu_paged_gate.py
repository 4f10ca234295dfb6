"""The forget gate far into a sequence: running sums much larger than a token's log f keep what each token adds."""
import pytest
import torch

import paged_ref as R
from test_gpu_paged import DEV, to_cache

pytestmark = pytest.mark.gpu
BASE = -300000.0  # a sum after 1.5 million tokens at -0.2; fp32 numbers are 2^-5 apart here


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def far_case(dtype, d, t, total, seed):
    """t cached tokens whose sums lie at BASE, and `total` new ones whose log f are less than half a step of that.  beta 0:
    keys stay as they are, so that nothing but the gate changes from call to call."""
    c = R.make_case(dtype, d, 4, 2, 16, [t], [total], True, seed=seed, slack=20, width_slack=2)
    g = torch.Generator().manual_seed(seed)
    c["beta"].zero_()
    c["log_f"] = -0.015 * torch.rand(total, 2, generator=g) - 1e-4
    c["a_pool"] = torch.where(torch.isnan(c["a_pool"]), c["a_pool"], torch.full_like(c["a_pool"], BASE))
    return c


@pytest.mark.parametrize("dtype,d,n,calls", [("bf16", 64, 1, 150), ("bf16", 128, 1, 150), ("bf16", 64, 5, 60), ("bf16", 64, 40, 10),
                                             ("bf16", 128, 300, 3), ("fp32", 64, 1, 150), ("fp32", 128, 1, 60), ("fp32", 64, 40, 10)])
def test_sums_far_into_a_sequence(cuda_lib, dtype, d, n, calls):
    """Many calls of few tokens against the definition over all tokens at once.  o: the bounds of one call (no key is
    rounded).  Sums: of a call's n terms, fp32 roundings of at most n 2^-24 |their sum|; what the calls then add up as a
    pair of fp32 numbers is off by 2^-48 of 3e5 each."""
    t, total = 40, n * calls
    c = far_case(dtype, d, t, total, seed=n + d)
    scale = 0.05
    o, _, _, _, a = R.extend_ref(c, scale)
    cache = to_cache(c)
    dev = {x: c[x].to(DEV) for x in ("q", "k", "v", "w", "beta", "log_f")}
    outs = []
    for i in range(calls):
        s = slice(n * i, n * (i + 1))
        x = {y: v[s] if v[s].data_ptr() % 16 == 0 else v[s].clone() for y, v in dev.items()}
        outs.append(cache.extend(x["q"], x["k"], x["v"], x["w"], x["beta"], log_f=x["log_f"], q_start=i32([0, n]), max_new=n, scale=scale))
        cache.advance(i32([0, n]))
    cache.check()
    got = torch.cat(outs).cpu().double()
    u = R.U[dtype] * (2 if dtype == "bf16" else 256)
    assert float((got - o).norm() / o.norm()) <= u
    sums = cache.a_pool.cpu().double() + cache.a_rest.cpu().double()
    assert torch.equal(torch.isnan(sums), torch.isnan(a))
    bound = n * 2.0 ** -24 * float(c["log_f"].double().sum(0).abs().max()) + calls * 2.0 ** -48 * abs(BASE)
    assert float(torch.nan_to_num(sums - a).abs().max()) <= bound
    # the fp32 numbers are the sums' nearest ones
    assert float(torch.nan_to_num(cache.a_pool.cpu().double() - a).abs().max()) <= 2.0 ** -6 + bound


def test_pages_take_the_rest_along(cuda_lib):
    """A fork and a compaction move both parts of the sums: parent and child give the same bits from there on, and the
    definition's outputs."""
    c = far_case("bf16", 64, 40, 70, seed=3)
    o, *_ = R.extend_ref(c, 0.05)
    k_table = torch.cat([c["k_table"], torch.full_like(c["k_table"], -1)])
    v_table = torch.cat([c["v_table"], torch.full_like(c["v_table"], -1)])
    cache = to_cache(dict(c, k_table=k_table, v_table=v_table, seq_len=torch.tensor([40, -1], dtype=torch.int32)))
    dev = {x: c[x].to(DEV) for x in ("q", "k", "v", "w", "beta", "log_f")}

    def call(x, start, max_new):
        o = cache.extend(x["q"], x["k"], x["v"], x["w"], x["beta"], log_f=x["log_f"], q_start=i32(start), max_new=max_new, scale=0.05)
        cache.advance(i32(start))
        return o

    for i in range(60):
        call({y: v[i : i + 1].clone() for y, v in dev.items()}, [0, 1, 1], 1)
    cache.fork(i32([0]), i32([1]))
    cache.compact()
    cache.reserve(i32([10, 10]))
    both = {y: torch.cat([v[60:70], v[60:70]]) for y, v in dev.items()}
    x = call(both, [0, 10, 20], 10).cpu()
    cache.check()
    assert torch.equal(x[:10], x[10:])
    assert float((x[:10].double() - o[60:]).norm() / o[60:].norm()) <= 2 * R.U["bf16"]


@pytest.mark.parametrize("dtype,n", [("bf16", [1, 1]), ("bf16", [6, 3]), ("bf16", [70, 1]), ("fp32", [1, 1]), ("fp32", [6, 40])])
def test_without_a_place_for_the_rest(cuda_lib, dtype, n):
    """The C ABI's cache may have none: the sums are then fp32 numbers, as they come in."""
    c = R.make_case(dtype, 64, 4, 2, 16, [40, 300], n, True, seed=sum(n))
    cache = to_cache(c)
    cache.c.a_rest = None
    from test_gpu_paged import run

    got, _ = run(c, 0.125, cache=cache)
    R.check_extend(c, got, R.extend_ref(c, 0.125), 0.125)
    cache.check()
