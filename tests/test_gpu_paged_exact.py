"""The paged attention held to what its formats leave: errors of a single rounding where there is a single one, peaked
softmax on inputs whose scores are exact, hidden pages against the definition."""
import math

import pytest
import torch

import paged_ref as R
from test_gpu_paged import DEV, run, to_cache

pytestmark = pytest.mark.gpu
R0 = 0.00166  # rms of bf16's relative rounding error: 2^-8 / sqrt(3) * sqrt(mean of 1 / m^2), m log-uniform in [1, 2)


@pytest.mark.parametrize("d,hq,hkv,t,n,fox,window", [
    (64, 4, 4, [900, 300], [1, 1], False, 0), (128, 8, 2, [900, 300], [1, 1], False, 0), (64, 8, 2, [900, 300], [1, 1], True, 200),
    (64, 2, 2, [700, 300], [8, 5], False, 0), (64, 1, 1, [700, 300], [16, 9], True, 0), (128, 4, 2, [700, 300], [8, 5], False, 0)])
def test_streaming_pass_rounds_once(cuda_lib, d, hq, hkv, t, n, fox, window):
    """Single tokens and drafts hold z, P and the rewrite's coefficients as bf16 pairs: each of the at most 16 roundings
    of a term is 2^-18 of it, so beside the rounding of o, and of the stored key, at most 2^-14 of the norm is off."""
    c = R.make_case("bf16", d, hq, hkv, 32, t, n, fox, seed=d + sum(n), nan_fill=False)
    scale = 1 / math.sqrt(d)
    o, _, k, _, _ = R.extend_ref(c, scale, window, 4 if window else 0)
    got, cache = run(c, scale, window, 4 if window else 0)
    cache.check()
    for x, ref in ((got["o"], o), (got["k"], k)):
        own = float((ref.to(torch.bfloat16).double() - ref).norm())
        assert float((x.double() - ref).norm()) <= own + 2.0 ** -14 * float(ref.norm())


@pytest.mark.parametrize("d,hq,hkv,t,n,roundings", [
    (64, 4, 2, 0, 200, 1), (128, 4, 4, 0, 200, 1),    # one block, nothing cached: o's own rounding
    (64, 4, 2, 1500, 200, 2), (64, 2, 2, 1500, 600, 2),  # P beside it
    (128, 8, 2, 1500, 30, 2), (128, 8, 2, 1500, 300, 3)])  # and, above 128 query rows at head dim 128, z
def test_prompts_round_as_often_as_they_say(cuda_lib, d, hq, hkv, t, n, roundings):
    """Independent roundings of bf16's relative rms R0 each (scores have a deviation of about 1, so that z's moves them
    by R0); a tenth on top for what pairs leave, the sample, and, over several blocks, the carried keys' copies."""
    c = R.make_case("bf16", d, hq, hkv, 64, [t], [n], seed=d + n, nan_fill=False)
    scale = 1 / math.sqrt(d)
    o, *_ = R.extend_ref(c, scale)
    got, cache = run(c, scale)
    cache.check()
    assert float((got["o"].double() - o).norm() / o.norm()) <= 1.1 * math.sqrt(roundings) * R0


@pytest.mark.parametrize("dtype,d,n", [("bf16", 64, [1, 1]), ("bf16", 128, [1, 1]), ("bf16", 64, [8, 3]), ("bf16", 64, [70, 20]),
                                       ("bf16", 128, [70, 20]), ("bf16", 128, [300, 20]), ("fp32", 64, [1, 1]), ("fp32", 128, [70, 20])])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_peaked_softmax(cuda_lib, dtype, d, n, sign):
    """Scores up to 2000 in steps of 8, rising and falling along the sequence: the running maximum moves at nearly every
    tile.  Queries and keys are small whole numbers along two axes and beta is 0, so that every product is exact; the
    score in log2 units is then off by three fp32 roundings (2900 2^-24 each, 3.6e-4 as a factor of p), beside which P and
    o are rounded (bf16) or the sums of about a thousand terms are (fp32, 2^-13)."""
    c = R.make_case(dtype, d, 4, 2, 32, [900, 333], n, seed=d + sum(n), nan_fill=False)
    g = torch.Generator().manual_seed(4)

    def ramps(rows):  # whole numbers 0..255, in a scattered order with rising and falling stretches
        x = torch.randint(0, 256, (rows, 2, 2), generator=g).double()
        x[: rows // 3], _ = x[: rows // 3].sort(0)
        x[rows // 3 : rows // 2], _ = x[rows // 3 : rows // 2].sort(0, descending=True)
        return x

    def keys(rows):
        k = torch.zeros(rows, 2, d)
        k[..., :2] = ramps(rows)
        return k.to(R.DT[dtype])

    for b, t in enumerate(c["t"]):
        pos = torch.arange(t)
        c["k_pool"][c["k_table"][b, pos // 32].long(), :, pos % 32] = keys(t)
    c["k"] = keys(sum(n))
    q = torch.zeros(sum(n), 4, d)
    for i in range(sum(n)):
        for h in range(4):
            q[i, h, (i + h) % 2] = 8.0
    c["q"] = q.to(R.DT[dtype])
    c["beta"].zero_()
    o, A, *_ = R.extend_ref(c, sign)
    got, cache = run(c, sign)
    cache.check()
    off = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -13
    err = (got["o"].double() - o).abs()
    assert (err <= off * o.abs() + (off + 3.6e-4) * A + 1e-30).all(), float((err / A).max())


@pytest.mark.parametrize("dtype,d,n", [("bf16", 64, [1, 1, 1]), ("bf16", 128, [1, 1, 1]), ("bf16", 64, [8, 8, 8]), ("bf16", 64, [70, 70, 70]),
                                       ("bf16", 128, [70, 300, 1]), ("fp32", 64, [1, 1, 1]), ("fp32", 128, [5, 40, 1])])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("pool", ["k", "v", "both"])
def test_rows_of_a_missing_page_are_hidden(cuda_lib, dtype, d, n, fox, pool):
    """A page that is missing among the cached ones: the sequence without its rows, and nothing written there.  (Without a
    window positions only order the rows, so that this is the definition with the page's column taken out.)"""
    P = 16
    c = R.make_case(dtype, d, 4, 2, P, [100, 100, 100], n, fox, seed=d + sum(n))
    bad = dict(c, k_table=c["k_table"].clone(), v_table=c["v_table"].clone())
    without = dict(c, k_table=c["k_table"].clone(), v_table=c["v_table"].clone(), t=[100, 100 - P, 100])
    kept = int(c["k_table"][1, 2])
    for x in ("k", "v"):
        if pool in (x, "both"):
            bad[x + "_table"][1, 2] = 10 ** 9 if x == "k" else -1
        row = c[x + "_table"][1]
        without[x + "_table"][1] = torch.cat([row[:2], row[3:], torch.tensor([-1], dtype=torch.int32)])
    ref = R.extend_ref(without, 0.125)
    got, cache = run(bad, 0.125)
    with pytest.raises(RuntimeError, match="page-table"):
        cache.check()
    if pool == "v":  # the key page is there: whether its rows are moved on is left open
        got["k"][kept] = ref[2][kept].to(got["k"].dtype)
    R.check_extend(without, got, ref, 0.125)
