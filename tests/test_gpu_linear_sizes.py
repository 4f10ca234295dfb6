"""Linear attention at the sizes of a training step and of a serving program: several waves of blocks in one segment each, long
float32 sequences, states as exact as float32 sums, forks of large states."""
import math

import pytest
import torch

from linear_ref import check, final_state, reference
from test_gpu_linear import inputs, run
from test_gpu_linear_serving import DEV, expect, make, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d,batch,hq,hkv,L", [("bf16", 64, 10, 32, 32, 700), ("bf16", 64, 20, 64, 16, 400), ("bf16", 128, 8, 40, 40, 500),
                                                    ("bf16", 128, 24, 32, 8, 600), ("fp32", 64, 10, 32, 32, 300), ("fp32", 128, 12, 26, 13, 200)])
def test_several_waves_of_whole_sequences(cuda_lib, dtype, d, batch, hq, hkv, L):
    pa = cuda_lib
    desc = pa.path_linear_desc_t(batch, hq, hkv, L, d, pa.PATH_BF16 if dtype == "bf16" else pa.PATH_FP32, 0.2)
    assert pa.path_linear_workspace_size(desc, 1) == 256, "one segment: no states in the workspace"
    if dtype == "bf16":  # (the float32 forward of these is cut)
        assert pa.path_linear_workspace_size(desc, 0) == 256
    q, k, v, do = inputs(dtype, d, batch, hq, hkv, L, seed=30)
    ld = -torch.logspace(-4, 0.5, hkv, device=DEV)
    got = run(q, k, v, do, ld, 0.2)
    for b in range(batch):
        s = slice(b, b + 1)
        want = reference(q[s], k[s], v[s], do[s], ld, 0.2)
        for n in got:
            check(n, got[n][s], *want[n], dtype, terms=L * (hq // hkv) + 2 * d + 64)


@pytest.mark.parametrize("d,hq,hkv,L", [(64, 2, 2, 9000), (128, 2, 1, 6001)])
def test_long_sequences_of_float32(cuda_lib, d, hq, hkv, L):
    q, k, v, do = inputs("fp32", d, 1, hq, hkv, L, seed=31)
    ld = torch.tensor([-0.003, -1e-5][:hkv], device=DEV)
    got, want = run(q, k, v, do, ld, 0.125), reference(q, k, v, do, ld, 0.125)
    for n in got:
        check(n, got[n], *want[n], "fp32", terms=L * (hq // hkv) + 2 * d + 64)
        # (roundings of independent sums: of the d products of a weight, of its tokens', and of the states on the way)
        assert float((got[n].double() - want[n][0]).norm()) <= math.sqrt(2 * (L * (hq // hkv) + d)) * 2.0 ** -24 * float(want[n][0].norm()), n


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [[1], [9, 16], [17], [100, 40, 128], [129], [200, 3]])
def test_states_are_as_exact_as_float32_sums(cuda_lib, dtype, d, n):
    """A state element is a sum of n weighted products: each is rounded twice (2^-24) and so is each sum on the way, independently.
    Two bf16 numbers for a weighted token would leave 2^-17 of it, in the norm 2^-17 / sqrt(3) = 4e-6 of the state; three leave
    2^-25."""
    cache, q, k, v, _ = make(dtype, d, 2, 2, n, seed=32)
    cache.state.zero_()
    ld = torch.tensor([-0.013, -0.0002], device=DEV)
    cache.extend(q, k, v, ld, q_start=starts(n), max_new=max(n))
    cache.check()
    at = 0
    for b, m in enumerate(n):
        kh, vh = (t[at : at + m].permute(1, 0, 2) for t in (k, v))
        want, A = final_state(kh, vh, ld, torch.zeros_like(cache.state[b]))
        err = cache.state[b].double() - want
        assert bool((err.abs() <= (m + 64) * 2.0 ** -24 * A).all())
        assert float(err.norm()) <= math.sqrt(2 * m + 2) * 2.0 ** -24 * float(want.norm()), (m, float(err.norm() / want.norm()))
        at += m


def test_forks_and_resets_of_large_states(cuda_lib):
    """Every slot of a speculative step: states behind 2^31 bytes."""
    from softmax_attention_chunk_gb300.linear import LinearCache

    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    slots, H, d = 1200, 32, 128
    cache = LinearCache(slots, H, d)
    assert cache.state.numel() * 4 > 1 << 31
    cache.state.view(slots, -1)[:] = torch.arange(slots, device=DEV, dtype=torch.float32)[:, None]
    tail = torch.randn(H, d, d, device=DEV)
    cache.state[slots // 2 - 1] = tail
    parents, children = list(range(slots // 2)), list(range(slots - 1, slots // 2 - 1, -1))
    cache.fork(i32(parents), i32(children))
    cache.check()
    for p, c in zip(parents[:-1], children[:-1]):
        if p % 37 == 0 or p > 590:
            assert bool((cache.state[p] == p).all()) and bool((cache.state[c] == p).all())
    assert torch.equal(cache.state[children[-1]], tail) and torch.equal(cache.state[parents[-1]], tail)
    cache.reset(i32(children))
    cache.check()
    assert bool((cache.state[slots // 2 :] == 0).all()) and torch.equal(cache.state[slots // 2 - 1], tail)


def test_a_serving_step_of_many_slots(cuda_lib):
    """Prompts, drafts and single tokens of 96 slots with 32 heads of dim 128: the walk's blocks are several waves too."""
    n = [[300, 1, 5, 0, 130, 17][b % 6] for b in range(96)]
    cache, q, k, v, ld = make("bf16", 128, 32, 16, n, seed=33)
    before = cache.state.clone()
    o = cache.extend(q, k, v, ld, q_start=starts(n), max_new=300, scale=0.2)
    cache.check()
    for b, rows, (want, A), (state, SA) in expect(before, q, k, v, ld, n, 0.2):
        check("o", o[rows], want, A, "bf16", terms=n[b] + 320)
        assert bool(((cache.state[b].double() - state).abs() <= (n[b] + 64) * 2.0 ** -24 * SA + 1e-30).all())
