"""Linear attention over whole sequences (softmax_attention_chunk_gb300.linear.linear_attention): outputs and gradients against
the definition in 64 bits, gradients against differences, and the calls around them."""
import math

import pytest
import torch

from linear_ref import DT, check, reference

pytestmark = pytest.mark.gpu
DEV = "cuda"


def inputs(dtype, d, batch, hq, hkv, L, seed=0):
    g = torch.Generator(device=DEV).manual_seed(100 + seed)
    r = lambda h: torch.randn(batch, h, L, d, generator=g, device=DEV).to(DT[dtype])  # noqa: E731
    return r(hq), r(hkv), r(hkv), r(hq)


def decays(hkv):
    """From forgetting at once to never, and what lies outside the range."""
    some = [-0.3, -0.01, 0.0, -math.inf, -3.0, -1e-4, -30.0, 0.5]
    return torch.tensor([some[i % 8] for i in range(hkv)], device=DEV)


def run(q, k, v, do, ld, scale):
    from softmax_attention_chunk_gb300.linear import linear_attention

    q, k, v = (t.detach().requires_grad_() for t in (q, k, v))
    o = linear_attention(q, k, v, ld, scale=scale)
    return dict(zip(("o", "dq", "dk", "dv"), (o.detach(), *torch.autograd.grad(o, (q, k, v), do))))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch,hq,hkv,L", [(1, 1, 1, 1), (2, 2, 2, 2), (1, 3, 3, 31), (1, 8, 8, 64), (3, 4, 2, 127), (1, 3, 1, 128),
                                            (2, 8, 1, 129), (1, 16, 1, 257), (2, 6, 3, 300), (1, 8, 8, 1000)])
def test_outputs_and_gradients(cuda_lib, dtype, d, batch, hq, hkv, L):
    q, k, v, do = inputs(dtype, d, batch, hq, hkv, L)
    ld = decays(hkv)
    got, want = run(q, k, v, do, ld, 0.3), reference(q, k, v, do, ld, 0.3)
    for n in got:
        check(n, got[n], *want[n], dtype, terms=L * (hq // hkv) + 2 * d + 64)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch,hq,hkv,L", [(1, 1, 1, 1), (1, 2, 1, 3), (2, 2, 2, 17), (1, 3, 1, 64), (1, 4, 4, 128)])
def test_few_short_sequences_are_as_exact_as_their_outputs_type(cuda_lib, d, batch, hq, hkv, L):
    """Weights of two bf16 numbers: 2^-16 of each, beside the output's 2^-8 and float32 sums (of d products in a weight, L of them
    in an output; 64 for the decay and what is multiplied)."""
    q, k, v, do = inputs("bf16", d, batch, hq, hkv, L, seed=11)
    ld, G = torch.full((hkv,), -0.02, device=DEV), hq // hkv
    got = run(q, k, v, do, ld, 0.3)
    gap = torch.arange(L, device=DEV)[:, None] - torch.arange(L, device=DEV)[None, :]
    w = torch.where(gap >= 0, 0.3 * torch.exp(ld[0].double() * gap.clamp(min=0)), 0.0)
    x, y, z, g = (t.double().repeat_interleave(1 if t.shape[1] == hq else G, 1) for t in (q, k, v, do))
    heads = lambda t: t.view(batch, hkv, G, L, d).sum(2)  # noqa: E731
    same = lambda t: t  # noqa: E731
    for name, a, b, c, m, add in (("o", x, y, z, w, same), ("dq", g, z, y, w, same), ("dk", z, g, x, w.mT, heads), ("dv", y, x, g, w.mT, heads)):
        p = a @ b.mT
        want, size = add((p * m) @ c), add((p.abs() * m) @ c.abs())
        sums = add(((a.abs() @ b.abs().mT) * m) @ c.abs()) * (2 * d + 2 * L * G + 64) * 2.0 ** -24
        far = (got[name].double() - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -16 * size + sums) * (1 + 2.0 ** -7)
        assert far.max() <= 0, (name, float(far.max()))


@pytest.mark.parametrize("dtype,d,hq,hkv,L", [("fp32", 64, 1, 1, 3001), ("bf16", 64, 2, 1, 5000), ("bf16", 128, 1, 1, 4097), ("bf16", 128, 8, 2, 2300)])
def test_long_sequences_of_few_heads(cuda_lib, dtype, d, hq, hkv, L):
    """Cut into segments that run side by side."""
    q, k, v, do = inputs(dtype, d, 1, hq, hkv, L, seed=1)
    ld = torch.tensor([-0.002, -0.05][:hkv], device=DEV)
    got, want = run(q, k, v, do, ld, 0.125), reference(q, k, v, do, ld, 0.125)
    for n in got:
        check(n, got[n], *want[n], dtype, terms=L * (hq // hkv) + 2 * d + 64)


def test_gradients_against_differences(cuda_lib):
    """o is linear in q, in k and in v: a difference of any size along one of them is the derivative, up to the sums' rounding."""
    from softmax_attention_chunk_gb300.linear import linear_attention

    q, k, v, do = inputs("fp32", 64, 2, 4, 2, 150, seed=2)
    ld = torch.tensor([-0.1, -0.004], device=DEV)
    got = run(q, k, v, do, ld, 0.2)
    for i, n in enumerate(("dq", "dk", "dv")):
        args = [q, k, v]
        step = torch.randn_like(args[i])
        value = []
        for s in (1.0, -1.0):
            moved = [t + s * step if j == i else t for j, t in enumerate(args)]
            value.append((linear_attention(*moved, ld, scale=0.2).double() * do.double()).sum())
        along = (got[n].double() * step.double()).sum()
        size = (got[n].double() * step.double()).norm() * math.sqrt(got[n].numel())
        assert abs(float((value[0] - value[1]) / 2 - along)) <= 400 * 2.0 ** -24 * float(size), n


def test_strides_broadcasts_and_leaves_that_need_no_gradient(cuda_lib):
    from softmax_attention_chunk_gb300.linear import linear_attention

    q, k, v, do = inputs("bf16", 64, 2, 4, 4, 90, seed=3)
    ld = torch.tensor([-0.5, -0.05, -0.005, -0.0], device=DEV)
    base = run(q, k, v, do, ld, 1.0)
    # tokens before heads in memory, one k for all heads, only k's gradient
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)
    k1 = k[:, :1].clone().requires_grad_()
    o = linear_attention(qt, k1.expand(-1, 4, -1, -1), v, torch.stack([ld, ld], 1)[:, 0])
    full = run(q, k1.detach().expand(-1, 4, -1, -1), v, do, ld, 1.0)
    assert torch.equal(o, full["o"])
    (gk,) = torch.autograd.grad(o, (k1,), do.transpose(1, 2).contiguous().transpose(1, 2))
    assert torch.equal(gk, full["dk"].sum(1, keepdim=True))
    again = run(q, k, v, do, ld, 1.0)
    assert all(torch.equal(base[n], again[n]) for n in base)


def test_empty_sequences_and_batches(cuda_lib):
    for shape in ((2, 3, 0, 64), (0, 3, 5, 64)):
        q = torch.randn(shape, device=DEV)
        got = run(q, q, q, q, torch.zeros(3, device=DEV), 1.0)
        assert all(t.shape == shape for t in got.values())


def test_refusals(cuda_lib):
    from softmax_attention_chunk_gb300.linear import linear_attention

    q, k, v, _ = inputs("bf16", 64, 1, 4, 2, 9)
    ld = torch.zeros(2, device=DEV)
    with pytest.raises(ValueError, match="gradient"):
        linear_attention(q, k, v, ld.clone().requires_grad_())
    for bad in ((q, k, v.float(), ld), (q.half(), k.half(), v.half(), ld), (q, k[:, :, :8], v, ld), (q, k, v, ld[:1]), (q, k, v, ld.double()),
                (q[:, :3], k, v, ld), (q[..., :32], k[..., :32], v[..., :32], ld), (q, k, v, ld.cpu()), (q[0], k[0], v[0], ld)):
        with pytest.raises((ValueError, RuntimeError)):
            linear_attention(*bad)
    o = linear_attention(q.requires_grad_(), k, v, ld)
    (g,) = torch.autograd.grad(o.sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), q)


def test_nan_and_infinity_stay_in_their_sequence_and_head(cuda_lib):
    q, k, v, do = inputs("bf16", 64, 2, 4, 2, 200, seed=4)
    ld = torch.tensor([-0.02, -0.4], device=DEV)
    clean = run(q, k, v, do, ld, 1.0)
    k2, v2 = k.clone(), v.clone()
    k2[1, 1, 50] = math.inf
    v2[1, 1, 60] = math.nan
    got = run(q, k2, v2, do, ld, 1.0)
    for n in ("o", "dq"):
        assert torch.equal(got[n][0], clean[n][0]) and torch.equal(got[n][1, :2], clean[n][1, :2])
    for n in ("dk", "dv"):
        assert torch.equal(got[n][0], clean[n][0]) and torch.equal(got[n][1, 0], clean[n][1, 0])
    assert bool(got["o"][1, 2:, 60:].isnan().any())
    nan_head = run(q, k, v, do, torch.tensor([math.nan, -0.4], device=DEV), 1.0)
    assert bool(nan_head["o"][:, :2].isnan().all()) and torch.equal(nan_head["o"][:, 2:], clean["o"][:, 2:])


def test_another_stream_and_a_captured_step(cuda_lib):
    from softmax_attention_chunk_gb300.linear import linear_attention

    q, k, v, do = inputs("bf16", 128, 1, 4, 4, 700, seed=5)
    ld = torch.tensor([-0.5, -0.05, -0.005, -0.0005], device=DEV)
    want = run(q, k, v, do, ld, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(q, k, v, do, ld, 0.1)
    side.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)
    sq, sk, sv = (torch.zeros_like(t).requires_grad_() for t in (q, k, v))

    def step():
        o = linear_attention(sq, sk, sv, ld, scale=0.1)
        return (o.detach(), *torch.autograd.grad(o, (sq, sk, sv), do))

    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    with torch.no_grad():
        sq.copy_(q), sk.copy_(k), sv.copy_(v)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[n]) for a, n in zip(out, ("o", "dq", "dk", "dv")))


def test_two_calls_at_once(cuda_lib):
    a, b = inputs("bf16", 64, 1, 2, 2, 3000, seed=6), inputs("bf16", 64, 1, 2, 2, 3000, seed=7)
    ld = torch.tensor([-0.02, -0.001], device=DEV)
    want = run(*a, ld, 1.0), run(*b, ld, 1.0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got = []
        for x, st in zip((a, b), s):
            with torch.cuda.stream(st):
                got.append(run(*x, ld, 1.0))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(g[n], w[n]) for n in w)


@pytest.mark.parametrize("dtype,d,hq,hkv,L", [("bf16", 64, 2, 1, 3000), ("bf16", 128, 2, 2, 900), ("fp32", 64, 2, 1, 900)])
@pytest.mark.parametrize("wanted", ["q", "k", "v", "qk", "qv", "kv"])
def test_some_of_the_gradients(cuda_lib, dtype, d, hq, hkv, L, wanted):
    """Those that are wanted alone: dk and dv share their segments' states where both are."""
    from softmax_attention_chunk_gb300.linear import linear_attention

    q, k, v, do = inputs(dtype, d, 1, hq, hkv, L, seed=8)
    ld = torch.tensor([-0.01, -0.2][:hkv], device=DEV)
    want = reference(q, k, v, do, ld, 0.2)
    t = {n: x.clone().requires_grad_(n in wanted) for n, x in zip("qkv", (q, k, v))}
    o = linear_attention(t["q"], t["k"], t["v"], ld, scale=0.2)
    for n, g in zip(wanted, torch.autograd.grad(o, [t[n] for n in wanted], do)):
        check("d" + n, g, *want["d" + n], dtype, terms=L * (hq // hkv) + 2 * d + 64)


def test_status_of_a_workspace(cuda_lib):
    pa = cuda_lib
    q, k, v, _ = inputs("bf16", 64, 2, 4, 4, 500, seed=9)
    ld, o = torch.tensor([-0.1] * 4, device=DEV), torch.empty_like(q)
    desc = pa.path_linear_desc_t(2, 4, 4, 500, 64, pa.PATH_BF16, 1.0)
    n = pa.path_linear_workspace_size(desc, 0)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)  # (whatever lay there)
    assert pa.path_linear_fwd(desc, q.data_ptr(), k.data_ptr(), v.data_ptr(), ld.data_ptr(), o.data_ptr(), ws.data_ptr(), n, pa._stream()) == 0
    assert pa.path_linear_workspace_status(desc, ws.data_ptr(), n, pa._stream()) == (0, 0)


def test_a_parameter_as_decay_without_gradients(cuda_lib):
    from softmax_attention_chunk_gb300.linear import linear_attention

    q, k, v, _ = inputs("bf16", 64, 1, 2, 2, 50, seed=10)
    ld = torch.nn.Parameter(torch.tensor([-0.1, -0.2], device=DEV))
    with torch.no_grad():
        assert torch.equal(linear_attention(q, k, v, ld), linear_attention(q, k, v, ld.detach()))


def test_outputs_beside_others_in_memory(cuda_lib):
    """Nothing is written outside o: its neighbours in one allocation stay."""
    pa = cuda_lib
    for L, d in ((1, 64), (129, 64), (300, 128)):
        q, k, v, _ = inputs("bf16", d, 1, 3, 3, L, seed=11)
        ld = torch.tensor([-0.1, -0.01, -1.0], device=DEV)
        room = torch.full((q.numel() + 4096,), 5.0, dtype=torch.bfloat16, device=DEV)
        desc = pa.path_linear_desc_t(1, 3, 3, L, d, pa.PATH_BF16, 1.0)
        n = pa.path_linear_workspace_size(desc, 0)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        o = room[2048 : 2048 + q.numel()]
        assert pa.path_linear_fwd(desc, q.data_ptr(), k.data_ptr(), v.data_ptr(), ld.data_ptr(), o.data_ptr(), ws.data_ptr(), n, pa._stream()) == 0
        assert bool((room[:2048] == 5.0).all()) and bool((room[2048 + q.numel() :] == 5.0).all())
