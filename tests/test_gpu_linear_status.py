"""Failure path of linear attention's tensor-core kernels, made to run without a fault: PATH_ATTN_DEBUG_STALL_NS has every block
wait on a barrier that nothing arrives at, for a short limit and before any copy or product.  The call that was asked to look
raises, forward and backward; the cache's status has the code; the next call is right."""
import pytest
import torch

from linear_ref import check, reference
from test_gpu_linear import inputs, run
from test_gpu_linear_serving import DEV, make, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,hq,hkv,L", [(64, 2, 2, 300), (64, 2, 1, 3000), (128, 4, 2, 700)])
def test_a_training_call_that_gives_up(cuda_lib, monkeypatch, d, hq, hkv, L):
    from softmax_attention_chunk_gb300.linear import linear_attention

    q, k, v, do = inputs("bf16", d, 1, hq, hkv, L, seed=12)
    ld = torch.tensor([-0.01, -0.2][:hkv], device=DEV)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    o = linear_attention(*leaves, ld, scale=0.3, check=True)
    monkeypatch.setenv("PATH_ATTN_DEBUG_STALL_NS", "1000000")
    with pytest.raises(RuntimeError, match="path_linear_fwd.*code 99"):
        linear_attention(q, k, v, ld, check=True)
    with pytest.raises(RuntimeError, match="path_linear_bwd.*code 99"):
        torch.autograd.grad(o, leaves, do, retain_graph=True)
    monkeypatch.delenv("PATH_ATTN_DEBUG_STALL_NS")
    want = reference(q, k, v, do, ld, 0.3)
    got = dict(zip(("o", "dq", "dk", "dv"), (o.detach(), *torch.autograd.grad(o, leaves, do))))
    same = run(q, k, v, do, ld, 0.3)
    for n in want:
        check(n, got[n], *want[n], "bf16", terms=L * (hq // hkv) + 2 * d + 64)
        assert torch.equal(got[n], same[n])


@pytest.mark.parametrize("d,n", [(64, [200, 1, 30]), (128, [3000, 2, 0])])
def test_a_cache_call_that_gives_up(cuda_lib, monkeypatch, d, n):
    cache, q, k, v, ld = make("bf16", d, 4, 2, n, seed=21)
    s = starts(n)
    want = cache.extend(q, k, v, ld, q_start=s, max_new=max(n), update=False)
    cache.check()
    monkeypatch.setenv("PATH_ATTN_DEBUG_STALL_NS", "1000000")
    cache.extend(q, k, v, ld, q_start=s, max_new=max(n), update=False)
    with pytest.raises(RuntimeError, match="bounded wait gave up .code 99."):
        cache.check()
    monkeypatch.delenv("PATH_ATTN_DEBUG_STALL_NS")
    assert torch.equal(cache.extend(q, k, v, ld, q_start=s, max_new=max(n), update=False), want)
    cache.check()


def test_check_of_the_other_forms(cuda_lib):
    """float32 kernels have no such waits; nothing is launched for nothing; a capture cannot wait for the device."""
    from softmax_attention_chunk_gb300.linear import linear_attention

    q, k, v, do = inputs("fp32", 64, 1, 2, 2, 100, seed=13)
    ld = torch.tensor([-0.01, -0.2], device=DEV)
    assert torch.equal(linear_attention(q, k, v, ld, check=True), linear_attention(q, k, v, ld))
    e = q[:, :, :0]
    assert linear_attention(e, e, e, ld, check=True).shape == e.shape
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="captur"):
            linear_attention(q, k, v, ld, check=True)
        o = linear_attention(q, k, v, ld)
    graph.replay()
    assert torch.equal(o, linear_attention(q, k, v, ld))
