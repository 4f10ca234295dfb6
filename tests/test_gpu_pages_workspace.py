"""Workspaces of page calls belong to the call: a captured one's stays with its graph."""
import pytest
import torch

from test_gpu_pages import Model

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def second_handle(c):
    from softmax_attention_chunk_gb300.paged import PagedCache

    return PagedCache.from_tensors(c.k_pool, c.v_pool, c.k_table, c.v_table, c.seq_len, c.k_ref, c.v_ref, extended=c.extended)


@pytest.mark.parametrize("planned", [False, True])
def test_memory_of_a_handle_that_is_gone_is_not_written(cuda_lib, planned):
    from softmax_attention_chunk_gb300.paged import PagedCache

    cache = PagedCache(slots=4, heads=1, head_dim=64, page_size=16, k_pages=30000, table_width=200)
    model = Model(cache)
    n = i32([5, 0, 40, 1])
    call = (lambda c: c.plan(n, 4000)) if planned else (lambda c: c.reserve(n))
    call(cache)
    cache.free(i32([0, 2, 3]))
    handle = second_handle(cache)
    size = handle._pages_bytes
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(handle)
    word = handle.status  # (the one tensor of the handle that the graph may write)
    del handle
    others = [torch.full((size,), 7, dtype=torch.uint8, device=DEV) for _ in range(8)]
    for step in ([5, 0, 40, 1], [300, 17, 0, 0], [2000, 0, 3, 16]):
        n.copy_(i32(step))
        graph.replay()
        model.reserve(step)
        for name in ("k_table", "v_table", "seq_len", "k_ref", "v_ref"):
            assert torch.equal(getattr(cache, name).cpu(), getattr(model, name)), name
    assert all(bool((t == 7).all()) for t in others) and int(word) == 0
