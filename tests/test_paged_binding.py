"""What PagedCache.extend hands to the library, on the CPU: the call is caught before it reaches the GPU."""
import pytest
import torch


@pytest.fixture
def cache(monkeypatch):
    from softmax_attention_chunk_gb300 import build_lib

    build_lib.build()
    from softmax_attention_chunk_gb300 import path_attn as pa
    from softmax_attention_chunk_gb300.paged import PagedCache

    c = PagedCache.__new__(PagedCache)
    c.device, c.slots, c.heads, c.head_dim, c.page_size, c.dtype, c.a_pool = torch.device("cpu"), 3, 2, 64, 16, torch.bfloat16, None
    c.c = pa.path_paged_cache_t(3, 2, 64, 16, 8, 30, 30, pa.PATH_BF16)
    c._plans, c.calls = {}, []
    monkeypatch.setattr(c, "_call", lambda fn, *args: c.calls.append((fn.__name__, args)), raising=False)
    return c


def tokens(n, heads_q=4):
    bf = lambda *s: torch.randn(*s).to(torch.bfloat16)  # noqa: E731
    return bf(n, heads_q, 64), bf(n, 2, 64), bf(n, 2, 64), bf(n, 2, 64), torch.rand(n, 2)


def test_call_with_its_own_workspace(cache):
    cache.extend(*tokens(9), q_start=torch.tensor([0, 4, 8, 9], dtype=torch.int32))
    (name, args), = cache.calls
    assert name == "path_paged_extend" and args[-1] > 0


def test_max_new_below_one_is_refused(cache):
    """No token would be looked at, o left as it was and nothing reported."""
    start = torch.tensor([0, 4, 8, 9], dtype=torch.int32)
    for bad in (0, -1):
        with pytest.raises(ValueError, match="max_new"):
            cache.extend(*tokens(9), q_start=start, max_new=bad)
    with pytest.raises(ValueError, match="max_new"):
        cache.extend(*tokens(3), max_new=0)
    assert cache.calls == []
    cache.extend(*tokens(0), q_start=torch.zeros(4, dtype=torch.int32))  # no tokens: nothing to do
    assert cache.calls == []


@pytest.mark.parametrize("ws", [lambda n: torch.empty(n, dtype=torch.uint8, device="meta"), lambda n: torch.empty(2 * n, dtype=torch.uint8)[::2],
                                lambda n: torch.empty(n, dtype=torch.float32), lambda n: torch.empty(n - 1, dtype=torch.uint8)])
def test_workspaces_that_are_none(cache, ws):
    """Another device, gaps, another type (whose elements are not bytes), too few bytes."""
    start = torch.tensor([0, 4, 8, 9], dtype=torch.int32)
    t = tokens(9)
    cache.extend(*t, q_start=start)
    n = cache.calls.pop()[1][-1]
    with pytest.raises(ValueError, match="ws"):
        cache.extend(*t, q_start=start, ws=ws(n))
    assert cache.calls == []
    cache.extend(*t, q_start=start, ws=torch.empty(n + 5, dtype=torch.uint8))
    assert cache.calls.pop()[1][-1] == n + 5


def test_tensors_off_a_16_byte_boundary(cache):
    """beta and log_f of a part of a packed batch may begin anywhere: the library gets aligned copies."""
    import ctypes

    cache.a_pool = torch.zeros(1)  # with a gate
    q, k, v, w, _ = tokens(9)
    start = torch.tensor([0, 4, 8, 9], dtype=torch.int32)
    beta, log_f = torch.rand(20, 2), -torch.rand(20, 2)
    kept = []
    cache._call = lambda fn, *a: (kept.append([ctypes.string_at(x, 72) for x in a[6:8]]), cache.calls.append((fn.__name__, a)))
    for s in (0, 1, 3, 11):
        cache.extend(q, k, v, w, beta[s : s + 9], log_f=log_f[s : s + 9], q_start=start)
        a = cache.calls.pop()[1]
        assert a[6] % 16 == 0 and a[7] % 16 == 0
        assert kept.pop() == [x[s : s + 9].contiguous().numpy().tobytes() for x in (beta, log_f)]
