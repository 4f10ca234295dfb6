"""What the serving calls hand to the library, on the CPU: the call is caught before it reaches the GPU.  Descriptors are kept by
the numbers of a call, never by the objects that hold them."""
import pytest
import torch

from test_paged_binding import cache, tokens  # noqa: F401  (cache: the fixture)

STARTS = torch.tensor([0, 4, 8, 9], dtype=torch.int32)


@pytest.fixture
def linear(monkeypatch):
    from softmax_attention_chunk_gb300 import build_lib

    build_lib.build()
    from softmax_attention_chunk_gb300 import path_attn as pa
    from softmax_attention_chunk_gb300.linear import LinearCache

    c = LinearCache.__new__(LinearCache)
    c.device, c._index, c.slots, c.heads, c.head_dim, c.dtype = torch.device("cpu"), -1, 3, 2, 64, torch.bfloat16
    c.c, c._plans, c.steps = pa.path_linear_cache_t(3, 2, 64, pa.PATH_BF16), {}, []

    def call(fn, step, *args):
        s = step._obj
        c.steps.append((s.heads_q, s.total_tokens, s.max_new, round(s.scale, 6), s.update))

    monkeypatch.setattr(c, "_call", call, raising=False)
    return c


def test_numbers_that_change_in_their_tensor(linear):
    q, k, v, _, _ = tokens(9)
    ld = torch.zeros(2)
    scale, most, update = torch.tensor(0.5), torch.tensor(4), torch.tensor(True)
    linear.extend(q, k, v, ld, q_start=STARTS, max_new=most, scale=scale, update=update)
    scale.fill_(0.25), most.fill_(9), update.fill_(False)
    linear.extend(q, k, v, ld, q_start=STARTS, max_new=most, scale=scale, update=update)
    linear.extend(q, k, v, ld, q_start=STARTS, max_new=9, scale=0.25, update=False)
    assert linear.steps == [(4, 9, 4, 0.5, 1), (4, 9, 9, 0.25, 0), (4, 9, 9, 0.25, 0)] and len(linear._plans) == 2


def test_numbers_of_attention_that_change_in_their_tensor(cache):  # noqa: F811
    most, scale, window, sinks, multi = torch.tensor(4), torch.tensor(0.5), torch.tensor(8), torch.tensor(1), torch.tensor(1)
    t = tokens(9)
    for _ in range(2):
        cache.extend(*t, q_start=STARTS, max_new=most, scale=scale, window=window, sinks=sinks, max_multi=multi)
        most.fill_(9), scale.fill_(0.25), window.fill_(16), sinks.fill_(2), multi.fill_(3)
    got = [(d.max_new, d.scale, d.window, d.sinks, d.max_multi) for d in (a[0] for _, a in cache.calls)]
    assert got == [(4, 0.5, 8, 1, 1), (9, 0.25, 16, 2, 3)]


def test_numbers_of_verification_that_change_in_their_tensor(cache):  # noqa: F811
    cache._verifications, cache.status, got = {}, torch.zeros(1, dtype=torch.int32), []
    cache._library = lambda fn, desc, *args: got.append(desc._obj.max_new)
    target, most = torch.rand(9, 50), torch.tensor(4)
    args = (target, torch.zeros(9, dtype=torch.int32), torch.rand(9))
    cache.verify(*args, q_start=STARTS, max_new=most)
    most.fill_(9)
    cache.verify(*args, q_start=STARTS, max_new=most)
    cache.verify(*args, q_start=STARTS)
    assert got == [4, 9, 9]
