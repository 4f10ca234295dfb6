"""Host-side checks of linear attention, draft verification and step plans: argument errors of the C ABI (nothing is launched:
the fake pointers are never used) and the bindings' refusals."""
import pytest
import torch

from test_paged_host import FAKE, cache, pa  # noqa: F401  (pa: the fixture)


def ldesc(pa, **kw):
    d = dict(batch=2, heads_q=4, heads=2, seqlen=100, head_dim=64, dtype=pa.PATH_BF16, scale=1.0)
    d.update(kw)
    return pa.path_linear_desc_t(**d)


def lcache(pa, **kw):
    d = dict(slots=3, heads=2, head_dim=64, dtype=pa.PATH_BF16, state=FAKE, status=FAKE)
    d.update(kw)
    return pa.path_linear_cache_t(**d)


def lstep(pa, **kw):
    d = dict(heads_q=4, total_tokens=9, max_new=5, scale=1.0, update=1)
    d.update(kw)
    return pa.path_linear_step_t(**d)


def fwd(pa, d, nbytes=None, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ld=FAKE, o=FAKE, ws=FAKE)
    a.update(kw)
    n = pa.path_linear_workspace_size(d, 0) if nbytes is None else nbytes
    return pa.path_linear_fwd(d, a["q"], a["k"], a["v"], a["ld"], a["o"], a["ws"], n, None)


def bwd(pa, d, nbytes=None, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ld=FAKE, do=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, ws=FAKE)
    a.update(kw)
    n = pa.path_linear_workspace_size(d, 1) if nbytes is None else nbytes
    return pa.path_linear_bwd(d, a["q"], a["k"], a["v"], a["ld"], a["do"], a["dq"], a["dk"], a["dv"], a["ws"], n, None)


def extend(pa, c, s, nbytes=None, **kw):
    a = dict(q_start=FAKE, q=FAKE, k=FAKE, v=FAKE, ld=FAKE, o=FAKE, ws=FAKE)
    a.update(kw)
    n = pa.path_linear_extend_workspace_size(c, s) if nbytes is None else nbytes
    return pa.path_linear_extend(c, s, a["q_start"], a["q"], a["k"], a["v"], a["ld"], a["o"], a["ws"], n, None)


@pytest.mark.parametrize("field,value,want", [("batch", 0, 1), ("heads_q", 3, 1), ("heads_q", 0, 1), ("heads", 0, 1), ("seqlen", 0, 1), ("head_dim", 0, 1),
                                              ("dtype", 3, 1), ("scale", float("inf"), 1), ("scale", float("nan"), 1), ("head_dim", 96, 2),
                                              ("heads_q", 34, 2), ("batch", 70000, 2), ("seqlen", 1 << 30, 2)])
def test_descriptors(pa, field, value, want):
    d = ldesc(pa, **{field: value})
    assert pa.path_linear_workspace_size(d, 0) == pa.path_linear_workspace_size(d, 1) == 0
    assert fwd(pa, d, 1 << 40) == want and bwd(pa, d, 1 << 40) == want
    assert pa.path_linear_workspace_status(d, FAKE, 256, None)[0] == want


@pytest.mark.parametrize("name", ["q", "k", "v", "ld", "o", "ws"])
def test_forward_pointers(pa, name):
    for bad in (None, FAKE + 2):
        assert fwd(pa, ldesc(pa), **{name: bad}) == 1
    assert fwd(pa, ldesc(pa), nbytes=100) == 3


@pytest.mark.parametrize("name", ["q", "k", "v", "ld", "do", "ws", "dq", "dk", "dv"])
def test_backward_pointers(pa, name):
    for bad in (None, FAKE + 2):
        if bad or name not in ("dq", "dk", "dv"):  # (a gradient may be left out, not all of them)
            assert bwd(pa, ldesc(pa), **{name: bad}) == 1
    assert bwd(pa, ldesc(pa), dq=None, dk=None, dv=None) == 1
    assert bwd(pa, ldesc(pa), nbytes=100) == 3


@pytest.mark.parametrize("field,value,want", [("slots", 0, 1), ("heads", 0, 1), ("head_dim", 0, 1), ("dtype", 7, 1), ("head_dim", 32, 2),
                                              ("slots", 70000, 2), ("heads", 2000, 2)])
def test_caches(pa, field, value, want):
    c = lcache(pa, **{field: value})
    s = lstep(pa, heads_q=max(1, c.heads) * 2)
    assert pa.path_linear_extend_workspace_size(c, s) == 0
    assert extend(pa, c, s, 1 << 40) == want
    assert pa.path_linear_fork(c, FAKE, FAKE, 1, None) == want and pa.path_linear_status(c, None)[0] == want


@pytest.mark.parametrize("field,value,want", [("heads_q", 3, 1), ("heads_q", 64, 2), ("total_tokens", -1, 1), ("max_new", -1, 1), ("scale", float("nan"), 1),
                                              ("total_tokens", (1 << 22) + 1, 2)])
def test_steps(pa, field, value, want):
    s = lstep(pa, **{field: value})
    assert pa.path_linear_extend_workspace_size(lcache(pa), s) == 0
    assert extend(pa, lcache(pa), s, 1 << 40) == want


def test_extend_pointers(pa):
    many = lstep(pa, total_tokens=90, max_new=50)
    for name in ("q", "k", "v", "ld", "o", "ws"):
        for bad in (None, FAKE + 2):
            assert extend(pa, lcache(pa), many, **{name: bad}) == 1, name
            if name != "ws":
                assert extend(pa, lcache(pa), lstep(pa), **{name: bad}) == 1, name
    for name in ("state", "status"):
        for bad in (None, FAKE + 2):
            c = lcache(pa, **{name: bad})
            assert extend(pa, c, lstep(pa)) == 1 and pa.path_linear_status(c, None)[0] == 1
            assert pa.path_linear_fork(c, None, FAKE, 1, None) == 1
    assert extend(pa, lcache(pa), many, nbytes=8) == 3
    assert extend(pa, lcache(pa), lstep(pa), q_start=FAKE + 1) == 1
    assert extend(pa, lcache(pa), lstep(pa), q_start=None) == 1  # nine tokens for three slots
    assert extend(pa, lcache(pa), lstep(pa, total_tokens=3, max_new=0), q_start=None) == 1
    assert extend(pa, lcache(pa), lstep(pa, total_tokens=0)) == 0 and extend(pa, lcache(pa), lstep(pa, max_new=0)) == 0
    c = lcache(pa)
    assert pa.path_linear_fork(c, None, FAKE, 4, None) == 1 and pa.path_linear_fork(c, None, FAKE, -1, None) == 1
    assert pa.path_linear_fork(c, None, None, 1, None) == 1 and pa.path_linear_fork(c, FAKE + 1, FAKE, 1, None) == 1
    assert pa.path_linear_fork(c, FAKE, FAKE, 0, None) == 0


def test_workspaces(pa):
    """Segments' states, a few times what the sequences' own take; nothing where heads alone fill the GPU."""
    assert pa.path_linear_workspace_size(ldesc(pa, batch=32, heads_q=32, heads=32, seqlen=4096), 1) <= 4096
    n = pa.path_linear_workspace_size(ldesc(pa, batch=1, heads_q=8, heads=8, seqlen=1 << 20, head_dim=128), 1)
    assert 256 < n < 1 << 28
    c = lcache(pa, slots=4096, heads=8, head_dim=128)
    n = pa.path_linear_extend_workspace_size(c, lstep(pa, heads_q=32, total_tokens=1 << 16, max_new=1 << 16))
    assert 256 <= n < 1 << 31
    assert pa.path_linear_extend_workspace_size(c, lstep(pa, heads_q=32, total_tokens=4096, max_new=16)) == 256


def verify(pa, status=FAKE, **kw):
    d = dict(slots=3, total_tokens=9, max_new=4, vocab=100, dtype=pa.PATH_FP32, target_stride=100, draft_stride=100)
    a = dict(q_start=FAKE, tokens=FAKE, uniform=FAKE, target=FAKE, draft=FAKE, keep=FAKE, next=FAKE)
    for k, v in kw.items():
        (d if k in d else a)[k] = v
    return pa.path_draft_verify(pa.path_verify_desc_t(**d), *a.values(), status, None)


@pytest.mark.parametrize("kw,want", [(dict(slots=0), 1), (dict(total_tokens=-1), 1), (dict(max_new=-1), 1), (dict(vocab=0), 1), (dict(dtype=2), 1),
                                     (dict(target_stride=99), 1), (dict(draft_stride=50), 1), (dict(slots=1 << 17), 2), (dict(vocab=(1 << 20) + 1, target_stride=1 << 21, draft_stride=1 << 21), 2)]
                         + [({n: bad}, 1) for n in ("q_start", "tokens", "uniform", "target", "keep", "next", "status") for bad in (None, FAKE + 1)]
                         + [(dict(draft=FAKE + 2), 1)])
def test_verification(pa, kw, want):
    assert verify(pa, **kw) == want


def test_plans(pa):
    n = pa.path_pages_workspace_size(cache(pa))

    def plan(tokens=9, nbytes=n, **kw):
        a = dict(n_new=FAKE, from_start=FAKE, q_start=FAKE, slot=FAKE, position=FAKE, k_row=FAKE, v_row=FAKE, source=FAKE, ws=FAKE)
        a.update(kw)
        return pa.path_pages_plan(cache(pa), a["n_new"], a["from_start"], tokens, a["q_start"], a["slot"], a["position"], a["k_row"], a["v_row"], a["source"],
                                  a["ws"], nbytes, None)

    for name in ("from_start", "q_start", "slot", "position", "k_row", "v_row", "source", "ws"):
        for bad in (None, FAKE + 1):
            assert plan(**{name: bad}) == 1, name
    assert plan(n_new=FAKE + 2) == 1 and plan(tokens=-1) == 1 and plan(tokens=(1 << 22) + 1) == 2 and plan(nbytes=n - 1) == 3


def test_linear_cache_refusals(pa):
    from softmax_attention_chunk_gb300.linear import LinearCache

    for kw in (dict(slots=0), dict(heads=0), dict(head_dim=96), dict(dtype=torch.float16)):
        with pytest.raises(ValueError):
            LinearCache(**{**dict(slots=2, heads=2, head_dim=64, device="cpu"), **kw})
    with pytest.raises(ValueError):  # (not on a GPU)
        LinearCache.from_tensors(torch.zeros(2, 2, 64, 64))
    with pytest.raises(ValueError):
        LinearCache.from_tensors(torch.zeros(2, 2, 64, 128))
