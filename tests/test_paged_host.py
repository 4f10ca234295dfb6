"""Host-side checks of paged serving that need no GPU: argument errors of the C ABI (nothing is launched: the fake
pointers are never used), the index logic that the kernels share with the host, and the binding's refusals."""
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20


@pytest.fixture(scope="module")
def pa():
    from softmax_attention_chunk_gb300 import build_lib

    build_lib.build()
    from softmax_attention_chunk_gb300 import path_attn

    return path_attn


def cache(pa, **kw):
    d = dict(slots=3, heads=2, head_dim=64, page_size=16, table_width=8, k_pages=30, v_pages=20, cache_dtype=pa.PATH_BF16,
             k_pool=FAKE, v_pool=FAKE, a_pool=None, k_table=FAKE, v_table=FAKE, seq_len=FAKE, k_ref=FAKE, v_ref=FAKE,
             status=FAKE)
    d.update(kw)
    return pa.path_paged_cache_t(**d)


def desc(pa, **kw):
    d = dict(heads_q=4, total_tokens=9, max_new=5, scale=1.0, window=0, sinks=0)
    d.update(kw)
    return pa.path_paged_desc_t(**d)


def extend(pa, c, d, nbytes=None, **kw):
    a = dict(q_start=FAKE, q=FAKE, k=FAKE, v=FAKE, w=FAKE, beta=FAKE, log_f=None, o=FAKE, ws=FAKE)
    a.update(kw)
    n = pa.path_paged_workspace_size(c, d) if nbytes is None else nbytes
    return pa.path_paged_extend(c, d, a["q_start"], a["q"], a["k"], a["v"], a["w"], a["beta"], a["log_f"], a["o"], a["ws"], n,
                                None)


@pytest.mark.parametrize("field,value,want", [("slots", 0, 1), ("heads", -1, 1), ("page_size", 0, 1), ("table_width", 0, 1),
                                              ("k_pages", 0, 1), ("v_pages", -3, 1), ("cache_dtype", 5, 1), ("head_dim", 0, 1),
                                              ("head_dim", 96, 2), ("page_size", 48, 2), ("page_size", 8, 2),
                                              ("slots", 70000, 2), ("table_width", 1 << 27, 2), ("k_pages", 1 << 30, 2),
                                              ("heads", 2000, 2)])
def test_cache_sizes(pa, field, value, want):
    c = cache(pa, **{field: value})
    assert pa.path_pages_workspace_size(c) == 0
    assert pa.path_paged_workspace_size(c, desc(pa, heads_q=c.heads if c.heads > 0 else 1)) == 0
    assert pa.path_pages_compact(c, FAKE, 1 << 40, None) == want
    assert pa.path_paged_advance(c, None, None) == want
    assert pa.path_paged_status(c, None)[0] == want
    assert extend(pa, c, desc(pa), nbytes=1 << 40) == want


@pytest.mark.parametrize("field", ["k_pool", "v_pool", "k_table", "v_table", "seq_len", "k_ref", "v_ref", "status"])
def test_cache_pointers(pa, field):
    n = pa.path_pages_workspace_size(cache(pa))
    for bad in (None, FAKE + 2):
        c = cache(pa, **{field: bad})
        assert pa.path_pages_compact(c, FAKE, n, None) == 1
        assert extend(pa, c, desc(pa), nbytes=1 << 40) == 1
    assert pa.path_pages_compact(cache(pa, a_pool=FAKE + 4), FAKE, n, None) == 1


def test_extend_arguments(pa):
    c, d = cache(pa), desc(pa)
    n = pa.path_paged_workspace_size(c, d)
    assert n > 0
    assert extend(pa, c, d, nbytes=n - 1) == 3
    for f in ("q", "k", "v", "w", "beta", "o"):
        assert extend(pa, c, d, **{f: None}) == 1 and extend(pa, c, d, **{f: FAKE + 8}) == 1
    assert extend(pa, c, d, ws=FAKE + 16) == 1 and extend(pa, c, d, q_start=FAKE + 2) == 1
    assert extend(pa, c, d, log_f=FAKE) == 1                       # a forget gate without its cache
    assert extend(pa, cache(pa, a_pool=FAKE), d) == 1              # and the other way round
    assert extend(pa, cache(pa, a_pool=FAKE), d, log_f=FAKE + 4) == 1
    assert extend(pa, c, d, q_start=None) == 1                     # 9 tokens for 3 slots
    assert extend(pa, c, desc(pa, total_tokens=3, max_new=0), q_start=None) == 1
    assert extend(pa, c, desc(pa, heads_q=3), nbytes=n) == 1       # not a multiple of the key heads
    assert extend(pa, c, desc(pa, heads_q=34), nbytes=n) == 2      # 17 query heads per key head
    assert extend(pa, c, desc(pa, scale=float("inf")), nbytes=n) == 1
    assert extend(pa, c, desc(pa, window=-1), nbytes=n) == 1 and extend(pa, c, desc(pa, sinks=-1), nbytes=n) == 1
    assert extend(pa, c, desc(pa, total_tokens=-1), nbytes=n) == 1
    assert extend(pa, c, desc(pa, total_tokens=1 << 23), nbytes=n) == 2
    assert extend(pa, c, desc(pa, total_tokens=0)) == 0            # nothing to do
    assert extend(pa, c, desc(pa, max_new=0)) == 0
    assert pa._lib.path_paged_workspace_size(None, None) == 0
    # a workspace for the largest call of a shape holds a smaller one
    assert pa.path_paged_workspace_size(c, desc(pa, total_tokens=500, max_new=500)) >= n


def test_page_call_arguments(pa):
    c = cache(pa)
    n = pa.path_pages_workspace_size(c)
    assert n > 0
    for call in (lambda ws, k: pa.path_pages_reserve(c, None, ws, k, None), lambda ws, k: pa.path_pages_compact(c, ws, k, None),
                 lambda ws, k: pa.path_pages_fork(c, FAKE, FAKE, 1, ws, k, None),
                 lambda ws, k: pa.path_pages_free(c, FAKE, 1, ws, k, None),
                 lambda ws, k: pa.path_pages_trim(c, 4, 0, ws, k, None)):
        assert call(FAKE, n - 1) == 3 and call(None, n) == 1 and call(FAKE + 16, n) == 1
    assert pa.path_pages_reserve(c, FAKE + 1, FAKE, n, None) == 1
    assert pa.path_pages_fork(c, None, FAKE, 1, FAKE, n, None) == 1
    assert pa.path_pages_fork(c, FAKE, FAKE, 4, FAKE, n, None) == 1     # more children than slots
    assert pa.path_pages_fork(c, FAKE, FAKE, -1, FAKE, n, None) == 1
    assert pa.path_pages_fork(c, FAKE, FAKE, 0, FAKE, n, None) == 0
    assert pa.path_pages_free(c, FAKE, 4, FAKE, n, None) == 1 and pa.path_pages_free(c, FAKE, 0, FAKE, n, None) == 0
    assert pa.path_pages_trim(c, 0, 0, FAKE, n, None) == 1 and pa.path_pages_trim(c, 4, -1, FAKE, n, None) == 1
    assert pa.path_paged_advance(c, FAKE + 2, None) == 1


def test_binding_refuses_cpu_tensors_and_bad_sizes(pa):
    from softmax_attention_chunk_gb300.paged import PagedCache

    with pytest.raises(ValueError):
        PagedCache(2, 2, 64, 16, 8, device="cpu")  # tensors of a cache lie on the GPU
    for kw in (dict(slots=0), dict(head_dim=96), dict(page_size=24), dict(k_pages=-1), dict(dtype=torch.float16)):
        with pytest.raises(ValueError):
            PagedCache(**{**dict(slots=2, heads=2, head_dim=64, page_size=16, k_pages=8, device="cpu"), **kw})
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        PagedCache.from_tensors(torch.zeros(4, 2, 16), torch.zeros(4, 2, 16, 64), z, z, z, z, z)


def test_index_logic_on_the_host(tmp_path):
    """Live tiles, spans of new tokens and page rows, bad pages and bad rows among them, as the kernels compute them."""
    exe = tmp_path / "paged_host_check"
    nvcc = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
    r = subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-o", str(exe),
                        os.path.join(ROOT, "tests", "paged_host_check.cu")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.stdout.strip() == "ok", out.stdout
