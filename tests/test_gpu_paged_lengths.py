"""Lengths that name more rows than there can be pages for."""
import pytest
import torch

from test_gpu_paged import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,n", [(torch.bfloat16, 1), (torch.bfloat16, 3), (torch.float32, 1)])
@pytest.mark.parametrize("slots", [4, 1030])
def test_more_units_than_there_are_numbers(cuda_lib, dtype, n, slots):
    """Slots of a billion tokens with pages for the newest only, as a window of that length would leave them: their 16-row
    tiles times 16 heads pass 32 bits.  The slots are left out, lengths and pools stay."""
    from softmax_attention_chunk_gb300.paged import PagedCache

    H, P, width = 16, 256, min(1 << 22, (1 << 26) // slots)
    pages = 4 * H
    cache = PagedCache(slots, H, 64, P, pages, table_width=width, dtype=dtype)
    g = torch.Generator(device=DEV).manual_seed(1)
    cache.k_pool.normal_(generator=g)
    cache.v_pool.normal_(generator=g)
    before = cache.k_pool.clone()
    cache.seq_len.fill_(width * P - 8)
    last = torch.arange(slots, device=DEV, dtype=torch.int32) % pages
    cache.k_table[:, -1] = last
    cache.v_table[:, -1] = last
    r = lambda *s: torch.randn(*s, device=DEV, generator=g).to(dtype)  # noqa: E731
    N = slots * n
    out = torch.full((N, H, 64), 3.0, dtype=dtype, device=DEV)
    start = torch.arange(0, N + 1, n, dtype=torch.int32, device=DEV)
    cache.extend(r(N, H, 64), r(N, H, 64), r(N, H, 64), r(N, H, 64), torch.ones(N, H, device=DEV), q_start=start, max_new=n, out=out)
    cache.advance(start)
    with pytest.raises(RuntimeError, match="page-table"):
        cache.check()
    assert (out == 3).all() and torch.equal(cache.k_pool[:, :, : P - 8], before[:, :, : P - 8])  # (rows with tokens)
    assert (cache.seq_len == width * P - 8).all()
