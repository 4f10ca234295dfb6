"""Drafts that a paged cache holds under forks, over linear attention's states: the rows given to the parents with update=False read
the parents' states, as a fork's copies would."""
import pytest
import torch

from test_gpu_linear_serving import DEV, make, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,n", [(64, [3, 1, 16, 2]), (128, [5, 0, 40, 7])])
def test_rows_of_children_given_to_their_parents(cuda_lib, d, n):
    B = len(n)
    cache, q, k, v, ld = make("bf16", d, 4, 2, n + [0] * B, seed=40)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    for_children = starts([0] * B + n)
    for_parents = torch.cat([for_children[B:], for_children[-1:].expand(B)])
    before = cache.state.clone()
    got = cache.extend(q, k, v, ld, q_start=for_parents, max_new=max(n), update=False)
    assert torch.equal(cache.state, before)
    cache.fork(i32(list(range(B))), i32(list(range(B, 2 * B))))
    want = cache.extend(q, k, v, ld, q_start=for_children, max_new=max(n), update=False)
    cache.check()
    assert torch.equal(got, want) and torch.equal(cache.state[:B], before[:B])
