"""Verification where nothing is left of the target: the row is read a second time, for itself."""
import pytest
import torch

from test_gpu_verify import case, i32, make_cache, reference, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V,pad", [(64, 0), (513, 3), (4096, 0), (33000, 8), (131072, 0), (1 << 20, 0)])
def test_target_below_the_draft_everywhere(cuda_lib, dtype, V, pad):
    """draft = 2 target: a draft is kept with u < 1/2, and of the first that is not, max(0, target - draft) is 0 throughout.  Slots
    of one kind beside slots of the other, a few to many loads of a warp, the same answer every time."""
    n = [3] * (8 if V > 100000 else 40)
    target, _, tokens, uniform = case(dtype, V, n, seed=V + pad, pad=pad)
    draft = torch.full_like(target, float("nan"))
    draft[1:] = 2 * target[:-1]
    draft[4::9] = target[4::9]  # (some have a residual)
    uniform[1::3] = torch.where(uniform[1::3] < 0.3, uniform[1::3], 0.5 + uniform[1::3] / 2)
    cache, s = make_cache(len(n)), starts(n)
    want = reference(target, draft, tokens, uniform, s)
    assert 1 in want[0] and max(want[0]) > 1
    for _ in range(10):
        keep, after = cache.verify(target, tokens, uniform, draft=draft, q_start=i32(s))
        assert (keep.tolist(), after.tolist()) == want
    cache.check()
