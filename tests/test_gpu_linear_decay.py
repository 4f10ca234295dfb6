"""States of linear attention over many calls with a decay close to 1, against the definition in 64 bits.

A decay is applied once per token (or per chunk) for as long as a sequence lives.  One float32 number for it would be off by up to
2^-25 of the state, the same way every time; with its rounding kept, a step leaves the roundings of its float32 sums alone: 2^-24 of
the state each at most, which the decay takes away again.  Where they are independent from step to step, the norm of all errors is
below sqrt(roundings not forgotten) 2^-24 of the largest state on the way (the last: it grows), beside 2^-22 for the decay's own
value over as many tokens as it remembers.

Tokens that repeat: where a token is added to a state that is a multiple of its last place (float32 chunks add token by token, and a
decay of exactly 1 changes nothing in between), what rounding takes depends on the token's own low bits alone, and is the same at
each repetition.  The errors within a period are then independent, and those of all periods are as many times as large."""
import math

import pytest
import torch

from linear_ref import DT, final_state

pytestmark = pytest.mark.gpu
DEV = "cuda"


def remembered(l, steps):
    """Sum of exp(l i) over i < steps."""
    return (1 - math.exp(l * steps)) / (1 - math.exp(l)) if l else steps


def bound(l, tokens, per_token):
    return math.sqrt(remembered(2 * l, tokens) * per_token) * 2.0 ** -24 + min(1.0, abs(l) * tokens) * 2.0 ** -22


def bound_of_repeated(l, tokens, per_token, period):
    return remembered(l * period, math.ceil(tokens / period)) * math.sqrt(period * per_token) * 2.0 ** -24


def run(dtype, d, calls, m, ld, slots=1, distinct=64):
    """Error of the states after `calls` calls of m tokens for each slot, in the norm, for each head.  The tokens repeat every
    `distinct` calls (None: never)."""
    from softmax_attention_chunk_gb300.linear import LinearCache

    g = torch.Generator(device=DEV).manual_seed(300 + m)
    ld = torch.tensor(ld, device=DEV)
    H, part = len(ld), distinct or 16

    def make():
        k, v = (torch.randn(part, slots, H, m, d, generator=g, device=DEV).to(DT[dtype]) for _ in range(2))
        pack = lambda t: t.permute(0, 1, 3, 2, 4).reshape(part, slots * m, H, d).contiguous()  # noqa: E731
        return k, v, pack(k), pack(v)

    tokens = make()
    q = torch.zeros_like(tokens[2][0])
    cache = LinearCache(slots, H, d, dtype=DT[dtype])
    cache.state.copy_(3.0 * torch.randn(cache.state.shape, generator=g, device=DEV))
    want, start = cache.state.double(), torch.arange(0, slots * m + 1, m, dtype=torch.int32, device=DEV)
    for c in range(0, calls, part):
        n = min(part, calls - c)
        k, v, kp, vp = tokens if distinct or c == 0 else make()
        for i in range(n):
            cache.extend(q, kp[i], vp[i], ld, q_start=start, max_new=m)
        seq = lambda t: t[:n].permute(1, 2, 0, 3, 4).reshape(slots, H, n * m, d)  # noqa: E731
        want = final_state(seq(k), seq(v), ld[None].expand(slots, H), want)[0]
    cache.check()
    return [float((cache.state[:, h].double() - want[:, h]).norm() / want[:, h].norm()) for h in range(H)]


@pytest.mark.parametrize("dtype,d", [("fp32", 64), ("bf16", 128)])
@pytest.mark.parametrize("m,calls", [(1, 20000), (16, 1500), (5, 4000)])
def test_single_and_draft_tokens(cuda_lib, dtype, d, m, calls):
    ld = [-1e-5, -1e-4, -3e-3, 0.0]
    for l, err in zip(ld, run(dtype, d, calls, m, ld)):
        # (S g + k v is rounded once: S g has other low bits at each repetition, S has not)
        assert err <= (bound(l, calls * m, 2) if l else bound_of_repeated(l, calls * m, 2, 64 * m)), (l, err)


@pytest.mark.parametrize("dtype,d", [("fp32", 64), ("fp32", 128), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("slots,m,calls", [(2, 128, 8000), (1, 4096, 256)])
def test_prompts_in_parts(cuda_lib, dtype, d, slots, m, calls):
    """Chunks one behind the other, and segments side by side.  float32 adds a chunk's products to the state one by one (a rounding
    each), bf16 a chunk's sum of 128."""
    ld = [-2e-6, 0.0]
    for l, err in zip(ld, run(dtype, d, calls, m, ld, slots, distinct=4)):
        each = 1 if dtype == "fp32" else 2 / 128
        same = bound_of_repeated(l, calls * m, each, 4 * m) if dtype == "fp32" or l == 0 else 0
        assert err <= bound(l, calls * m, 1 / 64 if same else each) + same, (l, err)


@pytest.mark.parametrize("dtype,d", [("fp32", 64), ("fp32", 128), ("bf16", 64)])
@pytest.mark.parametrize("slots,m,calls", [(2, 128, 8000), (1, 4096, 256)])
def test_prompts_in_parts_of_new_tokens(cuda_lib, dtype, d, slots, m, calls):
    ld = [-2e-6, -1.8e-6]
    for l, err in zip(ld, run(dtype, d, calls, m, ld, slots, distinct=None)):
        assert err <= bound(l, calls * m, 1 + 1 / 64 if dtype == "fp32" else 2 / 128), (l, err)
