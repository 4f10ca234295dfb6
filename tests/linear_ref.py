"""Linear attention in 64 bits from its definition, for the tests, and the tolerances of its kernels.

U is the largest error of one rounding, relative to the value.  bf16 kernels round, beside the output itself, either a
weighted product x_i . y_j or an element of the state before it meets its partner, and the weighted token that goes into the
state: three roundings on any path from the inputs to an output.  Each error is at most U times the sum of the magnitudes that
it passes through, so an element is off by at most U |o| + 2 U A, with A the same sums over magnitudes; and because the
roundings are independent and their errors spread over +- U, the norm of all errors is below U sqrt(3) / sqrt(3) = U times
the norm of the outputs.  Sums in float32 add one rounding per term: below (terms) 2^-24 A.
The state itself is kept in float32; bf16 kernels add its weighted tokens as two bf16 numbers, what is left is U^2.
"""
import torch

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def decay_log(log_decay):
    return torch.where(log_decay > 0, 0.0, torch.where(log_decay < -1e4, -1e4, log_decay.double()))


def walk(x, y, z, log_decay, scale, reverse=False, state=None):
    """(o, A) of x [..., L, d], y, z [..., L, d] with log_decay of their leading shape: every pair of tokens, in 64 bits."""
    x, y, z = x.double(), y.double(), z.double()
    L = x.shape[-2]
    i = torch.arange(L, device=x.device, dtype=torch.float64)
    gap = i[None, :] - i[:, None] if reverse else i[:, None] - i[None, :]
    l = decay_log(log_decay)[..., None, None]
    w = torch.where(gap >= 0, torch.exp(l * gap.clamp(min=0)), 0.0)
    o = (x @ y.transpose(-1, -2) * w) @ z
    A = (x.abs() @ y.abs().transpose(-1, -2) * w) @ z.abs()
    if state is not None:
        before = torch.exp(l * (i[:, None] + 1))
        o = o + before * (x @ state.double())
        A = A + before * (x.abs() @ state.double().abs())
    return o * scale, A * abs(scale)


def final_state(y, z, log_decay, state):
    """(state after the tokens, sum of magnitudes) [..., d, d]."""
    L = y.shape[-2]
    l = decay_log(log_decay)[..., None, None]
    left = torch.arange(L - 1, -1, -1, device=y.device, dtype=torch.float64)[:, None]
    w = y.double() * torch.exp(l * left)
    whole = torch.exp(l * L)
    return (whole * state.double() + w.transpose(-1, -2) @ z.double(),
            whole * state.double().abs() + w.abs().transpose(-1, -2) @ z.double().abs())


def check(name, got, want, A, dtype, terms):
    """Every element and the norm against the bounds above."""
    err = (got.double() - want).abs()
    u = U[dtype]
    bound = u * want.abs() + (2 * u if dtype == "bf16" else 0) * A + terms * 2.0 ** -24 * A + 1e-30
    assert bool((err <= bound).all()), (name, float((err / bound).max()))
    if dtype == "bf16" and want.numel() >= 256:
        assert float(err.norm()) <= u * float(want.norm()) + 1e-30, (name, float(err.norm() / want.norm()))


def grouped(t, heads):
    """[B, heads_q, L, d] as [B, heads, group, L, d]."""
    B, hq, L, d = t.shape
    return t.reshape(B, heads, hq // heads, L, d)


def reference(q, k, v, do, log_decay, scale):
    """{name: (value, A)} of o, dq, dk, dv."""
    H, d = k.shape[1], q.shape[-1]
    qg, dog = grouped(q, H), grouped(do, H)
    kg, vg = k[:, :, None].expand_as(qg), v[:, :, None].expand_as(qg)
    ld = log_decay[None, :, None].expand(qg.shape[:3])
    flat = lambda r: tuple(t.reshape(q.shape) for t in r)  # noqa: E731
    summed = lambda r: tuple(t.sum(2) for t in r)  # noqa: E731
    return dict(o=flat(walk(qg, kg, vg, ld, scale)), dq=flat(walk(dog, vg, kg, ld, scale)),
                dk=summed(walk(vg, dog, qg, ld, scale, True)), dv=summed(walk(kg, qg, dog, ld, scale, True)))
