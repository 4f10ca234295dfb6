"""Linear attention with a decay per head: S_t = g S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t, g = exp(log_decay[head]).

linear_attention(q, k, v, log_decay, scale=1.0) is the layer over whole sequences, differentiable in q, k and v (log_decay
is a constant of the model).  LinearCache holds the states of many sequences for serving, in the slots and the packing of
a PagedCache beside it:

    cache = LinearCache(slots=64, heads=8, head_dim=128)
    o = cache.extend(q, k, v, log_decay, q_start=starts, max_new=512)   # packed new tokens, as PagedCache.extend
    o = cache.extend(q, k, v, log_decay)                                # one token for every slot
    o = cache.extend(..., update=False)                                 # drafts: the states stay as they were
    # (drafts that a PagedCache holds under forks need none here: with a q_start that gives their rows to the parents,
    #  in the children's order, the parents' states are read)
    cache.fork(parents, children); cache.reset(slots)
    cache.check()                                                       # raises what the device found, if anything

Argument marshalling only: every step runs in the CUDA library, on the current stream of the tensors' device, without
synchronising (check() does).  Calls that change one cache must be ordered on one stream.  A call can be captured into a
CUDA graph: q_start and lists are read on the device; the cache's handle, whose status word it uses, outlives the graph.
(A training step is captured as torch asks for it: with leaves of which no eager graph is alive.)
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import path_attn as pa

TOKEN_MAX = 16  # new tokens of a slot up to which no workspace is used


_descs = {}  # (descriptor's numbers, backward?) -> reference to the descriptor, workspace bytes


class LinearAttentionFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay, scale, check):
        q, k, v, log_decay = q.contiguous(), k.contiguous(), v.contiguous(), log_decay.contiguous()
        dt = q.dtype
        if dt not in pa._DT:
            raise ValueError(f"unsupported dtype {dt}")
        if q.dim() != 4 or k.dim() != 4:
            raise ValueError(f"q is [B, heads_q, L, d], k and v [B, heads, L, d], got {tuple(q.shape)} and {tuple(k.shape)}")
        B, hq, L, d = q.shape
        H = k.shape[1]
        at = q.get_device()  # (below 0: host memory)
        if not (at >= 0 and k.dtype is dt and v.dtype is dt and log_decay.dtype is torch.float32 and k.shape == (B, H, L, d)
                and v.shape == k.shape and log_decay.shape == (H,) and k.get_device() == at and v.get_device() == at
                and log_decay.get_device() == at):
            for name, t, want, shape in (("q", q, dt, (B, hq, L, d)), ("k", k, dt, (B, H, L, d)), ("v", v, dt, (B, H, L, d)),
                                         ("log_decay", log_decay, torch.float32, (H,))):
                pa._need(t, want, shape, name)
                if t.device != q.device:
                    raise ValueError(f"{name} lies on {t.device}, q on {q.device}")
        o = torch.empty_like(q)
        ctx.save_for_backward(q, k, v, log_decay)
        ctx.desc, ctx.check = (B, hq, H, L, d, pa._DT[dt], float(scale)), check
        if q.numel():
            _launch(pa._lib.path_linear_fwd, 0, ctx.desc, check, q, k, v, log_decay, o)
        return o

    @staticmethod
    def backward(ctx, do):
        # (only a graph of the gradients themselves needs to know that there is none)
        return _backward_once(ctx, do) if torch.is_grad_enabled() else _backward(ctx, do)


def _backward(ctx, do):
    q, k, v, log_decay = ctx.saved_tensors
    new = torch.empty_like if q.numel() else torch.zeros_like
    dq, dk, dv = [new(t) if need else None for t, need in zip((q, k, v), ctx.needs_input_grad)]
    if q.numel() and not (dq is dk is dv is None):
        _launch(pa._lib.path_linear_bwd, 1, ctx.desc, ctx.check, q, k, v, log_decay, do.contiguous(), dq, dk, dv)
    return dq, dk, dv, None, None, None


_backward_once = once_differentiable(_backward)


def _launch(fn, for_backward, numbers, check, q, *tensors):
    if check and torch.cuda.is_current_stream_capturing():
        raise ValueError("check=True waits for the device: not while its stream is captured into a graph")
    key = (numbers, for_backward)
    made = _descs.get(key)
    if made is None:
        desc = pa.path_linear_desc_t(*numbers)
        n = pa.path_linear_workspace_size(desc, for_backward)
        if n == 0:
            raise ValueError(f"linear_attention: {desc.heads_q} query heads over {desc.heads} (a multiple, at most 16 times), "
                             f"head dim {desc.head_dim} (64 or 128), scale {desc.scale}, or sizes out of range")
        if len(_descs) >= 1024:
            _descs.clear()
        _descs[key] = made = (ctypes.byref(desc), n)
    desc, n = made
    ws = torch.empty(n, dtype=torch.uint8, device=q.device)
    args = [None if t is None else t.data_ptr() for t in tensors]
    index = q.get_device()
    if torch._C._cuda_getDevice() == index:  # (as torch.cuda.current_device, without its checks)
        rc = fn(desc, q.data_ptr(), *args, ws.data_ptr(), n, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(desc, q.data_ptr(), *args, ws.data_ptr(), n, pa._stream())
    if rc != pa.PATH_OK:
        pa._check(rc, fn.__name__)
    if check:
        with torch.cuda.device(index):
            rc, code = pa.path_linear_workspace_status(desc._obj, ws.data_ptr(), n, pa._stream())
        if rc != pa.PATH_OK:
            raise RuntimeError(f"{fn.__name__}: device status of the workspace: {pa.path_status_string(rc)} (code {code})")


def linear_attention(q, k, v, log_decay, scale=1.0, check=False):
    """o [B, heads_q, L, d] of q [B, heads_q, L, d], k and v [B, heads, L, d] (bf16 or float32, one dtype; heads_q a
    multiple of heads: query head hq reads key head hq // (heads_q // heads)) and log_decay [heads] float32, the natural
    logarithm of the decay per token, kept in [-10000, 0].  Sequences begin with a zero state.  check=True: this call and its
    backward synchronise and raise if a kernel gave up a bounded wait (what it wrote is then incomplete; without check nobody is
    told).  An infinity or NaN in a sequence may reach any output and gradient of that sequence and head, those of earlier
    tokens too: padding has to be clean.  The same call gives the same bits; a sequence in another batch may get other last ones."""
    if log_decay.requires_grad and torch.is_grad_enabled():
        raise ValueError("log_decay is a constant: linear_attention has no gradient for it")
    return LinearAttentionFunction.apply(q, k, v, log_decay, scale, check)


class LinearCache:
    """States [slots, heads, head_dim of k, head_dim of v] float32 of many sequences (path_linear_cache_t in
    include/path_attn.h).  A new cache's states are zero: empty sequences."""

    def __init__(self, slots, heads, head_dim, dtype=torch.bfloat16, device="cuda"):
        for name, x in (("slots", slots), ("heads", heads)):
            if int(x) <= 0:
                raise ValueError(f"{name} must be positive, got {x}")
        if head_dim not in (64, 128):
            raise ValueError(f"head_dim must be 64 or 128, got {head_dim}")
        if dtype not in pa._DT:
            raise ValueError(f"unsupported dtype {dtype}")
        self._bind(torch.zeros(slots, heads, head_dim, head_dim, dtype=torch.float32, device=device), dtype)

    @classmethod
    def from_tensors(cls, state, dtype=torch.bfloat16):
        """A cache over states that exist already (kept, not copied), for tokens of the given dtype."""
        self = cls.__new__(cls)
        self._bind(state, dtype)
        return self

    def _bind(self, state, dtype):
        if dtype not in pa._DT:
            raise ValueError(f"unsupported dtype {dtype}")
        if state.dim() != 4 or state.shape[2] != state.shape[3]:
            raise ValueError(f"states are [slots, heads, head_dim, head_dim], got {tuple(state.shape)}")
        pa._need(state, torch.float32, state.shape, "state")
        self.state, self.dtype, self.device = state, dtype, state.device
        self.slots, self.heads, self.head_dim = state.shape[:3]
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.c = pa.path_linear_cache_t(self.slots, self.heads, self.head_dim, pa._DT[dtype], pa._p(state), pa._p(self.status))
        self._ref, self._index = ctypes.byref(self.c), self.device.index
        self._plans = {}
        if pa.path_linear_extend_workspace_size(self.c, pa.path_linear_step_t(self.heads, 0, 0, 1.0, 1)) == 0:
            raise ValueError("unsupported cache (head_dim 64 or 128, at most 65535 slots and 1024 heads)")

    def extend(self, q, k, v, log_decay, q_start=None, max_new=None, scale=1.0, update=True, ws=None, out=None):
        """o [tokens, heads_q, head_dim] of the packed new tokens q [tokens, heads_q, head_dim], k, v [tokens, heads,
        head_dim]; log_decay [heads] float32.  q_start (int32 [slots + 1]): slot b's tokens are q_start[b] ..
        q_start[b + 1] - 1, at most max_new of them (default: all); without it, token b is slot b's.  A slot whose row of
        q_start is bad, or begins inside an earlier slot's tokens, is left out (check() tells).  The states take the
        tokens in; with update=False they stay.  out must not overlap the other tensors.  ws: uint8, at least
        path_linear_extend_workspace_size bytes, for one call at a time (default: a new one)."""
        dt, at = self.dtype, self._index
        # (numbers, whatever holds them: a tensor would be found by its identity, not by what it holds now)
        max_new, scale, update = None if max_new is None else int(max_new), float(scale), bool(update)
        key = (q.shape, k.shape, v.shape, q_start is None, max_new, scale, update)
        plan = self._plans.get(key)
        if plan is None or q.dtype is not dt or k.dtype is not dt or v.dtype is not dt or not (
                q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and q.get_device() == k.get_device() == v.get_device() == at):
            plan = self._plans[key] = self._plan(q, k, v, q_start, max_new, scale, update)
        step, n, chunks = plan
        self._need(log_decay, torch.float32, (self.heads,), "log_decay")
        if q_start is not None:
            self._need(q_start, torch.int32, (self.slots + 1,), "q_start")
        if out is None:
            out = torch.empty_like(q)
        else:
            self._need(out, dt, tuple(q.shape), "out")
        if out.shape[0] == 0:
            return out
        if ws is not None:
            if ws.dtype != torch.uint8 or ws.device != self.device or not ws.is_contiguous() or ws.numel() < n:
                raise ValueError(f"ws: expected at least {n} contiguous uint8 on {self.device}, got {ws.numel()} {ws.dtype} on "
                                 f"{ws.device} contiguous={ws.is_contiguous()}")
        elif chunks:
            ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        self._call(pa._lib.path_linear_extend, step, None if q_start is None else q_start.data_ptr(), q.data_ptr(), k.data_ptr(),
                   v.data_ptr(), log_decay.data_ptr(), out.data_ptr(), None if ws is None else ws.data_ptr(), n)
        return out

    def _plan(self, q, k, v, q_start, max_new, scale, update):
        """(descriptor, workspace bytes, whether they are used) of calls of these sizes, once their tensors are right."""
        if q.dim() != 3:
            raise ValueError(f"q: expected [tokens, heads_q, head_dim], got {tuple(q.shape)}")
        N, hq, _ = q.shape
        self._need(q, self.dtype, (N, hq, self.head_dim), "q")
        for name, t in (("k", k), ("v", v)):
            self._need(t, self.dtype, (N, self.heads, self.head_dim), name)
        if q_start is None and N != self.slots:
            raise ValueError(f"without q_start there is one token per slot: {N} tokens for {self.slots} slots")
        if max_new is None:
            max_new = 1 if q_start is None else N
        if N > 0 and max_new < 1:
            raise ValueError(f"max_new must be at least 1 for {N} tokens, got {max_new}")
        step = pa.path_linear_step_t(hq, N, max_new, scale, int(update))
        n = pa.path_linear_extend_workspace_size(self.c, step)
        if n == 0:
            raise ValueError(f"invalid sizes: {hq} query heads over {self.heads}, {N} tokens, scale {scale}")
        if len(self._plans) >= 1024:
            self._plans.clear()
        return ctypes.byref(step), n, min(max_new, N) > TOKEN_MAX

    def fork(self, parents, children):
        """children[i] takes the state of parents[i] (int32 lists on the device)."""
        self._list(parents, "parents")
        self._list(children, "children")
        if parents.numel() != children.numel():
            raise ValueError("parents and children have different lengths")
        if parents.numel():
            self._call(pa._lib.path_linear_fork, pa._p(parents), pa._p(children), parents.numel())

    def reset(self, slots):
        """The listed slots begin new sequences: their states become zero."""
        self._list(slots, "slots")
        if slots.numel():
            self._call(pa._lib.path_linear_fork, None, pa._p(slots), slots.numel())

    def check(self):
        """Raises RuntimeError with what the device recorded since the last check; synchronises."""
        from .paged import CODES

        with torch.cuda.device(self.device):
            rc, code = pa.path_linear_status(self.c, pa._stream())
        if rc != pa.PATH_OK:
            what = CODES.get(code, f"a kernel's bounded wait gave up (code {code})" if code else "")
            raise RuntimeError(f"linear cache: {pa.path_status_string(rc)}: {what}")

    # ---- helpers ----
    def _call(self, fn, *args):
        """The library's fn(cache, *args, stream) on the current stream of the cache's device; raises on a status."""
        if torch._C._cuda_getDevice() == self._index:  # (as torch.cuda.current_device, without its checks)
            rc = fn(self._ref, *args, torch._C._cuda_getCurrentRawStream(self._index))
        else:
            with torch.cuda.device(self.device):
                rc = fn(self._ref, *args, pa._stream())
        if rc != pa.PATH_OK:
            pa._check(rc, fn.__name__)

    def _need(self, t, dtype, shape, name):
        if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != self.device:
            pa._need(t, dtype, shape, name)
            raise ValueError(f"{name} lies on {t.device}, the cache on {self.device}")

    def _list(self, t, name):
        if t.dim() != 1 or t.numel() > self.slots:
            raise ValueError(f"{name}: a list of at most {self.slots} slots")
        self._need(t, torch.int32, tuple(t.shape), name)
