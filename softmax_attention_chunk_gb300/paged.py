"""Paged serving on the PaTH attention library: a cache of many sequences in pages, attention of new
tokens over it, and the management of its pages.

    cache = PagedCache(slots=64, heads=8, head_dim=128, page_size=64, k_pages=4096, v_pages=4096,
                       table_width=512)
    cache.reserve(n_new)                                  # int32 [slots] on the GPU; opens empty slots
    o = cache.extend(q, k, v, w, beta, q_start=starts, max_new=512)     # packed new tokens
    cache.advance(starts)
    cache.reserve(); o = cache.extend(q, k, v, w, beta); cache.advance()  # one token for every slot
    cache.fork(parents, children); cache.free(slots); cache.trim(window, sinks); cache.compact()
    cache.check()                                         # raises what the device found, if anything

Keys are held transported to the newest position, so a step rewrites every key of its sequence and key
pages are never shared; value pages are (fork).  What a step did to them cannot be taken back: draft tokens that
may be rejected are checked on a fork,
    cache.fork(parent, child); cache.reserve(n); o = cache.extend(..., q_start=for_child, max_new=m)
    cache.free(child); o = cache.extend(..., q_start=accepted_for_parent)   # or keep the child, if all are accepted
and advance() takes the tokens of an extend whole or not at all.  A slot that extend leaves out (its tokens'
pages are missing after a refused reserve, say) is passed over by advance().  Argument marshalling only: every step runs in the CUDA
library, on the current stream of the cache's device, without synchronising (check() does).  Calls that
change one cache must be ordered on one stream.  A call can be captured into a CUDA graph: it reads
lengths, tables and lists on the device.  Graphs and work still queued use the handle's tensors (its status word too; with
from_tensors those that it was not given): the handle outlives both.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import path_attn as pa

CODES = {1: "a needed page-table entry is not a page of the pool", 2: "a sequence would outgrow its table row",
         3: "slot out of range, listed twice, empty where it must not be, or in use", 4: "not enough free pages",
         5: "q_start falls, leaves the packed tokens, exceeds max_new, or (advance) is not what extend was given",
         6: "a drafted token is not in the vocabulary"}


class StepPlan(NamedTuple):
    """Where the packed new tokens of a step go (int32 on the device; -1 behind the last token)."""

    q_start: torch.Tensor   # [slots + 1]: for extend and advance
    slot: torch.Tensor      # [tokens]
    position: torch.Tensor  # in the sequence
    k_row: torch.Tensor     # row of the key pool: page * page_size + place in the page
    v_row: torch.Tensor     # of the value pool
    source: Optional[torch.Tensor]  # row of an earlier packing


class PagedCache:
    """Pools, page tables and counts of a paged cache (see path_paged_cache_t in include/path_attn.h)."""

    def __init__(self, slots, heads, head_dim, page_size, k_pages, v_pages=None, table_width=None,
                 dtype=torch.bfloat16, fox=False, device="cuda"):
        v_pages = k_pages if v_pages is None else v_pages
        table_width = k_pages if table_width is None else table_width
        for name, x in (("slots", slots), ("heads", heads), ("k_pages", k_pages), ("v_pages", v_pages),
                        ("table_width", table_width)):
            if int(x) <= 0:
                raise ValueError(f"{name} must be positive, got {x}")
        if dtype not in pa._DT:
            raise ValueError(f"unsupported dtype {dtype}")
        if head_dim not in (64, 128) or page_size not in (16, 32, 64, 128, 256):
            raise ValueError(f"head_dim must be 64 or 128 and page_size 16, 32, 64, 128 or 256, got {head_dim}, {page_size}")
        i32 = dict(dtype=torch.int32, device=device)
        self._bind(torch.zeros(k_pages, heads, page_size, head_dim, dtype=dtype, device=device),
                   torch.zeros(v_pages, heads, page_size, head_dim, dtype=dtype, device=device),
                   torch.full((slots, table_width), -1, **i32), torch.full((slots, table_width), -1, **i32),
                   torch.full((slots,), -1, **i32), torch.zeros(k_pages, **i32), torch.zeros(v_pages, **i32),
                   torch.zeros(v_pages, heads, page_size, dtype=torch.float32, device=device) if fox else None)

    @classmethod
    def from_tensors(cls, k_pool, v_pool, k_table, v_table, seq_len, k_ref, v_ref, a_pool=None, extended=None, a_rest=None):
        """A cache over tensors that exist already (kept, not copied).  extended (int32 [slots]; default: zeros) is
        what extend leaves for advance, a_rest (as a_pool; default: zeros) what rounding the gate's running sums to
        float32 left of them: a second handle of one cache takes the first one's."""
        self = cls.__new__(cls)
        self._bind(k_pool, v_pool, k_table, v_table, seq_len, k_ref, v_ref, a_pool, extended, a_rest)
        return self

    def _bind(self, k_pool, v_pool, k_table, v_table, seq_len, k_ref, v_ref, a_pool, extended=None, a_rest=None):
        if k_pool.dim() != 4 or v_pool.dim() != 4 or k_table.dim() != 2:
            raise ValueError("pools are [pages, heads, page_size, head_dim], tables [slots, table_width]")
        kp, H, P, d = k_pool.shape
        vp = v_pool.shape[0]
        slots, width = k_table.shape
        if k_pool.dtype not in pa._DT:
            raise ValueError(f"unsupported dtype {k_pool.dtype}")
        pa._need(k_pool, k_pool.dtype, (kp, H, P, d), "k_pool")
        pa._need(v_pool, k_pool.dtype, (vp, H, P, d), "v_pool")
        for name, t, shape in (("k_table", k_table, (slots, width)), ("v_table", v_table, (slots, width)),
                               ("seq_len", seq_len, (slots,)), ("k_ref", k_ref, (kp,)), ("v_ref", v_ref, (vp,))):
            pa._need(t, torch.int32, shape, name)
        if a_pool is not None:
            pa._need(a_pool, torch.float32, (vp, H, P), "a_pool")
        self.device = k_pool.device
        if extended is None:
            extended = torch.zeros(slots, dtype=torch.int32, device=self.device)
        pa._need(extended, torch.int32, (slots,), "extended")
        if a_pool is not None and a_rest is None:
            a_rest = torch.zeros_like(a_pool)
        if a_rest is not None:
            pa._need(a_rest, torch.float32, (vp, H, P), "a_rest")
            if a_pool is None:
                raise ValueError("a_rest goes with a_pool")
        for t in (v_pool, k_table, v_table, seq_len, k_ref, v_ref, a_pool, extended, a_rest):
            if t is not None and t.device != self.device:
                raise ValueError("the tensors of a cache lie on one device")
        self.k_pool, self.v_pool, self.a_pool = k_pool, v_pool, a_pool
        self.k_table, self.v_table, self.seq_len, self.k_ref, self.v_ref = k_table, v_table, seq_len, k_ref, v_ref
        self.extended, self.a_rest = extended, a_rest
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.slots, self.heads, self.head_dim, self.page_size, self.dtype = slots, H, d, P, k_pool.dtype
        p = pa._p
        self.c = pa.path_paged_cache_t(slots, H, d, P, width, kp, vp, pa._DT[k_pool.dtype], p(k_pool), p(v_pool),
                                       p(a_pool), p(k_table), p(v_table), p(seq_len), p(k_ref), p(v_ref),
                                       p(self.status), p(extended), p(a_rest))
        self._ref, self._index = ctypes.byref(self.c), self.device.index
        self._plans, self._verifications = {}, {}
        self._pages_bytes = pa.path_pages_workspace_size(self.c)
        if self._pages_bytes == 0:
            raise ValueError("unsupported cache (head_dim 64 or 128; page_size 16, 32, 64, 128 or 256; sizes in range)")

    # ---- attention ----
    def extend(self, q, k, v, w, beta, log_f=None, q_start=None, max_new=None, scale=1.0, window=0, sinks=0, ws=None,
               out=None, max_multi=0):
        """o [tokens, heads_q, head_dim] of the packed new tokens q [tokens, heads_q, head_dim], k, v, w [tokens,
        heads, head_dim], beta and log_f [tokens, heads] float32 (log_f exactly for a cache with fox).  q_start
        (int32 [slots + 1]): slot b's tokens are q_start[b] .. q_start[b + 1] - 1, at most max_new of them
        (default: all); without it, token b is slot b's.  At most max_multi slots have several tokens (0: any number;
        stated, a prompt among many single tokens needs the workspace of a prompt).  window > 0 hides all but the last `window` tokens and
        the first `sinks`.  The cache's keys are rewritten and the new rows appended; seq_len is not changed.  out
        must not overlap the other tensors.  ws: uint8, at least path_paged_workspace_size bytes, for one call at a
        time (default: a new one)."""
        if q.dim() != 3:
            raise ValueError(f"q: expected [tokens, heads_q, head_dim], got {tuple(q.shape)}")
        N, hq, d = q.shape
        kv = (N, self.heads, self.head_dim)
        self._need(q, self.dtype, (N, hq, self.head_dim), "q")
        for name, t in (("k", k), ("v", v), ("w", w)):
            self._need(t, self.dtype, kv, name)
        self._need(beta, torch.float32, kv[:2], "beta")
        if (log_f is None) != (self.a_pool is None):
            raise ValueError("log_f goes with a cache that has the forget gate (fox)")
        if log_f is not None:
            self._need(log_f, torch.float32, kv[:2], "log_f")
        if q_start is not None:
            self._need(q_start, torch.int32, (self.slots + 1,), "q_start")
        elif N != self.slots:
            raise ValueError(f"without q_start there is one token per slot: {N} tokens for {self.slots} slots")
        # (numbers, whatever holds them: a tensor would be found by its identity below, not by what it holds now)
        max_new = (1 if q_start is None else N) if max_new is None else int(max_new)
        scale, window, sinks, max_multi = float(scale), int(window), int(sinks), int(max_multi)
        if N > 0 and max_new < 1:
            raise ValueError(f"max_new must be at least 1 for {N} tokens, got {max_new}")
        key = (hq, N, max_new, scale, window, sinks, max_multi)
        plan = self._plans.get(key)
        if plan is None:  # descriptor and workspace size of calls of these sizes
            desc = pa.path_paged_desc_t(hq, N, max_new, scale, window, sinks, max_multi)
            n = pa.path_paged_workspace_size(self.c, desc)
            if n == 0:
                raise ValueError(f"invalid sizes: {hq} query heads over {self.heads}, {N} tokens, window {window}, sinks {sinks}")
            if len(self._plans) >= 1024:
                self._plans.clear()
            plan = self._plans[key] = (desc, n)
        desc, n = plan
        if out is None:
            out = torch.empty_like(q)
        else:
            self._need(out, self.dtype, tuple(q.shape), "out")
        if N == 0:
            return out
        if ws is None:
            ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        elif ws.dtype != torch.uint8 or ws.device != self.device or not ws.is_contiguous() or ws.numel() < n:
            raise ValueError(f"ws: expected at least {n} contiguous uint8 on {self.device}, got {ws.numel()} {ws.dtype} on "
                             f"{ws.device} contiguous={ws.is_contiguous()}")
        if beta.data_ptr() % 16:  # (of a part of a packed batch; the library wants 16-byte boundaries)
            beta = beta.clone()
        if log_f is not None and log_f.data_ptr() % 16:
            log_f = log_f.clone()
        p = pa._p
        self._call(pa.path_paged_extend, desc, p(q_start), q.data_ptr(), k.data_ptr(), v.data_ptr(), w.data_ptr(),
                   beta.data_ptr(), p(log_f), out.data_ptr(), ws.data_ptr(), ws.numel())
        return out

    def advance(self, q_start=None):
        """seq_len grows by the new tokens of an extend with the same q_start (check() reports another one); slots
        that it left out are passed over.  Without an extend before it: by rows that the caller wrote itself."""
        if q_start is not None:
            self._need(q_start, torch.int32, (self.slots + 1,), "q_start")
        self._call(pa.path_paged_advance, pa._p(q_start))

    def check(self):
        """Raises RuntimeError with what the device recorded since the last check; synchronises."""
        with torch.cuda.device(self.device):
            rc, code = pa.path_paged_status(self.c, pa._stream())
        if rc != pa.PATH_OK:
            what = CODES.get(code, f"a kernel's bounded wait gave up (code {code})" if code else "")
            raise RuntimeError(f"paged cache: {pa.path_status_string(rc)}: {what}")

    # ---- a step's tokens ----
    def plan(self, n_new, tokens, from_start=None):
        """reserve(n_new), and the StepPlan of these new tokens, packed in slot order into arrays of `tokens` rows.
        from_start (int32 [slots + 1]): the q_start of an earlier packing that began with the same tokens of each slot;
        source then says which of its rows each token is (draft tokens of which n_new were kept).  With more than
        `tokens` new tokens, or where reserve records an error, nothing is reserved and the plan is empty."""
        if n_new is not None:
            self._need(n_new, torch.int32, (self.slots,), "n_new")
        if from_start is not None:
            self._need(from_start, torch.int32, (self.slots + 1,), "from_start")
        tokens = int(tokens)
        if not 0 <= tokens <= 1 << 22:
            raise ValueError(f"tokens must be in 0 .. {1 << 22}, got {tokens}")
        count = 4 if from_start is None else 5
        flat = torch.empty(count * tokens + self.slots + 1, dtype=torch.int32, device=self.device)
        *maps, start = flat.split_with_sizes([tokens] * count + [self.slots + 1])
        at, row, ws = flat.data_ptr(), 4 * tokens, self._pages_workspace()
        self._library(pa._lib.path_pages_plan, self._ref, None if n_new is None else n_new.data_ptr(),
                      None if from_start is None else from_start.data_ptr(), tokens, at + count * row, at, at + row, at + 2 * row,
                      at + 3 * row, None if from_start is None else at + 4 * row, ws.data_ptr(), self._pages_bytes)
        return StepPlan(start, *maps) if count == 5 else StepPlan(start, *maps, None)

    def verify(self, target, tokens, uniform, draft=None, q_start=None, max_new=None):
        """(keep, next), int32 [slots]: how many of each slot's packed tokens stay, the first (known) one among them, and
        the token after those.  A slot's tokens (int32, packed as for extend with the same q_start) are a known one, then
        its drafts; target [tokens, vocab] (bf16 or float32) holds the target's probabilities after each token, draft (the
        same, or None: the drafts are certain) those that each was drawn from.  Draft i stays if those before it do and
        uniform[i] * draft[i][x] < target[i - 1][x]; next is drawn with the uniform of the slot's first token from
        max(0, target - draft) of the first draft that went, or from target behind the last token.  Slots without tokens
        get 0 and -1.  Rows may be apart (a stride), their entries not.  Of drafts on forks keep and next stand at the children:
        the parents' new tokens are those counts, moved to the parents' slots."""
        max_new = None if max_new is None else int(max_new)
        key = (target.shape, target.dtype, target.stride(), None if draft is None else draft.stride(), max_new)
        desc = self._verifications.get(key)
        if desc is None:
            desc = ctypes.byref(self._verification(target, draft, max_new))
            if len(self._verifications) >= 1024:
                self._verifications.clear()
            self._verifications[key] = desc
        N = target.shape[0]
        if target.device != self.device or (draft is not None and (draft.dtype != target.dtype or draft.shape != target.shape
                                                                   or draft.device != self.device)):
            raise ValueError(f"target and draft: expected one type and shape on {self.device}, got {target.dtype} {tuple(target.shape)} on "
                             f"{target.device}" + ("" if draft is None else f" and {draft.dtype} {tuple(draft.shape)} on {draft.device}"))
        self._need(tokens, torch.int32, (N,), "tokens")
        self._need(uniform, torch.float32, (N,), "uniform")
        if q_start is None:
            raise ValueError("q_start is needed: it says which tokens are whose")
        self._need(q_start, torch.int32, (self.slots + 1,), "q_start")
        keep = torch.empty(self.slots, dtype=torch.int32, device=self.device)
        after = torch.empty(self.slots, dtype=torch.int32, device=self.device)
        self._library(pa._lib.path_draft_verify, desc, q_start.data_ptr(), tokens.data_ptr(), uniform.data_ptr(), target.data_ptr(),
                      None if draft is None else draft.data_ptr(), keep.data_ptr(), after.data_ptr(), self.status.data_ptr())
        return keep, after

    def _verification(self, target, draft, max_new):
        """The descriptor of calls with rows like these."""
        if target.dim() != 2 or target.dtype not in pa._DT:
            raise ValueError(f"target: expected [tokens, vocab] bf16 or float32, got {target.dtype} {tuple(target.shape)}")
        N, vocab = target.shape
        strides = []
        for name, t in (("target", target), ("draft", draft)):
            if t is not None and (t.shape != target.shape or (vocab > 1 and t.stride(1) != 1) or (N > 1 and t.stride(0) < vocab)):
                raise ValueError(f"{name}: expected {tuple(target.shape)} with contiguous rows, got {tuple(t.shape)} strides {t.stride()}")
            strides.append(vocab if t is None or N <= 1 else t.stride(0))
        max_new = N if max_new is None else max_new
        if max_new < 0 or not 0 < vocab <= 1 << 20:
            raise ValueError(f"max_new must not be negative and vocab in 1 .. {1 << 20}, got {max_new} and {vocab}")
        return pa.path_verify_desc_t(self.slots, N, max_new, vocab, pa._DT[target.dtype], *strides)

    # ---- pages ----
    def reserve(self, n_new=None):
        """Pages for n_new[b] (int32 [slots]; None: 1 for every slot in use) more tokens per slot; an empty
        slot with n_new > 0 is opened."""
        if n_new is not None:
            self._need(n_new, torch.int32, (self.slots,), "n_new")
        self._pages("reserve", pa._p(n_new))

    def fork(self, parents, children):
        """children[i] (an empty slot) becomes a copy of parents[i] (int32 lists on the device)."""
        self._list(parents, "parents")
        self._list(children, "children")
        if parents.numel() != children.numel():
            raise ValueError("parents and children have different lengths")
        if parents.numel():
            self._pages("fork", pa._p(parents), pa._p(children), parents.numel())

    def free(self, slots):
        """The listed slots become empty and their pages return."""
        self._list(slots, "slots")
        if slots.numel():
            self._pages("free", pa._p(slots), slots.numel())

    def trim(self, window, sinks=0):
        """Returns the pages whose rows a window and first tokens hide from every later token."""
        self._pages("trim", int(window), int(sinks))

    def compact(self):
        """Moves the pages in use to the front of each pool."""
        self._pages("compact")

    # ---- helpers ----
    def _pages_workspace(self):
        # (for one call, on its stream: a captured call's lies in the graph's memory and stays when the handle goes)
        return torch.empty(self._pages_bytes, dtype=torch.uint8, device=self.device)

    def _pages(self, name, *args):
        ws = self._pages_workspace()
        self._call(getattr(pa, "path_pages_" + name), *args, ws.data_ptr(), self._pages_bytes)

    def _call(self, fn, *args):
        """fn(cache, *args, stream) on the current stream of the cache's device; raises on a status."""
        if torch._C._cuda_getDevice() == self._index:  # (as torch.cuda.current_device, without its checks)
            rc = fn(self.c, *args, torch._C._cuda_getCurrentRawStream(self._index))
        else:
            with torch.cuda.device(self.device):
                rc = fn(self.c, *args, pa._stream())
        if rc != pa.PATH_OK:
            pa._check(rc, fn.__name__)

    def _library(self, fn, *args):
        """The library's fn(*args, stream), as _call."""
        if torch._C._cuda_getDevice() == self._index:
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(self._index))
        else:
            with torch.cuda.device(self.device):
                rc = fn(*args, pa._stream())
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
