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
lengths, tables and lists on the device.
"""
from __future__ import annotations

import torch

from . import path_attn as pa

CODES = {1: "a needed page-table entry is not a page of the pool", 2: "a sequence would outgrow its table row",
         3: "slot out of range, listed twice, empty where it must not be, or in use", 4: "not enough free pages",
         5: "q_start falls, leaves the packed tokens, exceeds max_new, or (advance) is not what extend was given"}


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
        self._index = self.device.index
        self._plans = {}
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
        if max_new is None:
            max_new = 1 if q_start is None else N
        if N > 0 and max_new < 1:
            raise ValueError(f"max_new must be at least 1 for {N} tokens, got {max_new}")
        key = (hq, N, max_new, scale, window, sinks, max_multi)
        plan = self._plans.get(key)
        if plan is None:  # descriptor and workspace size of calls of these sizes
            desc = pa.path_paged_desc_t(hq, N, int(max_new), float(scale), int(window), int(sinks), int(max_multi))
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
    def _pages(self, name, *args):
        ws = torch.empty(self._pages_bytes, dtype=torch.uint8, device=self.device)
        self._call(getattr(pa, "path_pages_" + name), *args, ws.data_ptr(), ws.numel())

    def _call(self, fn, *args):
        """fn(cache, *args, stream) on the current stream of the cache's device; raises on a status."""
        if torch._C._cuda_getDevice() == self._index:  # (as torch.cuda.current_device, without its checks)
            rc = fn(self.c, *args, torch._C._cuda_getCurrentRawStream(self._index))
        else:
            with torch.cuda.device(self.device):
                rc = fn(self.c, *args, pa._stream())
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
