"""Page management against a plain model on the CPU: reserve, fork, free, trim, compact, and their refusals."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Model:
    """The same cache on the CPU, one page after the other."""

    def __init__(self, cache):
        self.P = cache.page_size
        for n in ("k_pool", "v_pool", "a_pool", "k_table", "v_table", "seq_len", "k_ref", "v_ref"):
            t = getattr(cache, n)
            setattr(self, n, None if t is None else t.cpu().clone())

    def take(self, ref):
        p = int((ref == 0).nonzero()[0])
        ref[p] = 1
        return p

    def reserve(self, n_new):
        for b, n in enumerate(n_new):
            if n <= 0:
                continue
            ln = max(int(self.seq_len[b]), 0)
            self.seq_len[b] = ln
            for x in range(-(-ln // self.P), -(-(ln + n) // self.P)):
                if self.k_table[b, x] < 0:
                    self.k_table[b, x] = self.take(self.k_ref)
                if self.v_table[b, x] < 0:
                    self.v_table[b, x] = self.take(self.v_ref)

    def fork(self, parents, children):
        moves_k, moves_v = [], []
        for p, c in zip(parents, children):
            ln = int(self.seq_len[p])
            self.k_table[c] = self.v_table[c] = -1
            for x in range(-(-ln // self.P)):
                if self.k_table[p, x] >= 0:
                    n = self.take(self.k_ref)
                    moves_k.append((int(self.k_table[p, x]), n))
                    self.k_table[c, x] = n
                if self.v_table[p, x] >= 0:
                    if (x + 1) * self.P > ln:
                        n = self.take(self.v_ref)
                        moves_v.append((int(self.v_table[p, x]), n))
                    else:
                        n = int(self.v_table[p, x])
                        self.v_ref[n] += 1
                    self.v_table[c, x] = n
            self.seq_len[c] = ln
        self.move(moves_k, moves_v)

    def move(self, mk, mv):
        for a, b in mk:
            self.k_pool[b] = self.k_pool[a]
        for a, b in mv:
            self.v_pool[b] = self.v_pool[a]
            if self.a_pool is not None:
                self.a_pool[b] = self.a_pool[a]

    def drop(self, b, x):
        if self.k_table[b, x] >= 0:
            self.k_ref[self.k_table[b, x]] = 0
        if self.v_table[b, x] >= 0:
            self.v_ref[self.v_table[b, x]] -= 1
        self.k_table[b, x] = self.v_table[b, x] = -1

    def free(self, slots):
        for b in slots:
            for x in range(self.k_table.shape[1]):
                self.drop(b, x)
            self.seq_len[b] = -1

    def trim(self, window, sinks):
        for b, ln in enumerate(self.seq_len.tolist()):
            for x in range(self.k_table.shape[1]):
                rows = range(x * self.P, (x + 1) * self.P)
                if ln > 0 and all(j >= sinks and j <= ln - window and j < ln - 1 for j in rows):
                    self.drop(b, x)

    def compact(self):
        out = []
        for table, ref in ((self.k_table, self.k_ref), (self.v_table, self.v_ref)):
            n = int((ref > 0).sum())
            src = [p for p in range(n, len(ref)) if ref[p] > 0]
            dst = [p for p in range(n) if ref[p] <= 0]
            for a, b in zip(src, dst):
                ref[b], ref[a] = int(ref[a]), 0
                table[table == a] = b
            out.append(list(zip(src, dst)))
        self.move(*out)

    def same(self, cache):
        torch.cuda.synchronize()
        for n in ("k_table", "v_table", "seq_len", "k_ref", "v_ref", "k_pool", "v_pool", "a_pool"):
            x = getattr(self, n)
            if x is not None:
                assert torch.equal(x, getattr(cache, n).cpu()), n


def make(slots=6, heads=2, d=64, P=16, pages=120, width=30, dtype=torch.bfloat16, fox=True, v_pages=None):
    from softmax_attention_chunk_gb300.paged import PagedCache

    c = PagedCache(slots, heads, d, P, pages, v_pages=v_pages, table_width=width, dtype=dtype, fox=fox)
    g = torch.Generator(device=DEV).manual_seed(3)
    for t in (c.k_pool, c.v_pool) + ((c.a_pool,) if fox else ()):
        t.normal_(generator=g)
    return c


@pytest.mark.parametrize("P,heads,d,dtype,fox", [(16, 2, 64, torch.bfloat16, True), (64, 3, 128, torch.float32, False),
                                                 (256, 1, 128, torch.bfloat16, True), (32, 16, 64, torch.bfloat16, False)])
def test_against_the_model(cuda_lib, P, heads, d, dtype, fox):
    c = make(heads=heads, d=d, P=P, dtype=dtype, fox=fox)
    m = Model(c)

    def grow(n):
        c.reserve(i32(n))
        m.reserve(n)
        m.same(c)
        start = [0]
        for x in n:
            start.append(start[-1] + x)
        c.advance(i32(start))
        for b, x in enumerate(n):
            m.seq_len[b] += x if m.seq_len[b] >= 0 else 0
        m.same(c)

    grow([5 * P + 3, 0, P, 1, 0, 0])
    grow([1, 0, 1, P, 0, 0])
    c.fork(i32([0, 3, 0]), i32([4, 1, 5]))
    m.fork([0, 3, 0], [4, 1, 5])
    m.same(c)
    grow([P, 1, 0, 2 * P, 3, 1])
    c.free(i32([0, 1]))
    m.free([0, 1])
    m.same(c)
    c.reserve()  # one more for every slot in use
    m.reserve([0, 0] + [1] * 4)
    m.same(c)
    c.compact()
    m.compact()
    m.same(c)
    grow([3 * P, 2, 0, 1, 1, 2 * P])
    for w, s in ((2 * P, 0), (P + 3, 1), (1, 0)):
        c.trim(w, s)
        m.trim(w, s)
        m.same(c)
    c.compact()
    m.compact()
    m.same(c)
    c.compact()  # nothing left to move
    m.same(c)
    live = [b for b in range(6) if int(m.seq_len[b]) >= 0]
    c.free(i32(live))
    m.free(live)
    m.same(c)
    c.check()
    assert int(c.k_ref.sum()) == 0 and int(c.v_ref.sum()) == 0


def test_many_pages_and_slots(cuda_lib):
    """Pools longer than one pass of the bookkeeping block, more slots than its threads."""
    c = make(slots=1500, heads=1, P=16, pages=20000, width=24, fox=False)
    m = Model(c)
    g = torch.Generator().manual_seed(1)
    n = torch.randint(0, 150, (1500,), generator=g).tolist()
    n[700:900] = [0] * 200
    c.reserve(i32(n))
    m.reserve(n)
    start = torch.tensor([0] + n).cumsum(0).int()
    c.advance(start.to(DEV))
    for b, x in enumerate(n):
        if m.seq_len[b] >= 0:
            m.seq_len[b] += x
    m.same(c)
    gone = [b for b in range(0, 1500, 3) if n[b]]
    c.free(i32(gone))
    m.free(gone)
    m.same(c)
    par = [b for b in range(1, 1500) if b % 3 == 1 and n[b]][:200]
    kids = [k for k in range(700, 900) if int(m.seq_len[k]) < 0][: len(par)]
    par = par[: len(kids)]
    c.fork(i32(par), i32(kids))
    m.fork(par, kids)
    m.same(c)
    c.compact()
    m.compact()
    m.same(c)
    c.check()


def test_refusals_leave_everything(cuda_lib):
    c = make(slots=4, pages=8, width=6)
    c.reserve(i32([40, 10, 0, 0]))
    c.advance(i32([0, 40, 50, 50, 50]))
    c.check()
    m = Model(c)
    P = c.page_size

    def refused(what, call):
        call()
        with pytest.raises(RuntimeError, match=what):
            c.check()
        m.same(c)

    refused("not enough free pages", lambda: c.reserve(i32([0, 0, 6 * P, 0])))
    refused("outgrow", lambda: c.reserve(i32([6 * P, 0, 0, 0])))
    refused("listed twice", lambda: c.fork(i32([0, 1]), i32([2, 2])))
    refused("in use", lambda: c.fork(i32([0]), i32([1])))
    refused("in use", lambda: c.fork(i32([0]), i32([0])))
    refused("empty", lambda: c.fork(i32([3]), i32([2])))
    refused("out of range", lambda: c.fork(i32([0]), i32([4])))
    refused("out of range", lambda: c.fork(i32([-1]), i32([2])))
    refused("not enough free pages", lambda: c.fork(i32([0, 0]), i32([2, 3])))
    refused("listed twice", lambda: c.free(i32([0, 0])))
    refused("empty", lambda: c.free(i32([2])))
    refused("out of range", lambda: c.free(i32([99])))
    refused("outgrow", lambda: c.advance(i32([0, 7 * P, 7 * P, 7 * P, 7 * P])))
    refused("q_start", lambda: c.advance(i32([0, -1, -1, -1, -1])))
    c.fork(i32([]), i32([]))
    c.free(i32([]))
    c.reserve(i32([0, 0, 0, -5]))
    m.same(c)
    # a parent whose table names a page that the pool has not
    c.k_table[1, 0] = 1000
    m.k_table[1, 0] = 1000
    refused("page-table", lambda: c.fork(i32([1]), i32([2])))


def test_captured_fork_reads_its_lists_at_replay(cuda_lib):
    c = make(slots=6)
    c.reserve(i32([50, 20, 0, 0, 0, 0]))
    c.advance(i32([0, 50, 70, 70, 70, 70, 70]))
    par, chi = i32([0]), i32([2])
    m = Model(c)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.fork(par, chi)
    m.same(c)
    for p, k in ((0, 2), (1, 5), (0, 3)):
        par.fill_(p)
        chi.fill_(k)
        g.replay()
        m.fork([p], [k])
        m.same(c)
    c.check()
