"""Measured cases of the paged serving operators of PaTH attention.

Two operators over one paged cache (keys in one pool of pages, values in another, a table of page
numbers per sequence slot for each):

* ``extend``: attention of new tokens (a prompt chunk, a few draft tokens or one token per sequence)
  over the cached ones.  The new tokens' transitions H = I - beta w w^T are applied to every cached key
  in place, the new keys and values are appended, and each new token attends to what it sees.
* ``pages``: a beam step (children forked from their parents, the parents freed) and the compaction
  of a pool with holes.

``own`` false computes the plain form (elementary torch operations in 32 bits), true calls the
framework.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _extend(name, dtype, d, hq, hkv, page, seqs, t_lo, t_hi, n_lo, n_hi, fox=False, window=0, sinks=0):
    c = dict(op="extend", dtype=dtype, d=d, hq=hq, hkv=hkv, page=page, seqs=seqs, t_lo=t_lo, t_hi=t_hi, n_lo=n_lo,
             n_hi=n_hi, fox=fox, window=window, sinks=sinks)
    return dict(c, name=name) if name else c


def _pages(name, op, dtype, d, hkv, page, seqs, t_lo, t_hi, children, fox=False):
    c = dict(op=op, dtype=dtype, d=d, hkv=hkv, page=page, seqs=seqs, t_lo=t_lo, t_hi=t_hi, children=children, fox=fox)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user, a short answer being written: latency of a single step
        _extend("token_one", "bf16", 64, 16, 16, 64, 1, 515, 515, 1, 1),
        # a server's ordinary step: a batch of conversations of very different lengths, grouped heads
        _extend("token_ragged", "bf16", 128, 32, 8, 64, 48, 1, 4096, 1, 1),
        # few long documents at head dim 64, every head its own keys
        _extend("token_long", "bf16", 64, 32, 32, 128, 4, 31000, 32768, 1, 1),
        # endless streams: forget gate, sliding window and first tokens kept, small pages
        _extend("token_window", "bf16", 64, 16, 16, 16, 24, 6000, 16384, 1, 1, fox=True, window=4096, sinks=4),
        # draft tokens of a small model checked at once
        _extend("draft_check", "bf16", 64, 16, 8, 32, 16, 2000, 8192, 8, 8),
        # a chunk of a prompt behind an earlier part of it
        _extend("prompt_chunk", "bf16", 64, 32, 32, 64, 1, 8000, 8000, 512, 512),
        # the largest: a long prompt's last chunks, grouped heads of dim 128
        _extend("prompt_long", "bf16", 128, 32, 8, 64, 1, 32768, 32768, 2048, 2048),
        # one prompt chunk in the same call as a batch of single tokens
        _extend("prompt_and_tokens", "bf16", 128, 16, 4, 64, 24, 100, 6000, 1, 700),
        # the exact mode, ragged prompt chunks with the forget gate
        _extend("chunk_exact_mode", "fp32", 64, 8, 8, 32, 3, 0, 1500, 5, 97, fox=True),
        # one conversation branched in two
        _pages("fork_one", "fork", "bf16", 64, 16, 64, 1, 300, 300, 1),
        # a beam step over a batch
        _pages("beam_step", "fork", "bf16", 64, 16, 64, 8, 1500, 4000, 4),
        # a pool with holes after a busy hour, made dense
        _pages("compact", "compact", "bf16", 128, 8, 64, 48, 500, 8000, 0, fox=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))))


def draw(rng: random.Random):
    dtype = "fp32" if rng.random() < 0.15 else "bf16"
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 16, 32] if d == 64 else [1, 2, 4, 8, 16])
    page = rng.choice([16, 32, 64, 128, 256])
    fox = rng.random() < 0.3
    kind = rng.choice(["token", "token", "draft", "chunk", "chunk", "mixed", "fork", "compact"])
    if kind in ("fork", "compact"):
        seqs = _log(rng, 1, 48)
        # at most 1 GB of cached keys and values
        t_hi = _log(rng, 16, max(16, min(16384, (1 << 30) // (seqs * hkv * d * 8))))
        return _pages(None, kind, dtype, d, hkv, page, seqs, max(1, int(t_hi * rng.random())), t_hi,
                      rng.choice([1, 2, 3, 4]) if kind == "fork" else 0, fox)
    g = rng.choice([1, 1, 2, 4, 8]) if hkv <= 8 else 1
    hq = hkv * g
    window, sinks = 0, 0
    if rng.random() < 0.25:
        window, sinks = _log(rng, 16, 8192), rng.choice([0, 1, 4, 70])
    if kind == "token":
        n_lo = n_hi = 1
        seqs = _log(rng, 1, 64)
    elif kind == "draft":
        n_lo, n_hi = 1, rng.randint(2, 16)
        seqs = _log(rng, 1, 32)
    elif kind == "chunk":
        n_hi = _log(rng, 17, 2048 if dtype == "bf16" else 300)
        n_lo = max(1, int(n_hi * rng.random()))
        seqs = _log(rng, 1, 4)
    else:
        n_lo, n_hi = 1, _log(rng, 33, 1024 if dtype == "bf16" else 200)
        seqs = _log(rng, 2, 32)
    # at most 1 GB of cached keys and values, and at most a quarter of the largest case's products
    t_hi = min(32768, (1 << 30) // (seqs * hkv * d * 8))
    t_hi = min(t_hi, int((6.0e10 if dtype == "bf16" else 4.0e9) / (seqs * n_hi * hq * d) * 2))
    t_hi = _log(rng, 1, max(t_hi, 64))
    return _extend(None, dtype, d, hq, hkv, page, seqs, int(t_hi * rng.random()), t_hi, n_lo, n_hi, fox, window, sinks)


def _spread(lo, hi, n, by):
    """n whole numbers over lo..hi, both ends among them (n > 1), in a scattered order that the case fixes."""
    if n == 1:
        return [hi]
    r = random.Random(by)
    v = [lo + (hi - lo) * i // (n - 1) for i in range(n)]
    r.shuffle(v)
    return v


def _lens(c):
    """Cached tokens of each sequence and (extend) its new ones."""
    t = _spread(c["t_lo"], c["t_hi"], c["seqs"], 1)
    if c["op"] != "extend":
        return t, None
    if c["n_hi"] > 64 and c["n_lo"] == 1 and c["seqs"] > 4:  # one prompt chunk among single tokens
        n = [1] * c["seqs"]
        n[c["seqs"] // 2] = c["n_hi"]
    else:
        n = _spread(c["n_lo"], c["n_hi"], c["seqs"], 2)
    return t, n


def _live(c, t, n):
    """Cached rows that some new token sees, and those that a later one still sees (they are rewritten)."""
    if not c["window"]:
        return t, t
    first = lambda p: min(t, max(c["sinks"], p - c["window"] + 1))  # noqa: E731
    s = min(t, c["sinks"])
    return s + t - max(s, first(t)), s + t - max(s, first(t + n))


def _pairs(c, t, n):
    """(query token, visible key) pairs."""
    w = c["window"]
    if not w:
        return n * t + n * (n + 1) // 2
    total = 0
    for i in range(n):
        p = t + i
        lo = max(0, p - w + 1)
        total += p + 1 - lo + min(c["sinks"], lo)
    return total


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    t, n = _lens(c)
    d, hkv = c["d"], c["hkv"]
    if c["op"] != "extend":
        k, v = _moved_pages(c)
        page = c["page"] * hkv * d * e
        counts = 4 * 2 * _pool_pages(c)  # every reference count is looked at
        return {"bytes": 2 * (k * page + v * (page + (c["page"] * hkv * 4 if c["fox"] else 0))) + counts, "flops": 0}
    hq = c["hq"]
    byts, fl = 0, 0
    for a, b in zip(t, n):
        seen, kept = _live(c, a, b)
        byts += hkv * (seen * (2 * d * e + (4 if c["fox"] else 0)) + kept * d * e)
        byts += b * (hq * 2 * d * e + hkv * (5 * d * e + 4 + (8 if c["fox"] else 0)))
        fl += 4 * hq * d * _pairs(c, a, b)
        fl += 2 * hkv * d * kept * min(2 * b, d)  # cached keys: two products with n columns, or one with d
        fl += hkv * 2 * b * min(b, 64) * d * 4 + hq * 2 * b * min(b, 64) * d * 2 + 2 * hq * b * d * max(0, b // 2)
    return {"bytes": byts, "flops": fl}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _moved_pages(c):
    """Key and value pages that a pages case copies (the case fixes them)."""
    t, _ = _lens(c)
    P = c["page"]
    if c["op"] == "fork":
        return sum(-(-x // P) for x in t) * c["children"], sum(1 for x in t if x % P) * c["children"]
    return tuple(sum(1 for p in used if p >= len(used)) for used in _placed(c))


def _placed(c):
    """Pages that a case's sequences hold in each pool, in table order: scattered, with holes."""
    t, n = _lens(c)
    need = sum(-(-(x + (n[i] if n else 0)) // c["page"]) for i, x in enumerate(t))
    total = _pool_pages(c)
    return random.Random(7).sample(range(total), need), random.Random(8).sample(range(total), need)


def _pool_pages(c):
    t, n = _lens(c)
    need = sum(-(-(x + (n[i] if n else 0)) // c["page"]) for i, x in enumerate(t))
    if c["op"] == "fork":
        return need + need * c["children"] + c["seqs"] + 3
    return need + (need if c["op"] == "compact" else need // 4) + 3


def prepare(case, seed):
    """The cache (pools, tables, counts) and the new tokens of a step, on the GPU."""
    c = case
    dev = "cuda"
    dt = DTYPES[c["dtype"]]
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 11)
    t, n = _lens(c)
    B, H, d, P = c["seqs"], c["hkv"], c["d"], c["page"]
    slots = B * (1 + c.get("children", 0)) if c["op"] == "fork" else B
    total = _pool_pages(c)
    need = [-(-(x + (n[i] if n else 0)) // P) for i, x in enumerate(t)]
    width = max(need) + 1

    def normal(*shape):
        out = torch.empty(*shape, dtype=dt, device=dev)
        return out.normal_(0.0, 1.0, generator=g)

    k_pool, v_pool = normal(total, H, P, d), normal(total, H, P, d)
    # tables, lengths and reference counts: one block of int32, in this order
    meta = torch.full((slots * (2 * width + 1) + 2 * total,), -1, dtype=torch.int32)
    kt, vt, sl, kr, vr = _views(meta, slots, width, total)
    kr.zero_()
    vr.zero_()
    kp, vp = _placed(c)
    at = 0
    for b in range(B):
        kt[b, : need[b]] = torch.tensor(kp[at : at + need[b]], dtype=torch.int32)
        vt[b, : need[b]] = torch.tensor(vp[at : at + need[b]], dtype=torch.int32)
        sl[b] = t[b]
        at += need[b]
    kr[torch.tensor(kp, dtype=torch.long)] = 1
    vr[torch.tensor(vp, dtype=torch.long)] = 1
    s = dict(case=c, k_pool=k_pool, v_pool=v_pool, meta0=meta.to(dev), meta=meta.to(dev), slots=slots, width=width, total=total)
    s["a_pool"] = None
    if c["fox"]:  # running sums of log sigmoid(N(2, 1)), as a sequence's earlier steps leave them
        a = torch.zeros(total, H, P, device=dev)
        for b in range(B):
            rows = need[b] * P
            f = torch.log(torch.sigmoid(torch.randn(rows, H, generator=g, device=dev, dtype=torch.float64) + 2.0))
            run_ = torch.cumsum(f, 0).float().reshape(need[b], P, H).permute(0, 2, 1)
            a[vt[b, : need[b]].to(dev).long()] = run_
        s["a_pool"] = a
    if c["op"] == "extend":
        N = sum(n)
        w = torch.randn(N, H, d, generator=g, device=dev)
        s["q"], s["k"], s["v"] = normal(N, c["hq"], d), normal(N, H, d), normal(N, H, d)
        s["w"] = (w / w.norm(dim=-1, keepdim=True)).to(dt)
        s["beta"] = 2.0 * torch.sigmoid(torch.randn(N, H, generator=g, device=dev))
        s["log_f"] = torch.log(torch.sigmoid(torch.randn(N, H, generator=g, device=dev) + 2.0)) if c["fox"] else None
        starts = [0]
        for x in n:
            starts.append(starts[-1] + x)
        s["q_start"] = torch.tensor(starts, dtype=torch.int32, device=dev)
        s["max_new"] = max(n)
    elif c["op"] == "fork":
        kids = c["children"]
        s["parents"] = torch.tensor([b for b in range(B) for _ in range(kids)], dtype=torch.int32, device=dev)
        s["children"] = torch.arange(B, B * (1 + kids), dtype=torch.int32, device=dev)
        s["old"] = torch.arange(B, dtype=torch.int32, device=dev)
    if own:  # the handle that a serving program keeps: the tensors above under the framework's name
        from softmax_attention_chunk_gb300.paged import PagedCache

        kt, vt, sl, kr, vr = _views(s["meta"], slots, width, total)
        s["cache"] = PagedCache.from_tensors(k_pool, v_pool, kt, vt, sl, kr, vr, a_pool=s["a_pool"])
    return s


def _views(meta, slots, width, total):
    """Key table, value table, lengths, key and value reference counts inside the block."""
    a = slots * width
    return (meta[:a].view(slots, width), meta[a : 2 * a].view(slots, width), meta[2 * a : 2 * a + slots],
            meta[2 * a + slots : 2 * a + slots + total], meta[2 * a + slots + total :])


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(state):
    s = state
    c = s["case"]
    if c["op"] == "extend":
        if own:
            o = s["cache"].extend(s["q"], s["k"], s["v"], s["w"], s["beta"], log_f=s["log_f"], q_start=s["q_start"],
                                  max_new=s["max_new"], scale=1.0 / math.sqrt(c["d"]), window=c["window"],
                                  sinks=c["sinks"])
        else:
            o = _extend_plain(s)
        out = dict(o=o, k=s["k_pool"], v=s["v_pool"])
    else:
        s["meta"].copy_(s["meta0"])  # the tables as they were before the step
        if own:
            if c["op"] == "fork":
                s["cache"].fork(s["parents"], s["children"])
                s["cache"].free(s["old"])
            else:
                s["cache"].compact()
        elif c["op"] == "fork":
            _fork_plain(s)
        else:
            _compact_plain(s)
        out = dict(meta=s["meta"], k=s["k_pool"], v=s["v_pool"])
    if c["fox"]:
        out["a"] = s["a_pool"]
    return out


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _unit_lower_inverse(L):
    """(I + L)^-1 of strictly lower triangular L [..., n, n], n a power of two: blocks of one row are
    their own inverse, and two neighbours join into one of twice the size,
    [[A, 0], [B, C]]^-1 = [[A^-1, 0], [-C^-1 B A^-1, C^-1]]."""
    n = L.shape[-1]
    T = torch.eye(n, device=L.device, dtype=L.dtype).expand(L.shape).contiguous()
    size = 1
    while size < n:
        m = n // (2 * size)
        X = T.view(*L.shape[:-2], m, 2, size, m, 2, size)
        Y = L.view(*L.shape[:-2], m, 2, size, m, 2, size)
        i = torch.arange(m, device=L.device)
        A = X[..., i, 0, :, i, 0, :]
        Cc = X[..., i, 1, :, i, 1, :]
        Bb = Y[..., i, 1, :, i, 0, :]
        X[..., i, 1, :, i, 0, :] = -(Cc @ Bb @ A)
        size *= 2
    return T


def _extend_plain(s):
    c = s["case"]
    d, H, G, P, B = c["d"], c["hkv"], c["hq"] // c["hkv"], c["page"], c["seqs"]
    t, n = _lens(c)
    dev = s["q"].device
    kt, vt, sl, _, _ = _views(s["meta"], s["slots"], s["width"], s["total"])
    tmax, nmax = max(t), max(n)
    npad = 1 << (nmax - 1).bit_length()
    t0 = sl.long()
    q0 = s["q_start"].long()
    cnt = q0[1:] - q0[:-1]
    i = torch.arange(npad, device=dev)
    real = i[None, :] < cnt[:, None]  # [B, npad]
    tok = torch.where(real, q0[:-1, None] + i[None, :], 0)
    z = real[..., None, None]
    q = torch.where(z, s["q"][tok].float(), 0.0).view(B, npad, H, G, d).permute(0, 2, 3, 1, 4)  # [B, H, G, n, d]
    k, v, w = (torch.where(z, s[x][tok].float(), 0.0).permute(0, 2, 1, 3) for x in ("k", "v", "w"))  # [B, H, n, d]
    beta = torch.where(real[..., None], s["beta"][tok], 0.0).permute(0, 2, 1)[..., None]  # [B, H, n, 1]
    # the new tokens' transitions as one triangular system
    low = torch.tril(torch.ones(npad, npad, device=dev, dtype=torch.bool))
    strict = torch.tril(low, -1)
    U = _unit_lower_inverse(torch.where(strict, beta * (w @ w.transpose(-1, -2)), 0.0)) * beta.transpose(-1, -2)
    N2 = torch.where(strict, w @ k.transpose(-1, -2), 0.0)
    A = torch.where(low, q @ w.transpose(-1, -2)[:, :, None], 0.0) @ U[:, :, None]
    Z = q - A @ w[:, :, None]
    Snew = q @ k.transpose(-1, -2)[:, :, None] - A @ N2[:, :, None]
    knew = k - (U @ N2).transpose(-1, -2) @ w
    # the cached rows
    j = torch.arange(tmax, device=dev)
    have = j[None, :] < t0[:, None]  # [B, tmax]
    kpage = torch.where(have, kt[:, j // P].long(), 0)
    vpage = torch.where(have, vt[:, j // P].long(), 0)
    row = (j % P)[None, :].expand(B, tmax)
    zc = have[..., None, None]
    Kc = torch.where(zc, s["k_pool"][kpage, :, row].float(), 0.0).permute(0, 2, 1, 3)  # [B, H, t, d]
    Vc = torch.where(zc, s["v_pool"][vpage, :, row].float(), 0.0).permute(0, 2, 1, 3)
    scale = 1.0 / math.sqrt(d)
    pos = t0[:, None] + i[None, :]  # [B, npad]
    oldm = have[:, None, :].expand(B, npad, tmax)
    newm = low[None] & real[:, None, :]
    if c["window"]:
        W, S = c["window"], c["sinks"]
        oldm = oldm & ((j[None, None, :] > pos[:, :, None] - W) | (j[None, None, :] < S))
        newm = newm & ((pos[:, None, :] > pos[:, :, None] - W) | (pos[:, None, :] < S))
    Sc = Z @ Kc.transpose(-1, -2)[:, :, None] * scale  # [B, H, G, n, t]
    Snew = Snew * scale
    if c["fox"]:
        # sums of log f: differences of running sums in 64 bits
        lf = torch.where(real[..., None], s["log_f"][tok].double(), 0.0).permute(0, 2, 1)
        cum = torch.cumsum(lf, -1)  # [B, H, n]
        aj = torch.where(have[..., None], s["a_pool"][vpage, :, row], 0.0).permute(0, 2, 1).double()  # [B, H, t]
        last = torch.where(t0 > 0, t0 - 1, 0)
        a0 = torch.where((t0 > 0)[:, None], s["a_pool"][vt[torch.arange(B, device=dev), last // P].clamp(min=0).long(), :, last % P], 0.0).double()
        Sc = Sc + ((a0[..., None] + cum)[..., None] - aj[:, :, None, :]).float()[:, :, None]
        Snew = Snew + (cum[..., None] - cum[:, :, None, :]).float()[:, :, None]
    Sc = torch.where(oldm[:, None, None], Sc, -math.inf)
    Snew = torch.where(newm[:, None, None], Snew, -math.inf)
    top = Snew.amax(-1, keepdim=True)
    if tmax:
        top = torch.maximum(top, Sc.amax(-1, keepdim=True))
    top = torch.where(torch.isfinite(top), top, 0.0)
    Pc, Pn = torch.exp(Sc - top), torch.exp(Snew - top)
    den = Pc.sum(-1, keepdim=True) + Pn.sum(-1, keepdim=True)
    o = (Pc @ Vc[:, :, None] + Pn @ v[:, :, None]) / den  # [B, H, G, n, d]
    out = torch.empty_like(s["q"])
    out[tok[real]] = o.permute(0, 3, 1, 2, 4).reshape(B, npad, H * G, d)[real].to(out.dtype)
    # cached keys that a later token sees, moved past the new tokens
    keep = have
    if c["window"]:
        keep = have & ((j[None, :] > (t0 + cnt)[:, None] - c["window"]) | (j[None, :] < c["sinks"]))
    Kn = Kc - ((Kc @ w.transpose(-1, -2)) @ U.transpose(-1, -2)) @ w
    s["k_pool"][kpage[keep], :, row[keep]] = Kn.permute(0, 2, 1, 3)[keep].to(s["k_pool"].dtype)
    # appended rows
    seq = torch.arange(B, device=dev)[:, None].expand(B, npad)[real]
    p = pos[real]
    kp, vp = kt[seq, p // P].long(), vt[seq, p // P].long()
    s["k_pool"][kp, :, p % P] = knew.permute(0, 2, 1, 3)[real].to(s["k_pool"].dtype)
    s["v_pool"][vp, :, p % P] = s["v"][tok[real]]
    if c["fox"]:
        s["a_pool"][vp, :, p % P] = (a0[..., None] + cum).float().permute(0, 2, 1)[real]
    return out


def _lowest_free(ref, count):
    return torch.argsort((ref > 0).to(torch.int8), stable=True)[:count]


def _fork_plain(s):
    c = s["case"]
    P, kids = c["page"], c["children"]
    t, _ = _lens(c)
    kt, vt, sl, kr, vr = _views(s["meta"], s["slots"], s["width"], s["total"])
    dev = kt.device
    par, chi = s["parents"].long(), s["children"].long()
    plen = sl[par].long()
    col = torch.arange(s["width"], device=dev)
    has = col[None, :] < ((plen + P - 1) // P)[:, None]  # [children, width]
    full = col[None, :] < (plen // P)[:, None]
    part = has & ~full
    moved = sum(-(-x // P) for x in t) * kids
    dst = _lowest_free(kr, moved)
    src = kt[par][has].long()
    s["k_pool"][dst] = s["k_pool"][src]
    kr[dst] = 1
    rows = torch.full_like(kt[par], -1)
    rows[has] = dst.to(torch.int32)
    kt[chi] = rows
    shared = vt[par][full].long()
    vr.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    moved = sum(1 for x in t if x % P) * kids
    dst = _lowest_free(vr, moved)
    src = vt[par][part].long()
    s["v_pool"][dst] = s["v_pool"][src]
    if c["fox"]:
        s["a_pool"][dst] = s["a_pool"][src]
    vr[dst] = 1
    rows = torch.where(full, vt[par], -1)
    rows[part] = dst.to(torch.int32)
    vt[chi] = rows
    sl[chi] = sl[par]
    # the parents leave
    old = s["old"].long()
    kr[kt[old][kt[old] >= 0].long()] = 0
    gone = vt[old][vt[old] >= 0].long()
    vr.index_add_(0, gone, -torch.ones_like(gone, dtype=torch.int32))
    kt[old] = -1
    vt[old] = -1
    sl[old] = -1


def _dense(table, ref, pools):
    """Used pages above the number of used ones move into the holes below it, both in rising order."""
    used = ref > 0
    count = used.sum()
    index = torch.arange(ref.numel(), device=ref.device)
    src = index[used & (index >= count)]
    dst = index[~used & (index < count)]
    for p in pools:
        p[dst] = p[src]
    to = index.clone()
    to[src] = dst
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table))
    ref[dst] = ref[src]
    ref[src] = 0


def _compact_plain(s):
    kt, vt, sl, kr, vr = _views(s["meta"], s["slots"], s["width"], s["total"])
    _dense(kt, kr, [s["k_pool"]])
    _dense(vt, vr, [s["v_pool"]] + ([s["a_pool"]] if s["case"]["fox"] else []))


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    """One token after the other, as the definition says: every key so far is multiplied by the
    token's H = I - beta w w^T, the token's own key is added, the token attends."""
    c = case
    s = prepare(c, seed)
    if c["op"] != "extend":
        return None  # copies and whole numbers: nothing is computed
    t, n = _lens(c)
    if sum(n) > 6000:
        return None
    H, G, P, d = c["hkv"], c["hq"] // c["hkv"], c["page"], c["d"]
    kt, vt, _, _, _ = _views(s["meta"], s["slots"], s["width"], s["total"])
    kt, vt = kt.cpu().long(), vt.cpu().long()
    o = torch.zeros(sum(n), H, G, d, dtype=torch.float64, device="cuda")
    k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
    a_pool = s["a_pool"].double() if c["fox"] else None
    at = 0
    for b in range(c["seqs"]):
        T, N = t[b], n[b]
        p = torch.arange(T + N)
        kp, vp, r = kt[b, p // P].cuda(), vt[b, p // P].cuda(), (p % P).cuda()
        K = k_pool[kp, :, r].transpose(0, 1).contiguous()  # [H, T + N, d]
        V = v_pool[vp, :, r].transpose(0, 1).contiguous()
        V[:, T:] = s["v"][at : at + N].double().transpose(0, 1)
        F = None
        if c["fox"]:
            F = a_pool[vp, :, r].transpose(0, 1).contiguous()
        p = p.cuda()
        for x in range(N):
            u = at + x
            live = T + x + 1
            w, be = s["w"][u].double(), s["beta"][u].double()  # [H, d], [H]
            old = K[:, : live - 1]
            old -= (old @ w[:, :, None]) * (be[:, None] * w)[:, None, :]
            K[:, live - 1] = s["k"][u].double()
            lg = (s["q"][u].double().view(H, G, d) @ K[:, :live].transpose(1, 2)) / math.sqrt(d)
            if c["fox"]:
                before = F[:, live - 2] if live > 1 else torch.zeros(H, dtype=torch.float64, device="cuda")
                F[:, live - 1] = before + s["log_f"][u].double()
                lg += (F[:, live - 1 : live] - F[:, :live])[:, None, :]
            if c["window"]:
                hidden = (p[:live] <= live - 1 - c["window"]) & (p[:live] >= c["sinks"])
                lg.masked_fill_(hidden[None, None], -math.inf)
            o[u] = torch.softmax(lg, -1) @ V[:, :live]
        write = torch.ones(T + N, dtype=torch.bool, device="cuda")
        if c["window"]:
            write = (p > T + N - c["window"]) | (p < c["sinks"]) | (p >= T)
        k_pool[kp[write], :, r[write]] = K[:, write].transpose(0, 1)
        v_pool[vp[T:], :, r[T:]] = V[:, T:].transpose(0, 1)
        if c["fox"]:
            a_pool[vp[T:], :, r[T:]] = F[:, T:].transpose(0, 1)
        at += N
    out = dict(o=o.view(sum(n), H * G, d), k=k_pool, v=v_pool)
    if c["fox"]:
        out["a"] = a_pool
    return out
