"""Plain 64-bit form of the paged operators for the tests, from their definitions (CPU, one token after the
other), a builder of scattered caches, and the tolerances."""
import math

import torch

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}  # half a step of each type


def make_case(dtype, d, hq, hkv, page, t, n, fox=False, seed=0, slack=3, width_slack=1, nan_fill=True):
    """Pools with scattered pages for sequences of t cached tokens (t < 0: an empty slot) and packed new tokens, n
    each.  Pool rows that hold no cached token are NaN (nan_fill): nothing may read them."""
    g = torch.Generator().manual_seed(1000003 * seed + 17)
    dt = DT[dtype]
    B = len(t)
    need = [0 if x < 0 else -(-(x + m) // page) for x, m in zip(t, n)]
    total = sum(need) + slack
    width = max(need + [1]) + width_slack
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    fill = float("nan") if nan_fill else 0.0
    c = dict(dtype=dtype, d=d, hq=hq, hkv=hkv, page=page, t=list(t), n=list(n), fox=fox,
             k_pool=torch.full((total, hkv, page, d), fill, dtype=dt), v_pool=torch.full((total, hkv, page, d), fill, dtype=dt),
             a_pool=torch.full((total, hkv, page), fill) if fox else None,
             k_table=torch.full((B, width), -1, dtype=torch.int32), v_table=torch.full((B, width), -1, dtype=torch.int32),
             seq_len=torch.tensor(t, dtype=torch.int32), k_ref=torch.zeros(total, dtype=torch.int32),
             v_ref=torch.zeros(total, dtype=torch.int32))
    kp, vp = torch.randperm(total, generator=g), torch.randperm(total, generator=g)
    at = 0
    for b in range(B):
        c["k_table"][b, : need[b]] = kp[at : at + need[b]].int()
        c["v_table"][b, : need[b]] = vp[at : at + need[b]].int()
        c["k_ref"][kp[at : at + need[b]]] = 1
        c["v_ref"][vp[at : at + need[b]]] = 1
        at += need[b]
        if t[b] > 0:
            pos = torch.arange(t[b])
            c["k_pool"][c["k_table"][b, pos // page].long(), :, pos % page] = rnd(t[b], hkv, d).to(dt)
            c["v_pool"][c["v_table"][b, pos // page].long(), :, pos % page] = rnd(t[b], hkv, d).to(dt)
            if fox:
                a = torch.cumsum(torch.log(torch.sigmoid(rnd(t[b], hkv).double() + 2)), 0).float()
                c["a_pool"][c["v_table"][b, pos // page].long(), :, pos % page] = a
    N = sum(n)
    w = rnd(N, hkv, d)
    c.update(q=rnd(N, hq, d).to(dt), k=rnd(N, hkv, d).to(dt), v=rnd(N, hkv, d).to(dt),
             w=(w / w.norm(dim=-1, keepdim=True)).to(dt), beta=2 * torch.sigmoid(rnd(N, hkv)),
             log_f=torch.log(torch.sigmoid(rnd(N, hkv) + 2)) if fox else None)
    s = [0]
    for m in n:
        s.append(s[-1] + m)
    c["q_start"] = torch.tensor(s, dtype=torch.int32)
    return c


def extend_ref(c, scale, window=0, sinks=0):
    """(o, A, k_pool, v_pool, a_pool) in 64 bits; A = sum_j p_j |v_j|, the scale of o's errors."""
    H, G, d, P = c["hkv"], c["hq"] // c["hkv"], c["d"], c["page"]
    N = c["q"].shape[0]
    o = torch.zeros(N, H, G, d, dtype=torch.float64)
    A = torch.zeros_like(o)
    kp, vp = c["k_pool"].double(), c["v_pool"].double()
    ap = c["a_pool"].double() if c["fox"] else None
    for b, (T, n) in enumerate(zip(c["t"], c["n"])):
        if T < 0 or n == 0:
            continue
        q0 = int(c["q_start"][b])
        pos = torch.arange(T + n)
        kt, vt = c["k_table"][b, pos // P].long(), c["v_table"][b, pos // P].long()
        K = torch.nan_to_num(kp[kt, :, pos % P]).transpose(0, 1).clone()
        V = torch.nan_to_num(vp[vt, :, pos % P]).transpose(0, 1).clone()
        a = torch.nan_to_num(ap[vt, :, pos % P]).transpose(0, 1).clone() if c["fox"] else None
        V[:, T:] = c["v"][q0 : q0 + n].double().transpose(0, 1)
        for i in range(n):
            u, p = q0 + i, T + i
            w, be = c["w"][u].double(), c["beta"][u].double().clamp(0, 2)
            K[:, :p] -= (K[:, :p] @ w[:, :, None]) * (be[:, None] * w)[:, None]
            K[:, p] = c["k"][u].double()
            s = (c["q"][u].double().view(H, G, d) @ K[:, : p + 1].transpose(1, 2)) * scale
            if c["fox"]:
                a[:, p] = (a[:, p - 1] if p else 0.0) + c["log_f"][u].double()
                s = s + (a[:, p, None] - a[:, : p + 1])[:, None]
            if window:
                j = pos[: p + 1]
                s.masked_fill_(((j <= p - window) & (j >= sinks))[None, None], -math.inf)
            pr = torch.softmax(s, -1)
            o[u] = pr @ V[:, : p + 1]
            A[u] = pr @ V[:, : p + 1].abs()
        keep = torch.ones(T + n, dtype=torch.bool)
        if window:
            keep = (pos > T + n - window) | (pos < sinks) | (pos >= T)
        kp[kt[keep], :, (pos % P)[keep]] = K[:, keep].transpose(0, 1)
        vp[vt[T:], :, (pos % P)[T:]] = V[:, T:].transpose(0, 1)
        if c["fox"]:
            ap[vt[T:], :, (pos % P)[T:]] = a[:, T:].transpose(0, 1)
    return o.view(N, H * G, d), A.view(N, H * G, d), kp, vp, ap


def check_extend(c, got, ref, scale, tokens=None, passes=1):
    """Compares o and the pools.  Tolerances, with u half a step of the storage type (bf16: products of bf16
    and TF32 operands, u_t = 2^-11 TF32's half step; fp32: u_t = u):
      o: the output's own rounding u |o|; the probabilities' rounding u A; scores off by at most
         e = scale (u + 4 u_t) |z| |k| (z rounded once; four chained products), which moves o by at most 2 e A;
         fp32 adds the sums of about d + 64 terms and ex2's 2^-22: 256 u in place of the u's.
      norms: roundings are independent, so the 2-norm of the error stays below 2 u |o| (three of them, rms u at
         most each) and of a key row below u |k| + 2 u_t |k_before| (one rounding, two chained products).
    passes: a bf16 call carries the keys over 4096 tokens of a slot at a time, so that many times are the keys rounded
    and the chained products behind them made: e's and the key rows' terms take that factor; two passes make the
    independent roundings of o four, still 2 u |o|."""
    assert passes in (1, 2)
    dt = c["dtype"]
    u = U[dt]
    o, A, kp, vp, ap = ref
    x = got["o"].double()
    sel = slice(None) if tokens is None else tokens
    assert torch.isfinite(x[sel]).all()
    knorm = max(float(torch.nan_to_num(c["k_pool"].double()).norm(dim=-1).max()), float(c["k"].double().norm(dim=-1).max()))
    zk = scale * float(c["q"].double().norm(dim=-1).max()) * knorm
    if dt == "bf16":
        e = passes * (u + 4 * 2.0 ** -11) * zk
        bound = u * o.abs() + (u + 2 * e) * A + 1e-30
        fro = 2 * u
        kfro = passes * (u + 2 * 2.0 ** -11)
    else:
        e = 256 * u * max(1.0, zk)
        bound = 256 * u * o.abs() + (256 * u + 2 * e) * A + 1e-30
        fro = 256 * u
        kfro = 64 * u
    err = (x - o).abs()
    assert (err[sel] <= bound[sel]).all(), float((err / bound)[sel].max())
    if o[sel].numel():
        rel = float((x - o)[sel].norm() / o[sel].norm())
        assert rel <= fro, rel
    k = got["k"].double()
    same = torch.isnan(kp)
    assert torch.equal(torch.isnan(k), same)
    k, kr = torch.where(same, 0.0, k), torch.where(same, 0.0, kp)
    rel = float((k - kr).norm() / max(float(kr.norm()), 1e-30))
    assert rel <= kfro, rel
    big = float(kr.norm(dim=-1).max()) if kr.numel() else 0.0
    assert float((k - kr).abs().max()) <= passes * (u + 8 * (2.0 ** -11 if dt == "bf16" else 16 * u)) * max(big, 1.0)
    assert torch.equal(torch.isnan(got["v"]), torch.isnan(vp))
    assert torch.equal(torch.nan_to_num(got["v"].double()), torch.nan_to_num(vp))
    if c["fox"]:
        assert torch.equal(torch.isnan(got["a"]), torch.isnan(ap))
        a, ar = torch.nan_to_num(got["a"].double()), torch.nan_to_num(ap)
        assert float(((a - ar).abs() - 8 * 2.0 ** -24 * ar.abs()).max()) <= 1e-6
