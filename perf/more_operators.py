"""Measured cases of linear attention, of draft verification and of a step's plan.

Four operators:

* ``train``: linear attention with a decay per head over whole sequences, forward and backward;
* ``linear``: the same over a cache of states: prompts, draft tokens or single tokens, packed;
* ``verify``: drafted tokens checked against the target's probabilities, and the next token drawn;
* ``plan``: pages, packing and row maps of a step from the slots' numbers of new tokens.

``own`` false computes the plain form (elementary torch operations in 32 bits, 64 where 32 lose what
matters), true calls the framework.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _case(name, **c):
    return dict(c, name=name) if name else c


def _train(name, dtype, d, batch, hq, hkv, length):
    return _case(name, op="train", dtype=dtype, d=d, batch=batch, hq=hq, hkv=hkv, length=length)


def _linear(name, dtype, d, hq, hkv, slots, n_lo, n_hi, update=True):
    return _case(name, op="linear", dtype=dtype, d=d, hq=hq, hkv=hkv, slots=slots, n_lo=n_lo, n_hi=n_hi, update=update)


def _verify(name, dtype, vocab, slots, n_lo, n_hi, draft=True, noise=0.5):
    return _case(name, op="verify", dtype=dtype, vocab=vocab, slots=slots, n_lo=n_lo, n_hi=n_hi, draft=draft, noise=noise)


def _plan(name, page, slots, t_lo, t_hi, n_lo, n_hi, source=False):
    return _case(name, op="plan", page=page, slots=slots, t_lo=t_lo, t_hi=t_hi, n_lo=n_lo, n_hi=n_hi, source=source)


def listed():
    return [
        # a check of a model in the exact mode: one short ragged sequence
        _train("train_exact_mode", "fp32", 64, 1, 8, 8, 333),
        # a training step's layer: the benchmark's heads and length, a part of its batch
        _train("train_ordinary", "bf16", 64, 8, 32, 32, 4096),
        # the largest: long sequences, grouped heads of dim 128
        _train("train_long_grouped", "bf16", 128, 2, 32, 8, 8192),
        # one user, a short answer being written: latency of a single step
        _linear("linear_token_one", "bf16", 64, 16, 16, 1, 1, 1),
        # a server's ordinary step: one token for each of a batch of conversations
        _linear("linear_tokens", "bf16", 128, 32, 32, 64, 1, 1),
        # draft tokens of a small model looked at before they are accepted
        _linear("linear_drafts", "bf16", 128, 16, 8, 48, 2, 9, update=False),
        # one prompt chunk in the same call as a batch of single tokens
        _linear("linear_prompt_and_tokens", "bf16", 128, 16, 4, 24, 1, 700),
        # a long prompt's last part
        _linear("linear_prompt_long", "bf16", 64, 32, 32, 1, 16384, 16384),
        # one user's drafts checked
        _verify("verify_one", "fp32", 32000, 1, 5, 5),
        # a batch's drafts checked over a large vocabulary
        _verify("verify_batch", "fp32", 131072, 64, 2, 9),
        # single tokens of a batch of conversations
        _plan("plan_tokens", 64, 48, 1, 4096, 1, 1),
        # prompts of very different lengths, with the accepted drafts' rows of the packing before
        _plan("plan_prompts", 16, 256, 0, 8000, 0, 500, source=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))))


def draw(rng: random.Random):
    dtype = "fp32" if rng.random() < 0.2 else "bf16"
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24, 32] if d == 64 else [1, 2, 3, 4, 5, 8, 12, 16])
    g = rng.choice([1, 1, 2, 3, 4, 8]) if hkv <= 8 else 1
    kind = rng.choice(["train", "train", "train", "token", "draft", "prompt", "mixed", "verify", "verify", "plan"])
    if kind == "train":
        batch = rng.choice([1, 1, 2, 3, 4, 8])
        most = (1 << (26 if dtype == "bf16" else 23)) // (batch * hkv * g * d)  # elements of q
        return _train(None, dtype, d, batch, hkv * g, hkv, _log(rng, 1, max(64, min(16384, most))))
    if kind == "verify":
        vocab, slots = _log(rng, 1000, 200000), _log(rng, 1, 64)
        n_hi = rng.randint(1, 9)
        while slots > 1 and slots * n_hi * vocab > 64 * 6 * 131072:
            slots -= 1
        return _verify(None, dtype, vocab, slots, rng.randint(1, n_hi), n_hi, rng.random() < 0.75, rng.choice([0.1, 0.5, 2.0]))
    if kind == "plan":
        slots = _log(rng, 1, 256)
        t_hi, n_hi = _log(rng, 1, 8000), rng.choice([1, 1, rng.randint(2, 16), _log(rng, 17, 500)])
        return _plan(None, rng.choice([16, 32, 64, 128, 256]), slots, int(t_hi * rng.random()), t_hi,
                     1 if n_hi == 1 else int(n_hi * rng.random()), n_hi, rng.random() < 0.5)
    if kind == "token":
        return _linear(None, dtype, d, hkv * g, hkv, _log(rng, 2, 100), 1, 1)
    if kind == "draft":
        n_hi = rng.randint(2, 16)
        return _linear(None, dtype, d, hkv * g, hkv, _log(rng, 1, 48), rng.randint(1, n_hi), n_hi, rng.random() < 0.5)
    slots = _log(rng, 1, 4) if kind == "prompt" else _log(rng, 5, 32)
    most = (1 << (24 if dtype == "bf16" else 21)) // (slots * hkv * g * d)  # elements of q, were every slot's prompt the longest
    n_hi = _log(rng, 66, max(100, min(16384, most)))
    return _linear(None, dtype, d, hkv * g, hkv, slots, 1 if kind == "mixed" else max(1, int(n_hi * rng.random())), n_hi)


def _spread(lo, hi, n, by):
    """n whole numbers over lo..hi, both ends among them (n > 1), in a scattered order that the case fixes."""
    if n == 1:
        return [hi]
    r = random.Random(by)
    v = [lo + (hi - lo) * i // (n - 1) for i in range(n)]
    r.shuffle(v)
    return v


def _new(c):
    """New tokens of each slot."""
    if c["n_hi"] > 64 and c["n_lo"] == 1 and c["slots"] > 4:  # one prompt among single tokens
        n = [1] * c["slots"]
        n[c["slots"] // 2] = c["n_hi"]
        return n
    return _spread(c["n_lo"], c["n_hi"], c["slots"], 2)


def _lens(c):
    return _spread(c["t_lo"], c["t_hi"], c["slots"], 1)


def work(case):
    c = case
    if c["op"] == "train":
        e = 2 if c["dtype"] == "bf16" else 4
        tokens = c["batch"] * c["length"]
        # q, do, o, dq and k, v, dk, dv once; states and their gradients: products with d x d
        return {"bytes": tokens * 4 * (c["hq"] + c["hkv"]) * c["d"] * e,
                "flops": tokens * 2 * c["d"] ** 2 * (4 * c["hq"] + 3 * c["hkv"])}
    n = _new(c)
    if c["op"] == "linear":
        e = 2 if c["dtype"] == "bf16" else 4
        d, live = c["d"], sum(1 for x in n if x)
        return {"bytes": live * c["hkv"] * d * d * (8 if c["update"] else 4) + sum(n) * 2 * (c["hq"] + c["hkv"]) * d * e,
                "flops": sum(n) * 2 * d * d * (c["hq"] + c["hkv"])}
    if c["op"] == "verify":
        e = 2 if c["dtype"] == "bf16" else 4
        rows = 2 if c["draft"] else 1
        return {"bytes": sum(n) * (8 + rows * e) + c["slots"] * (rows * c["vocab"] * e + 12), "flops": c["slots"] * 3 * c["vocab"]}
    k = _plan_sizes(c)
    # counts of the pools, table entries and counts of the pages given out, the maps
    return {"bytes": 2 * 4 * k["pages"] + 2 * 8 * k["fresh"] + c["slots"] * 16 + sum(n) * (24 if c["source"] else 20), "flops": 0}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _plan_sizes(c):
    t, n, P = _lens(c), _new(c), c["page"]
    held = [-(-x // P) for x in t]
    fresh = sum(-(-(x + y) // P) - h for x, y, h in zip(t, n, held))
    return dict(held=held, fresh=fresh, pages=sum(held) + fresh + fresh // 4 + 3,
                width=max(-(-(x + y) // P) for x, y in zip(t, n)) + 1)


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 23)
    return g


def _starts(n):
    out = [0]
    for x in n:
        out.append(out[-1] + x)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _decays(heads):
    """log of the decay per token: from almost 1/2 to almost 1, a power of two apart."""
    h = torch.arange(1, heads + 1, dtype=torch.float64)
    return (-torch.exp2(-8.0 * h / heads)).float().cuda()


def prepare(case, seed):
    c = case
    g = _generator(seed)
    s = dict(case=c)
    if c["op"] in ("train", "linear"):
        dt, d = DTYPES[c["dtype"]], c["d"]

        def normal(*shape):
            return torch.empty(*shape, dtype=dt, device="cuda").normal_(0.0, 1.0, generator=g)

        s["log_decay"], s["scale"] = _decays(c["hkv"]), 1.0 / math.sqrt(d)
        if c["op"] == "train":
            s["q"] = normal(c["batch"], c["hq"], c["length"], d).requires_grad_()
            s["k"] = normal(c["batch"], c["hkv"], c["length"], d).requires_grad_()
            s["v"] = normal(c["batch"], c["hkv"], c["length"], d).requires_grad_()
            s["do"] = normal(c["batch"], c["hq"], c["length"], d)
            return s
        n = _new(c)
        N = sum(n)
        s["q"], s["k"], s["v"] = normal(N, c["hq"], d), normal(N, c["hkv"], d), normal(N, c["hkv"], d)
        s["q_start"], s["max_new"] = _starts(n), max(n)
        # states as long sequences leave them: products k v^T under the head's decay
        spread = 1.0 / torch.sqrt(1.0 - torch.exp(2.0 * s["log_decay"]))
        s["state"] = torch.randn(c["slots"], c["hkv"], d, d, generator=g, device="cuda") * spread[:, None, None]
        if own:
            from softmax_attention_chunk_gb300.linear import LinearCache

            s["cache"] = LinearCache.from_tensors(s["state"], dtype=dt)
        return s
    if c["op"] == "verify":
        n = _new(c)
        N, V, dt = sum(n), c["vocab"], DTYPES[c["dtype"]]
        logits = torch.randn(N, V, generator=g, device="cuda") * 2.5
        s["target"] = torch.softmax(logits, -1).to(dt)
        # a draft model near the target: draft row i is where token i was drawn, target row i - 1 where it is checked
        near = torch.roll(logits, 1, 0) + c["noise"] * torch.randn(N, V, generator=g, device="cuda")
        draft = torch.softmax(near, -1).to(dt)
        s["tokens"] = torch.argmax(draft.float() / torch.empty(N, V, device="cuda").exponential_(generator=g), -1).to(torch.int32)
        s["draft"] = draft if c["draft"] else None
        s["uniform"] = torch.rand(N, generator=g, device="cuda")
        s["q_start"], s["max_new"] = _starts(n), max(n)
        slots, P, width, pages = c["slots"], 16, 1, c["slots"]
        t, held = [1] * slots, [1] * slots
    else:
        t, n, P, slots = _lens(c), _new(c), c["page"], c["slots"]
        k = _plan_sizes(c)
        held, width, pages = k["held"], k["width"], k["pages"]
        s["n_new"] = torch.tensor(n, dtype=torch.int32, device="cuda")
        s["tokens"] = sum(n)
        s["fresh"] = k["fresh"]
        # where the packing before had each slot's tokens: as many as now and some that were rejected
        r = random.Random(seed)
        s["from_start"] = _starts([x + r.randint(0, 3) for x in n]) if c["source"] else None
    # tables, lengths and reference counts: one block of int32, in this order
    meta = torch.full((slots * (2 * width + 1) + 2 * pages,), -1, dtype=torch.int32)
    kt, vt, sl, kr, vr = _views(meta, slots, width, pages)
    kr.zero_()
    vr.zero_()
    by = random.Random(int(seed) + 5)
    for table, ref in ((kt, kr), (vt, vr)):
        got = torch.tensor(by.sample(range(pages), sum(held)), dtype=torch.int32)
        at = 0
        for b, x in enumerate(held):
            table[b, :x] = got[at : at + x]
            at += x
        ref[got.long()] = 1
    sl.copy_(torch.tensor(t, dtype=torch.int32))
    s["meta0"], s["meta"], s["sizes"] = meta.cuda(), meta.cuda(), (slots, width, pages)
    if own:
        from softmax_attention_chunk_gb300.paged import PagedCache

        kt, vt, sl, kr, vr = _views(s["meta"], slots, width, pages)
        pool = torch.zeros(2, pages, 1, P, 64, dtype=torch.bfloat16, device="cuda")
        s["cache"] = PagedCache.from_tensors(pool[0], pool[1], kt, vt, sl, kr, vr)
    return s


def _views(meta, slots, width, pages):
    """Key table, value table, lengths, key and value reference counts inside the block."""
    a = slots * width
    return (meta[:a].view(slots, width), meta[a : 2 * a].view(slots, width), meta[2 * a : 2 * a + slots],
            meta[2 * a + slots : 2 * a + slots + pages], meta[2 * a + slots + pages :])


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(state):
    s = state
    c = s["case"]
    if c["op"] == "train":
        if own:
            from softmax_attention_chunk_gb300.linear import linear_attention

            o = linear_attention(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"])
            dq, dk, dv = torch.autograd.grad(o, (s["q"], s["k"], s["v"]), s["do"])
            return dict(o=o.detach(), dq=dq, dk=dk, dv=dv)
        with torch.no_grad():
            return _train_plain(s)
    if c["op"] == "linear":
        if own:
            o = s["cache"].extend(s["q"], s["k"], s["v"], s["log_decay"], q_start=s["q_start"], max_new=s["max_new"],
                                  scale=s["scale"], update=c["update"])
        else:
            o = _linear_plain(s)
        return dict(o=o, state=s["state"]) if c["update"] else dict(o=o)
    if c["op"] == "verify":
        if own:
            keep, after = s["cache"].verify(s["target"], s["tokens"], s["uniform"], draft=s["draft"], q_start=s["q_start"],
                                            max_new=s["max_new"])
        else:
            keep, after = _verify_plain(s)
        return dict(keep=keep, after=after)
    s["meta"].copy_(s["meta0"])  # the tables as they were before the step
    if own:
        p = s["cache"].plan(s["n_new"], s["tokens"], from_start=s["from_start"])
        out = dict(q_start=p.q_start, slot=p.slot, position=p.position, k_row=p.k_row, v_row=p.v_row)
        if c["source"]:
            out["source"] = p.source
    else:
        out = _plan_plain(s)
    return dict(out, meta=s["meta"])


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
CHUNK = 64


def _whole_chunks(length):
    """The chunk of sequences of this length (at most 16 tokens are one), and the length filled up to a multiple of it."""
    chunk = CHUNK if length > 16 else length
    return chunk, -(-length // chunk) * chunk


def _attend(x, y, z, log_decay, chunk, state=None):
    """o_i = sum_{j <= i} g^(i-j) (x_i . y_j) z_j + g^(i+1) state^T x_i of x [..., L, d], y, z [..., L, d] with log_decay of
    their leading shape, in chunks: inside one as a masked product, before it through the d x d state at its start, which is
    a weighted sum of the earlier chunks' own.  L is a multiple of the chunk."""
    *_, L, d = y.shape
    C, n = chunk, L // chunk
    cut = lambda t: t.reshape(*t.shape[:-2], n, C, d)  # noqa: E731
    x, y, z = cut(x), cut(y), cut(z)
    l = log_decay.double()[..., None]
    i = torch.arange(C, device=x.device, dtype=torch.float64)
    apart = i[:, None] - i[None, :]
    inside = torch.where(apart >= 0, torch.exp(l[..., None] * apart.clamp(min=0)), 0.0).float()  # [..., C, C]
    o = ((x @ y.transpose(-1, -2)) * inside[..., None, :, :]) @ z
    own_state = (y * torch.exp(l * (C - 1 - i)).float()[..., None, :, None]).transpose(-1, -2) @ z  # [..., n, d, d]
    m = torch.arange(n, device=x.device, dtype=torch.float64)
    gap = m[:, None] - m[None, :] - 1
    over = torch.where(gap >= 0, torch.exp(l[..., None] * C * gap.clamp(min=0)), 0.0).float()  # [..., n, n]
    before = (over @ own_state.reshape(*own_state.shape[:-3], n, d * d)).view(own_state.shape)
    if state is not None:
        before = before + torch.exp(l * C * m).float()[..., None, None] * state[..., None, :, :]
    o = o + (x @ before) * torch.exp(l * (i + 1)).float()[..., None, :, None]
    return o.reshape(*o.shape[:-3], L, d)


def _padded(t, L):
    return torch.nn.functional.pad(t.float(), (0, 0, 0, L - t.shape[-2]))


def _train_plain(s):
    c = s["case"]
    L, H, G = c["length"], c["hkv"], c["hq"] // c["hkv"]
    chunk, full = _whole_chunks(L)
    grouped = lambda t: _padded(t, full).view(c["batch"], H, -1, full, c["d"])  # noqa: E731
    q, k, v, do = grouped(s["q"]), grouped(s["k"]), grouped(s["v"]), grouped(s["do"])
    kg, vg = k.expand_as(q), v.expand_as(q)
    ld = s["log_decay"][None, :, None].expand(c["batch"], H, G)
    back = lambda x, y, z: _attend(x.flip(-2), y.flip(-2), z.flip(-2), ld, chunk).flip(-2).sum(2)  # noqa: E731
    done = lambda t: (t[..., :L, :] * s["scale"]).reshape(c["batch"], -1, L, c["d"]).to(s["q"].dtype)  # noqa: E731
    return dict(o=done(_attend(q, kg, vg, ld, chunk)), dq=done(_attend(do, vg, kg, ld, chunk)), dk=done(back(vg, do, q)),
                dv=done(back(kg, q, do)))


def _linear_plain(s):
    c = s["case"]
    H, G, d = c["hkv"], c["hq"] // c["hkv"], c["d"]
    dev = s["q"].device
    chunk, full = _whole_chunks(s["max_new"])
    first = s["q_start"][:-1].long()
    count = s["q_start"][1:].long() - first
    i = torch.arange(full, device=dev)
    real = i[None, :] < count[:, None]
    tok = torch.where(real, first[:, None] + i[None, :], 0)

    def rows(t):  # [slots, heads, full, d]
        return torch.where(real[..., None, None], t[tok].float(), 0.0).permute(0, 2, 1, 3)

    q = rows(s["q"]).reshape(c["slots"], H, G, full, d)
    k, v = rows(s["k"]), rows(s["v"])
    ld = s["log_decay"][None, :].expand(c["slots"], H)
    o = _attend(q, k[:, :, None].expand_as(q), v[:, :, None].expand_as(q), ld[..., None].expand(c["slots"], H, G), chunk,
                s["state"][:, :, None]) * s["scale"]
    out = torch.empty_like(s["q"])
    out[tok[real]] = o.reshape(c["slots"], H * G, full, d).permute(0, 2, 1, 3)[real].to(out.dtype)
    if c["update"]:
        l = ld.double()[..., None]
        left = (count[:, None] - 1 - i[None, :]).clamp(min=0)[:, None, :].double()  # tokens after each
        k = k * torch.exp(l * left).float()[..., None]
        s["state"].copy_(s["state"] * torch.exp(l * count[:, None, None]).float()[..., None] + k.transpose(-1, -2) @ v)
    return out


def _verify_plain(s):
    c = s["case"]
    dev = s["target"].device
    first = s["q_start"][:-1].long()
    count = s["q_start"][1:].long() - first
    i = torch.arange(1, max(2, s["max_new"]), device=dev)
    real = i[None, :] < count[:, None]
    tok = torch.where(real, first[:, None] + i[None, :], 1 if s["tokens"].numel() > 1 else 0)
    x = s["tokens"][tok].long()
    p = s["target"][(tok - 1).clamp(min=0), x].double()
    q = s["draft"][tok, x].double() if s["draft"] is not None else torch.ones_like(p)
    good = real & (s["uniform"][tok].double() * q < p)
    keep = 1 + good.to(torch.int32).cumprod(1).sum(1)
    all_kept = keep == count
    row = first + keep - 1
    r = s["target"][row].double()
    at = torch.where(all_kept, row, row + 1)  # the rejected token's place
    if s["draft"] is not None:
        rest = (r - s["draft"][at].double()).clamp(min=0)
    else:
        rest = r.scatter(1, s["tokens"][at].long()[:, None], 0.0)
    rest = torch.where(all_kept[:, None] | (rest.sum(-1, keepdim=True) <= 0), r, rest)
    run_ = rest.cumsum(-1)
    goal = s["uniform"][first].double()[:, None] * run_[:, -1:]
    v = torch.arange(c["vocab"], device=dev)
    last = torch.where(rest > 0, v, -1).amax(-1)
    after = torch.minimum((run_ <= goal).sum(-1), last)
    return keep.to(torch.int32), after.to(torch.int32)


def _plan_plain(s):
    c = s["case"]
    P = c["page"]
    slots, width, pages = s["sizes"]
    kt, vt, sl, kr, vr = _views(s["meta"], slots, width, pages)
    n, t = s["n_new"].long(), sl.long()
    dev = n.device
    col = torch.arange(width, device=dev)
    lacks = (col[None, :] >= ((t + P - 1) // P)[:, None]) & (col[None, :] < ((t + n + P - 1) // P)[:, None])
    for table, ref in ((kt, kr), (vt, vr)):
        got = torch.argsort((ref > 0).to(torch.int8), stable=True)[: s["fresh"]]  # lowest free numbers first
        table[lacks] = got.to(torch.int32)
        ref[got] = 1
    start = torch.nn.functional.pad(n.cumsum(0), (1, 0))
    tok = torch.arange(s["tokens"], device=dev)
    slot = (tok[:, None] >= start[None, 1:]).sum(1)
    inside = tok - start[slot]
    pos = t[slot] + inside
    row = lambda table: table[slot, pos // P] * P + (pos % P).to(torch.int32)  # noqa: E731
    whole = lambda x: x.to(torch.int32)  # noqa: E731
    out = dict(q_start=whole(start), slot=whole(slot), position=whole(pos), k_row=row(kt), v_row=row(vt))
    if c["source"]:
        out["source"] = whole(s["from_start"][slot].long() + inside)
    return out


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    c = case
    if c["op"] not in ("train", "linear"):
        return None  # whole numbers
    s = prepare(c, seed)
    H, G, d = c["hkv"], c["hq"] // c["hkv"], c["d"]
    scale = s["scale"]
    decay = s["log_decay"].double()
    if c["op"] == "train":
        # every pair of tokens, a block of queries of one batch entry and key head at a time
        B, L = c["batch"], c["length"]
        q, do = (s[x].detach().view(B, H, G, L, d) for x in ("q", "do"))
        o, dq = torch.empty(2, B, H, G, L, d, dtype=torch.float64, device="cuda")
        dk, dv = torch.zeros(2, B, H, L, d, dtype=torch.float64, device="cuda")
        pos = torch.arange(L, device="cuda")
        for b in range(B):
            for h in range(H):
                k, v = s["k"][b, h].detach().double(), s["v"][b, h].detach().double()
                for lo in range(0, L, 1024):
                    hi = min(L, lo + 1024)
                    gap = pos[lo:hi, None] - pos[None, :hi]
                    weight = torch.where(gap >= 0, scale * torch.exp(decay[h] * gap.clamp(min=0)), 0.0)
                    qb, db = q[b, h, :, lo:hi].double(), do[b, h, :, lo:hi].double()
                    prob = torch.einsum("gid,jd->gij", qb, k[:hi]) * weight
                    grad = torch.einsum("gid,jd->gij", db, v[:hi]) * weight
                    o[b, h, :, lo:hi] = torch.einsum("gij,jd->gid", prob, v[:hi])
                    dq[b, h, :, lo:hi] = torch.einsum("gij,jd->gid", grad, k[:hi])
                    dv[b, h, :hi] += torch.einsum("gij,gid->jd", prob, db)
                    dk[b, h, :hi] += torch.einsum("gij,gid->jd", grad, qb)
        return dict(o=o.view(B, H * G, L, d), dq=dq.view(B, H * G, L, d), dk=dk, dv=dv)
    # one token after the other, all slots side by side
    first, n = s["q_start"][:-1].long(), _new(c)
    S = s["state"].double()
    keep = torch.exp(decay)[None, :, None, None]
    o = torch.zeros(sum(n), H * G, d, dtype=torch.float64, device="cuda")
    q, k, v = (s[x].double() for x in ("q", "k", "v"))
    count = torch.tensor(n)
    for i in range(max(n)):
        live = torch.nonzero(count > i)[:, 0].cuda()
        t = first[live] + i
        now = S[live] * keep + k[t][..., :, None] * v[t][..., None, :]
        S[live] = now
        o[t] = torch.einsum("bhgd,bhde->bhge", q[t].view(-1, H, G, d), now).reshape(-1, H * G, d) * scale
    return dict(o=o, state=S) if c["update"] else dict(o=o)
