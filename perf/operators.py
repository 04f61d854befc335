"""Sliding-window attention with sinks, decoding over a paged cache, and the cache's page operators:
what is measured, with plain forms in elementary torch operations.

An attention mask with a window of W tokens and the first `sinks` tokens kept visible: query i sees key j where
j <= i and (i - j < W or j < sinks).  A cache holds K and V in pages [P, Hkv, page, d]; row s of `table` lists the
pages of sequence s, `lens[s]` its tokens, `refs[p]` how many sequences hold page p (0: free).  Pages are handed
out lowest free number first.  Which lengths and pages a case has follows from the case alone; the seed draws the
values.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # the first prompt of a small model: one short row block, so launch latency is what counts
        dict(name="prefill short", op="prefill", dtype="bf16", B=1, H=2, Hkv=2, N=128, d=64, window=32, sinks=4, fix=1),
        # a long document read through a window at a 7B model's head layout, keys shared by groups of four heads
        dict(name="prefill long", op="prefill", dtype="bf16", B=1, H=32, Hkv=8, N=16384, d=128, window=4096, sinks=4, fix=1),
        # a fine-tuning step on an odd length in half precision, window and sinks off every tile border
        dict(name="train odd", op="train", dtype="fp16", B=2, H=6, Hkv=3, N=777, d=64, window=191, sinks=5, fix=0),
        # the attention of a GPT-2 small training step, with a window of a quarter of the context
        dict(name="train gpt2s", op="train", dtype="bf16", B=8, H=12, Hkv=12, N=1024, d=64, window=256, sinks=4, fix=1),
        # long-context training at a 7B model's head layout
        dict(name="train long", op="train", dtype="bf16", B=1, H=32, Hkv=8, N=8192, d=128, window=1024, sinks=4, fix=1),
        # one user chatting with a small model: a single short sequence
        dict(name="decode one", op="decode", dtype="bf16", S=1, H=12, Hkv=12, d=64, page=16, len=100, window=0, sinks=0),
        # a batch of ragged sequences behind a window, in half precision; some slots of the batch are empty
        dict(name="decode window", op="decode", dtype="fp16", S=33, H=32, Hkv=4, d=128, page=16, len=6000, window=1024, sinks=4),
        # a full batch at long context: what a server spends its time on
        dict(name="decode batch", op="decode", dtype="bf16", S=64, H=32, Hkv=8, d=128, page=64, len=16384, window=0, sinks=0),
        # the token that each sequence of a batch gained, written to one layer's pages
        dict(name="append step", op="append", dtype="bf16", S=64, Hkv=8, d=128, page=16, len=2000, new=1),
        # the prompts of nine requests, written to one layer's pages
        dict(name="append prompts", op="append", dtype="fp16", S=9, Hkv=8, d=128, page=64, len=4001, new=4001),
        # every sequence of a small batch branches (parallel samples of one prompt), and each branch gets room for more
        dict(name="pages branch", op="pages", step="branch", dtype="bf16", L=4, S=64, Hkv=8, d=128, page=16, len=1500, forks=24, new=20),
        # a third of a server's sequences end, and the pool is compacted over all layers
        dict(name="pages retire", op="pages", step="retire", dtype="bf16", L=8, S=48, Hkv=8, d=128, page=16, len=2048, forks=0, new=0),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of lo .. hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "train", "train", "decode", "decode", "append", "pages", "pages"])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), d=rng.choice([64, 128]))
    c["Hkv"] = rng.choice([1, 2, 3, 4, 8])
    if op in ("prefill", "train"):
        c["H"] = c["Hkv"] * rng.choice([1, 2, 4])
        most = 16384 if op == "prefill" else 8192
        c["N"] = _log(rng, 1, most)
        # window and work stay within the largest listed case of the same kind
        c["window"] = _log(rng, 1, min(c["N"] + 7, 4096 if op == "prefill" else 1024))
        c["sinks"] = rng.choice([0, 1, 4, 4, 16, 130])
        c["B"] = rng.randint(1, max(1, min(4, most // c["N"])))
        c["fix"] = rng.choice([0, 1, 1, 5])
        if c["H"] > 32:
            c["H"] = c["Hkv"]
    else:
        c["page"] = rng.choice([16, 16, 32, 64, 128])
        if op == "decode":
            c["H"] = c["Hkv"] * rng.choice([g for g in (1, 2, 4, 8, 16) if g * c["Hkv"] <= 32])
            c["len"] = _log(rng, 1, 32768)
            c["S"] = rng.randint(1, max(1, min(96, (1 << 20) // c["len"])))
            c["window"] = rng.choice([0, 0, _log(rng, 1, 4096)])
            c["sinks"] = rng.choice([0, 4, 20]) if c["window"] else 0
        elif op == "append":
            c["S"] = _log(rng, 1, 128)
            c["new"] = rng.choice([1, 1, _log(rng, 2, 4000)])
            c["new"] = min(c["new"], max(1, 36000 // c["S"]))
            c["len"] = c["new"] + _log(rng, 1, 2000)
        else:
            c["S"] = rng.randint(4, 64)
            c["len"] = _log(rng, 20, 2000)
            c["L"] = rng.randint(1, 6)
            c["step"] = rng.choice(["branch", "retire"])
            c["forks"] = rng.randint(1, c["S"] // 2) if c["step"] == "branch" else 0
            c["new"] = rng.randint(1, 70) if c["step"] == "branch" else 0
    return c


# ---------------------------------------------------------------------------------------------------------------
# lengths and pages of a case


def _rng(c):
    """Random numbers that follow from the case alone (its values, not its name)."""
    return random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))


def _step(c, step):
    return c.get("step") == step


def _lens(c):
    """The sequences' lengths: the longest is c["len"], the others are spread below it; a batch of over 8 has empty slots."""
    r = _rng(c)
    lens = [max(1, int(c["len"] * r.uniform(0.05, 1.0))) for _ in range(c["S"])]
    if c["op"] == "append":   # old tokens and new ones: `new` of them, or a ragged number up to it
        lens = [max(c["new"], n) for n in lens]
    lens[r.randrange(c["S"])] = c["len"]
    if c["op"] == "decode" and c["S"] > 8:
        for s in r.sample(range(c["S"]), c["S"] // 16):
            lens[s] = 0
    if _step(c, "branch"):   # the slots that the branches go to
        for s in range(c["S"] - c["forks"], c["S"]):
            lens[s] = 0
        lens[0] = c["len"]
    return lens


def _news(c):
    """How many tokens an append writes to each sequence."""
    r = _rng(c)
    return [c["new"] if c["new"] == 1 else max(1, int(c["new"] * r.uniform(0.2, 1.0))) for _ in range(c["S"])]


def _pages(c):
    """(pages in the pool, refs, table, lens): every sequence's pages, at random places in the pool."""
    lens = _lens(c)
    n = [-(-x // c["page"]) for x in lens]
    width = -(-(c["len"] + c.get("new", 0)) // c["page"]) + 1
    total = sum(n)
    spare = 8 + (2 * c["forks"] + len(lens) * (1 + c["new"] // c["page"]) if _step(c, "branch") else 0)
    if _step(c, "branch"):                                        # the branches' own pages, and room for new tokens
        spare += c["forks"] * width
    pool = total + spare + total // 8
    ids = list(range(pool))
    _rng(c).shuffle(ids)
    refs, table = [0] * pool, [[-1] * width for _ in lens]
    at = 0
    for s, k in enumerate(n):
        for i in range(k):
            table[s][i] = ids[at]
            refs[ids[at]] = 1
            at += 1
    return pool, refs, table, lens


def _forks(c):
    """(from, to): which sequence each branch copies; one sequence may have several branches."""
    r = _rng(c)
    live = c["S"] - c["forks"]
    return [r.randrange(live) for _ in range(c["forks"])], list(range(live, c["S"]))


def _ended(c):
    return _rng(c).sample(range(c["S"]), max(1, c["S"] // 3))


# ---------------------------------------------------------------------------------------------------------------
# inputs


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    st = {"case": c}
    if c["op"] in ("prefill", "train"):
        st["q"] = rand(c["B"], c["H"], c["N"], c["d"])
        st["k"] = rand(c["B"], c["Hkv"], c["N"], c["d"])
        st["v"] = rand(c["B"], c["Hkv"], c["N"], c["d"])
        # trained models put weight on the first tokens: their keys are longer
        st["k"][:, :, :c["sinks"]] *= 2
        if c["op"] == "train":
            st["do"] = rand(c["B"], c["H"], c["N"], c["d"])
        return st
    pool, refs, table, lens = _pages(c)
    st["table"], st["lens"] = ints(table), ints(lens)
    layers = (c["L"],) if "L" in c else ()
    st["k_pages"] = torch.empty(*layers, pool, c["Hkv"], c["page"], c["d"], dtype=dt, device=dev).normal_(generator=g)
    st["v_pages"] = torch.empty(*layers, pool, c["Hkv"], c["page"], c["d"], dtype=dt, device=dev).normal_(generator=g)
    if c["op"] == "decode":
        st["q"] = rand(c["S"], c["H"], c["d"])
        st["pages_most"] = max(-(-n // c["page"]) for n in lens)
    elif c["op"] == "append":
        news = _news(c)
        st["cu"] = ints([sum(news[:s]) for s in range(c["S"] + 1)])
        st["k"], st["v"] = rand(sum(news), c["Hkv"], c["d"]), rand(sum(news), c["Hkv"], c["d"])
    else:
        st["refs"] = ints(refs)
        st["now"] = tuple(torch.empty_like(st[n]) for n in ("refs", "table", "lens"))
        if _step(c, "branch"):
            src, dst = _forks(c)
            st["src"], st["dst"] = ints(src), ints(dst)
            st["new"] = ints([c["new"]] * c["S"])
        else:
            st["ended"] = ints(_ended(c))
    return st


# ---------------------------------------------------------------------------------------------------------------
# plain forms


def _blocks(c, device):
    """Queries in blocks, each with the keys that it can see: the sinks, then a stretch of window + block keys.
    Returns (block, blocks, key positions [blocks, J], which of them each query sees [blocks, block, J])."""
    n, w, sinks = c["N"], min(c["window"], c["N"]), min(c["sinks"], c["N"])
    block = min(n, max(64, min(1024, w)))
    nb = -(-n // block)
    i = torch.arange(nb * block, device=device).view(nb, block, 1)
    stretch = torch.arange(nb, device=device).view(nb, 1) * block - (w - 1) + torch.arange(w - 1 + block, device=device)
    sink = torch.arange(sinks, device=device).expand(nb, sinks)
    near = stretch.view(nb, 1, -1)
    see_near = (near >= 0) & (near < n) & (near <= i) & (i - near < w)
    far = sink.reshape(nb, 1, sinks)
    see_far = (far <= i) & (i - far >= w)
    pos = torch.cat([sink, stretch.clamp(0, n - 1)], 1)
    return block, nb, pos, torch.cat([see_far, see_near], 2)


def _attention(st, backward):
    c = st["case"]
    q, k, v = st["q"], st["k"], st["v"]
    B, H, N, d = q.shape
    Hkv = c["Hkv"]
    G = H // Hkv
    scale = d ** -0.5
    block, nb, pos, see = _blocks(c, q.device)
    see = see.repeat(1, G, 1)                                     # [nb, G * block, J]

    def by_block(x):                                              # [B, H, N, d] -> [B, Hkv, nb, G * block, d]
        x = torch.cat([x.float(), x.new_zeros(B, H, nb * block - N, d, dtype=torch.float32)], 2)
        return x.view(B, Hkv, G, nb, block, d).transpose(2, 3).reshape(B, Hkv, nb, G * block, d)

    def by_row(x, last):                                          # and back
        x = x.reshape(B, Hkv, nb, G, block, last).transpose(2, 3).reshape(B, H, nb * block, last)
        return x[:, :, :N]

    qb, kb, vb = by_block(q), k.float()[:, :, pos], v.float()[:, :, pos]
    p = qb @ kb.transpose(-1, -2)
    p.mul_(scale).masked_fill_(~see, -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)       # rows past the end see nothing
    p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    l = torch.where(l == 0, torch.ones_like(l), l)
    p.div_(l)
    o = p @ vb
    lse = by_row(m + torch.log(l), 1).squeeze(-1)
    out = [by_row(o, d).to(q.dtype), lse.contiguous()]
    if backward:
        dob = by_block(st["do"])
        D = (dob * o).sum(-1, keepdim=True)

        def to_keys(x):                                           # [B, Hkv, nb, J, d] summed over blocks
            return torch.zeros(B, Hkv, N, d, device=q.device).index_add_(2, pos.reshape(-1), x.reshape(B, Hkv, -1, d))

        dv = to_keys(p.transpose(-1, -2) @ dob)
        ds = dob @ vb.transpose(-1, -2)
        ds.sub_(D).mul_(p)
        del p
        dq = by_row(ds @ kb * scale, d)
        dk = to_keys(ds.transpose(-1, -2) @ qb * scale)
        out += [dq.to(q.dtype), dk.to(q.dtype), dv.to(q.dtype)]
    return tuple(x.contiguous() for x in out)


def _decode(st):
    c = st["case"]
    q, lens = st["q"], st["lens"]
    S, H, d = q.shape
    Hkv = c["Hkv"]
    ids = st["table"][:, :st["pages_most"]].clamp(min=0).long()
    T = ids.shape[1] * c["page"]

    def keys(pages):                                              # [S, Hkv, T, d]
        return pages[ids].transpose(1, 2).reshape(S, Hkv, T, d).float()

    j = torch.arange(T, device=q.device)
    n = lens.view(S, 1)
    see = j < n
    if c["window"]:
        see &= (n - 1 - j < c["window"]) | (j < c["sinks"])
    s = q.float().view(S, Hkv, H // Hkv, d) @ keys(st["k_pages"]).transpose(-1, -2) * d ** -0.5
    s = s.masked_fill(~see.view(S, 1, 1, T), -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    o = p @ torch.where(see.view(S, 1, T, 1), keys(st["v_pages"]), torch.zeros((), device=q.device))
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    return o.view(S, H, d).to(q.dtype), (m + torch.log(l)).view(S, H)


def _append(st):
    c = st["case"]
    t = torch.arange(st["k"].shape[0], dtype=torch.int32, device=st["cu"].device)
    s = torch.searchsorted(st["cu"], t, right=True) - 1
    pos = st["lens"][s] - (st["cu"][s + 1] - t)
    page, row = st["table"][s, pos // c["page"]].long(), pos % c["page"]
    st["k_pages"][page, :, row] = st["k"]
    st["v_pages"][page, :, row] = st["v"]
    return st["k_pages"], st["v_pages"]


def _held(lens, page):
    return (lens + page - 1) // page


def _branch(st):
    c, page = st["case"], st["case"]["page"]
    refs, table, lens = st["now"]
    src, dst = st["src"].long(), st["dst"].long()
    # branches: whole pages are shared, the last one, if it is not full, is copied to a free page
    n = lens[src]
    whole, rest = (n // page).view(-1, 1), n % page
    col = torch.arange(table.shape[1], device=table.device)
    rows = table[src]
    shared = col < whole
    refs += torch.bincount(rows[shared], minlength=refs.numel()).int()
    part = rest > 0
    old = rows[part, whole[part, 0]].long()
    fresh = torch.nonzero(refs == 0)[:int(part.sum()), 0]
    refs[fresh] = 1
    mine = torch.where(shared, rows, table[dst])
    mine[part, whole[part, 0]] = fresh.int()
    table[dst] = mine
    lens[dst] = n
    used = (torch.arange(page, device=n.device) < rest[part].view(-1, 1)).view(-1, 1, page, 1)
    for pages in (st["k_pages"], st["v_pages"]):
        pages[:, fresh] = torch.where(used, pages[:, old], pages[:, fresh])
    # room for the tokens that follow
    longer = lens + st["new"]
    more = (col >= _held(lens, page).view(-1, 1)) & (col < _held(longer, page).view(-1, 1))
    fresh = torch.nonzero(refs == 0)[:int(more.sum()), 0]
    refs[fresh] = 1
    table[more] = fresh.int()
    lens.copy_(longer)
    return st["k_pages"], st["v_pages"], refs, table, lens


def _retire(st):
    page = st["case"]["page"]
    refs, table, lens = st["now"]
    ended = st["ended"].long()
    col = torch.arange(table.shape[1], device=table.device)
    rows = table[ended]
    mine = col < _held(lens[ended], page).view(-1, 1)
    refs -= torch.bincount(rows[mine], minlength=refs.numel()).int()
    table[ended] = torch.where(mine, torch.full_like(rows, -1), rows)
    lens[ended] = 0
    # live pages past the number of live pages move to the free ones before it
    live = (refs > 0).sum()
    at = torch.arange(refs.numel(), device=refs.device)
    src = torch.nonzero((refs > 0) & (at >= live))[:, 0]
    dst = torch.nonzero((refs == 0) & (at < live))[:, 0]
    for pages in (st["k_pages"], st["v_pages"]):
        pages[:, dst] = pages[:, src]
    to = at.int()
    to[src] = dst.int()
    refs[dst] = refs[src]
    refs[src] = 0
    held = col < _held(lens, page).view(-1, 1)
    table[held] = to[table[held].long()]
    return st["k_pages"], st["v_pages"], refs, table, lens, live.int().view(1)


def run(state):
    st, c = state, state["case"]
    op = c["op"]
    if op == "pages":                                # every pass begins with the same tables
        for to, name in zip(st["now"], ("refs", "table", "lens")):
            to.copy_(st[name])
    if not own:
        if op in ("prefill", "train"):
            return _attention(st, op == "train")
        return {"decode": _decode, "append": _append, "branch": _branch, "retire": _retire}[c.get("step", op)](st)
    from flashattention_bf16_fwd_b200 import cache, window
    if op in ("prefill", "train"):
        o, lse = window.attention_window_fwd(st["q"], st["k"], st["v"], c["window"], c["sinks"], fix_mode=c["fix"])
        if op == "prefill":
            return o, lse
        return (o, lse) + window.attention_window_bwd(st["q"], st["k"], st["v"], o, lse, st["do"], c["window"], c["sinks"])
    if op == "decode":
        return cache.attention_decode(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"], window=c["window"],
                                      sinks=c["sinks"])
    if op == "append":
        cache.cache_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["lens"], st["cu"])
        return st["k_pages"], st["v_pages"]
    refs, table, lens = st["now"]
    pools = (st["k_pages"], st["v_pages"])
    if _step(c, "branch"):
        cache.cache_fork(*pools, refs, table, lens, st["src"], st["dst"])
        cache.cache_reserve(refs, table, lens, st["new"], c["page"])
        return (*pools, refs, table, lens)
    cache.cache_free(refs, table, lens, st["ended"], c["page"])
    live = cache.cache_compact(*pools, refs, table, lens)
    return (*pools, refs, table, lens, live)


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without


def _pairs(c):
    """Visible (query, key) pairs of one head."""
    n, w, sinks = c["N"], min(c["window"], c["N"]), min(c["sinks"], c["N"])
    near = w * (w + 1) // 2 + (n - w) * w
    # sink j is outside the window of the queries from j + w on
    far = sum(max(0, n - w - j) for j in range(sinks))
    return near + far


def work(case):
    c = case
    if c["op"] in ("prefill", "train"):
        heads, pairs = c["B"] * c["H"], _pairs(c)
        q = heads * c["N"] * c["d"] * 2
        kv = c["B"] * c["Hkv"] * c["N"] * c["d"] * 2
        lse = heads * c["N"] * 4
        if c["op"] == "prefill":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * c["d"] * pairs * heads}
        # q, k, v, do in; o, lse, dq, dk, dv out
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 14 * c["d"] * pairs * heads}
    token = c["Hkv"] * c["d"] * 2 * 2                             # K and V of a token in one layer
    lens = _lens(c)
    if c["op"] == "decode":
        w, sinks = c["window"], c["sinks"]
        seen = sum(n if not w else min(n, w + min(sinks, max(0, n - w))) for n in lens)
        out = c["S"] * c["H"] * (c["d"] * 4 + 4)
        return {"bytes": seen * token + out + 4 * sum(-(-n // c["page"]) for n in lens) + 4 * c["S"],
                "flops": 4 * c["d"] * seen * c["H"]}
    if c["op"] == "append":
        return {"bytes": 2 * sum(_news(c)) * token, "flops": 0}
    pool, refs, table, lens = _pages(c)
    entries = sum(len(r) for r in table)
    tables = 4 * (2 * pool + 2 * entries + 2 * c["S"])            # refs, table and lens, read and written
    if _step(c, "branch"):
        src, _ = _forks(c)
        moved = sum(lens[s] % c["page"] for s in src)
    else:
        ended = set(_ended(c))
        for s in ended:
            for p in table[s]:
                if p >= 0:
                    refs[p] = 0
        live = sum(r > 0 for r in refs)
        moved = sum(r > 0 for r in refs[live:]) * c["page"]
    return {"bytes": tables + 2 * moved * token * c["L"], "flops": 0}


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits, one head or one sequence after the other


def exact(case, seed):
    c = case
    if c["op"] not in ("prefill", "train", "decode"):
        return None                                               # whole numbers and copies
    st = prepare(c, seed)
    scale = 1.0 / math.sqrt(c["d"])
    q, dev = st["q"].double(), st["q"].device
    if c["op"] == "decode":
        o = torch.zeros_like(q)
        lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=dev)
        G = c["H"] // c["Hkv"]
        for s, n in enumerate(_lens(c)):
            if n == 0:
                continue
            pos = torch.arange(n, device=dev)
            if c["window"]:
                pos = pos[(pos < c["sinks"]) | (pos > n - 1 - c["window"])]
            page = st["table"][s, pos // c["page"]].long()
            ks = st["k_pages"][page, :, pos % c["page"]].double().repeat_interleave(G, 1)     # [n, H, d]
            vs = st["v_pages"][page, :, pos % c["page"]].double().repeat_interleave(G, 1)
            x = torch.einsum("hd,nhd->hn", q[s], ks) * scale
            lse[s] = torch.logsumexp(x, -1)
            o[s] = torch.einsum("hn,nhd->hd", torch.exp(x - lse[s][:, None]), vs)
        return o, lse
    B, H, N, d = q.shape
    i = torch.arange(N, device=dev)
    hidden = (i[None, :] > i[:, None]) | ((i[:, None] - i[None, :] >= c["window"]) & (i[None, :] >= c["sinks"]))
    outs = [torch.zeros_like(q), torch.zeros(B, H, N, dtype=torch.float64, device=dev)]
    if c["op"] == "train":
        outs += [torch.zeros_like(q), torch.zeros_like(st["k"], dtype=torch.float64), torch.zeros_like(st["v"], dtype=torch.float64)]
    for b in range(B):
        for h in range(H):
            g = h // (H // c["Hkv"])
            kk, vv = st["k"][b, g].double(), st["v"][b, g].double()
            x = (q[b, h] @ kk.T * scale).masked_fill_(hidden, -math.inf)
            top = torch.logsumexp(x, -1)
            p = x.sub_(top[:, None]).exp_()
            o = p @ vv
            outs[0][b, h], outs[1][b, h] = o, top
            if c["op"] == "train":
                do = st["do"][b, h].double()
                outs[4][b, g] += p.T @ do
                ds = p.mul_(do @ vv.T - (do * o).sum(-1)[:, None])
                outs[2][b, h] = ds @ kk * scale
                outs[3][b, g] += ds.T @ q[b, h] * scale
    return tuple(outs)
