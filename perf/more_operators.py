"""Workloads of the event history held in 8 bits: pages reserved for new
events on the GPU, the append that encodes keys and values, and attention over
the encoded cache.

A cache holds E4M3 codes, and for each head and block of consecutive slots of
a page one power of two (a biased exponent byte) that its codes are multiplied
by.  A step reserves pages and slots from the users' counts of new events,
appends, and attends.  Each case is a dict of plain values; ``prepare`` makes
its inputs, ``run`` makes one pass through one operator: with ``own`` true by
the package's calls, else in elementary torch operations.  ``exact`` gives the
same outputs in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
CODE = torch.float8_e4m3fn
BIAS = 127  # of an exponent byte


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a quiet moment of serving: one event of 8 users
        dict(name="reserve, few users", op="reserve", S=8, new=1, len=300, page=16, ended=0, short=False),
        # one new event of each of 2048 users (the one-hot batch), some of whom have left
        dict(name="reserve, one event each", op="reserve", S=2048, new=1, len=1000, page=16, ended=16, short=False),
        # whole histories on first sight, and more of them than the pool has pages for
        dict(name="reserve, prompts", op="reserve", S=512, new=4096, len=8192, page=64, ended=8, short=True),
        # one new event of each of 2048 users, into blocks that others' older events fill in part
        dict(name="append 8 bits, one event each", op="append", S=2048, new=1, len=1000, hk=2, d=64, page=16, block=16,
             ragged=True, heads_first=False, dtype="f16"),
        # whole histories on first sight: ragged prompts, a scale for each 16 tokens of a head
        dict(name="append 8 bits, prompts", op="append", S=48, new=4095, len=4096, hk=8, d=128, page=64, block=16,
             ragged=True, heads_first=True, dtype="bf16"),
        # serving at low load: one event of a few users, short histories
        dict(name="attention 8 bits, few users", op="attn", S=4, new=1, len=300, hq=8, hk=2, d=64, page=16, block=16,
             ragged=True, heads_first=False, causal=True, window=0, dtype="f16"),
        # serving at high load: one event of each of 256 users, histories of every length up to 8192
        dict(name="attention 8 bits, many users", op="attn", S=256, new=1, len=8192, hq=16, hk=4, d=128, page=64,
             block=16, ragged=True, heads_first=True, causal=True, window=0, dtype="bf16"),
        # one user with a very long history: the long axis is split
        dict(name="attention 8 bits, one history", op="attn", S=1, new=1, len=262143, hq=16, hk=4, d=128, page=16,
             block=16, ragged=False, heads_first=False, causal=True, window=0, dtype="bf16"),
        # long chunks of new events on long histories: the largest
        dict(name="attention 8 bits, long chunks", op="attn", S=4, new=2048, len=8192, hq=16, hk=4, d=128, page=64,
             block=64, ragged=False, heads_first=True, causal=True, window=0, dtype="bf16"),
        # ranking: up to 200 candidate items of each of 64 users attend over the user's history, no shared heads
        dict(name="attention 8 bits, candidates", op="attn", S=64, new=200, len=2000, hq=8, hk=8, d=64, page=32,
             block=32, ragged=True, heads_first=False, causal=False, window=0, dtype="f16"),
        # full-precision queries, a few new events each, only the last 512 events seen
        dict(name="attention 8 bits, f32 window", op="attn", S=128, new=4, len=1500, hq=4, hk=2, d=64, page=32,
             block=8, ragged=True, heads_first=False, causal=True, window=512, dtype="f32"),
        # the interaction-heavy width: a few candidates of each user, heads of 256
        dict(name="attention 8 bits, wide heads", op="attn", S=96, new=3, len=3000, hq=8, hk=2, d=256, page=32,
             block=32, ragged=True, heads_first=True, causal=False, window=0, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_MOST = {}  # per operator, the largest listed case's bytes and flops


def _most(op):
    if not _MOST:
        for c in listed():
            w = work(c)
            b, f = _MOST.get(c["op"], (0, 0))
            _MOST[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    return _MOST[op]


def draw(rng):
    op = rng.choice(["reserve", "append", "append", "attn", "attn", "attn", "attn"])
    if op == "reserve":
        c = dict(op=op, S=_log(rng, 1, 8192), new=_log(rng, 1, 4096), len=_log(rng, 16, 16384),
                 page=rng.choice([8, 16, 20, 32, 64, 128]), ended=rng.choice([0, 0, 5, 16]), short=rng.random() < 0.25)
        c["len"] = max(c["len"], c["new"])
        while c["S"] * c["new"] > 512 * 4096 or c["S"] * c["len"] // c["page"] > 1 << 20:
            c["S"] = max(1, c["S"] * 2 // 3)
        return c
    hk, page = rng.choice([1, 2, 4, 8]), rng.choice([8, 16, 24, 32, 64, 128])
    d = rng.choice([32, 64, 64, 80, 96, 128, 128, 128])
    block = rng.choice([page, page, 16 if page % 16 == 0 else 8, 8, 1])
    if op == "append":
        c = dict(op=op, S=_log(rng, 1, 2048), new=_log(rng, 1, 4096), len=_log(rng, 16, 8192), hk=hk, d=d, page=page,
                 block=block, ragged=rng.random() < 0.8, heads_first=rng.random() < 0.5,
                 dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
        shrink = ("S", "new", "len")
    else:
        dtype = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
        new = rng.choice([1, 1, _log(rng, 2, 2048), _log(rng, 16, 2048)])
        if dtype == "f32":  # full precision serves short chunks
            new = min(new, 16)
        if d == 128 and new <= 16 and rng.random() < 0.25:
            d = 256
        c = dict(op=op, S=_log(rng, 1, 512), new=new, len=_log(rng, 16, 262144), hq=hk * rng.choice([1, 2, 3, 4, 8]),
                 hk=hk, d=d, page=page, block=block, ragged=rng.random() < 0.8, heads_first=rng.random() < 0.5,
                 causal=rng.random() < 0.7, window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]), dtype=dtype)
        shrink = ("S", "len")
    c["len"] = max(c["len"], c["new"])
    k = 0
    while _cost(c) > 1 and k < 200:  # no dearer than the largest listed case
        key = shrink[k % len(shrink)]
        c[key] = max(1, c[key] * 2 // 3)
        c["len"] = max(c["len"], c["new"])
        k += 1
    return c


def _cost(c):
    """A case's work over the largest listed one's; a batch is also held to the padded size of the plain form."""
    b, f = _most(c["op"])
    w = work(c)
    cost = w["bytes"] / b if c["op"] == "append" else max(w["bytes"] / b, w["flops"] / f)
    if c["op"] == "append":
        return max(cost, c["S"] * c["len"] * c["hk"] * c["d"] / (48 * 4096 * 8 * 128))
    return max(cost, c["S"] * c["len"] * c["hk"] * c["d"] / (256 * 8192 * 4 * 128),
               c["S"] * c["len"] * c["hq"] * c["new"] / (4 * 8192 * 16 * 2048))


def _lengths(c):
    """New tokens and stored tokens (the new ones among them, where they are stored) of each sequence."""
    S, new, most = c["S"], c["new"], c["len"]
    stored = c.get("causal", True)
    if not c["ragged"]:
        return [new] * S, [most] * S
    r = random.Random(S * 1000003 + new * 8191 + most)
    counts = [new] + [r.randint(1, new) for _ in range(S - 1)]
    lens = [most] + [r.randint(n if stored else 0, most) for n in counts[1:]]
    if S >= 16 and new > 1:  # an idle sequence in the batch
        counts[7] = 0
    if S >= 16 and not stored:  # candidates of a user without a history
        lens[9] = 0
    return counts, lens


def _asked(c):
    """New events of each user (below 0: the user has left) and events stored before."""
    r = random.Random(c["S"] * 1000003 + c["new"] * 8191 + c["len"])
    counts = [c["new"]] + [r.randint(0 if c["new"] > 1 else 1, c["new"]) for _ in range(c["S"] - 1)]
    before = [r.randint(0, c["len"] - max(n, 0)) for n in counts]
    if c["ended"]:
        for s in range(c["ended"] - 1, c["S"], c["ended"]):
            counts[s] = -1
    return counts, before


def _visible(c):
    """(query, key) pairs that the mask leaves, and stored tokens that some query sees."""
    pairs = seen = 0
    for n, length in zip(*_lengths(c)):
        if n == 0 or length == 0:
            continue
        w = c["window"] or length
        if not c["causal"]:
            pairs += n * min(w, length)
            seen += min(w, length)
            continue
        first = length - n + 1  # keys of the first query, without the window
        whole = max(0, min(n, w - first + 1)) if first <= w else 0  # queries that see everything before them
        pairs += whole * first + whole * (whole - 1) // 2 + (n - whole) * w
        seen += min(length, n - 1 + w)
    return pairs, seen


def work(case):
    c = case
    if c["op"] == "reserve":
        counts, before = _asked(c)
        pages = sum(-(-(b + max(n, 0)) // c["page"]) - -(-b // c["page"]) for n, b in zip(counts, before))
        gone = sum(-(-b // c["page"]) for n, b in zip(counts, before) if n < 0)
        # counts, lengths in and out, offsets; slot and position of a token; a page's number read and written
        return {"bytes": 32 * c["S"] + 16 * sum(max(n, 0) for n in counts) + 8 * (pages + gone) + 32, "flops": 0}
    es = SIZES[c["dtype"]]
    n = sum(_lengths(c)[0])
    if c["op"] == "append":
        el = 2 * n * c["hk"] * c["d"]
        return {"bytes": el * (es + 1) + 2 * c["hk"] * (n // c["block"] + c["S"]) + 20 * c["S"] + 4 * n // c["page"],
                "flops": 3 * el}
    pairs, seen = _visible(c)
    return {"bytes": 2 * n * c["hq"] * c["d"] * es + 4 * n * c["hq"] + 2 * seen * c["hk"] * c["d"]
            + 2 * c["hk"] * seen // c["block"] + 4 * seen // c["page"] + 16 * c["S"],
            "flops": 4 * c["d"] * c["hq"] * pairs}


# ---------------------------------------------------------------- the inputs

def _randn(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _exponents(top):
    """The smallest e with top <= 448 * 2^(e - 127), at least 1; 0 where top is 0."""
    bits = top.view(torch.int32)
    e = (bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()
    return torch.where(top > 0, e.clamp(min=1), 0)


def _power(e):
    """2^(e - 127) in 32 bits, of exponent bytes 1 .. 254; 0 of 0."""
    return (e.to(torch.int32) << 23).view(torch.float32)


def _encoded(x, e):
    """The codes, as bytes, of x whose blocks have the exponents e (broadcast over x)."""
    back = ((254 - e.to(torch.int32)).clamp(1, 253) << 23).view(torch.float32)
    return (x * back).clamp(-448, 448).to(CODE).view(torch.uint8)


def _cache(gen, pages, c):
    """A cache whose every page holds some user's tokens: codes [pages][page][heads][d] and exponents
    [pages][blocks][heads].  A head's keys and values have a spread of their own, and vary from token to token."""
    spread = torch.exp2(torch.randint(-2, 3, (c["hk"],), generator=gen, device="cuda").float())
    spread = spread * torch.exp2(torch.randn((pages, c["page"], 1), generator=gen, device="cuda") * 0.3)
    x = torch.randn((pages, c["page"], c["hk"], c["d"]), generator=gen, device="cuda") * spread[..., None]
    x = x.view(pages, -1, c["block"], c["hk"], c["d"])
    e = _exponents(x.abs().amax((2, 4)))
    codes = _encoded(x, e[:, :, None, :, None]).view(CODE).view(pages, c["page"], c["hk"], c["d"])
    if c["heads_first"]:
        codes = codes.transpose(1, 2).contiguous().transpose(1, 2)
    return codes, e.to(torch.uint8)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "reserve":
        return _prepare_reserve(c, gen, s)
    dtype = DTYPES[c["dtype"]]
    counts, lens = _lengths(c)
    S, n, page = c["S"], sum(counts), c["page"]
    s["lengths"] = torch.tensor(lens, dtype=torch.int64, device="cuda")
    s["offsets"] = torch.tensor([0] + counts, dtype=torch.int64, device="cuda").cumsum(0)
    s["n"], s["max_new"], s["max_len"] = n, max(counts), max(lens)
    need = [-(-length // page) for length in lens]
    P, pages = max(max(need), 1), sum(need) + 3
    order = torch.randperm(pages, generator=gen, device="cuda")[:sum(need)].to(torch.int32)
    table = torch.full((S, P), -1, dtype=torch.int32, device="cuda")
    has = torch.arange(P, device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None]
    table[has] = order
    s["page_table"] = table
    (s["k_cache"], s["k_exp"]), (s["v_cache"], s["v_exp"]) = _cache(gen, pages, c), _cache(gen, pages, c)
    if c["op"] == "append":
        # keys as normed and turned, values as they come out of the projection: views of wider rows
        kv = _randn(gen, (n, 2 * c["hk"], c["d"]), dtype, 1.5)
        s["k"], s["v"] = kv[:, :c["hk"]], kv[:, c["hk"]:]
        return s
    s["q"] = _randn(gen, (n, c["hq"], c["d"]), dtype, 0.5)
    s["scale"] = 1 / math.sqrt(c["d"])
    s["out"] = torch.empty((n, c["hq"], c["d"]), dtype=dtype, device="cuda")
    s["lse"] = torch.empty((n, c["hq"]), device="cuda")
    return s


def _prepare_reserve(c, gen, s):
    counts, before = _asked(c)
    S, page = c["S"], c["page"]
    held = [-(-b // page) for b in before]
    wanted = [-(-(b + max(n, 0)) // page) - h for n, b, h in zip(counts, before, held)]
    free = sum(wanted) * 3 // 4 if c["short"] else sum(wanted) + 17
    width, pages = max(-(-c["len"] // page), 1), sum(held) + free
    order = torch.randperm(max(pages, 1), generator=gen, device="cuda").to(torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    has = torch.arange(width, device="cuda")[None, :] < torch.tensor(held, device="cuda")[:, None]
    table[has] = order[:sum(held)]
    ring = torch.full((max(pages, 1),), -1, dtype=torch.int32, device="cuda")
    # a ring that has been gone around: its first free page lies anywhere
    head = int(torch.randint(0, 1 << 20, (1,), generator=gen, device="cuda"))
    at = (head + torch.arange(free, device="cuda")) % max(pages, 1)
    ring[at] = order[sum(held):sum(held) + free]
    as64 = lambda v: torch.tensor(v, dtype=torch.int64, device="cuda")
    n = sum(max(x, 0) for x in counts)
    s.update(counts=as64(counts), lengths=as64(before), page_table=table, ring=ring, state=as64([head, head + free]),
             n=n, gone=sum(h for x, h in zip(counts, held) if x < 0),
             new_state=torch.zeros(2, dtype=torch.int64, device="cuda"),
             offsets=torch.empty(S + 1, dtype=torch.int64, device="cuda"),
             new_lengths=torch.empty(S, dtype=torch.int64, device="cuda"),
             slots=torch.full((n + 5,), -7, dtype=torch.int64, device="cuda"),  # rows behind the last stay as they are
             positions=torch.full((n + 5,), -7, dtype=torch.int64, device="cuda"))
    return s


# ---------------------------------------------------------------- one pass

def _workspace(s, size):
    """A program keeps its workspace from call to call."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s["workspace"]


def run(state):
    return (_run_own if own else _run_plain)(state)


_RESERVED = ("offsets", "new_lengths", "page_table", "ring", "new_state", "slots", "positions")
_STORED = ("k_cache", "v_cache", "k_exp", "v_exp")


def _run_own(s):
    import sparse_dense_interaction_gb300 as sdi
    c = s["case"]
    if c["op"] == "reserve":
        sdi.dlrm_kv_reserve(s["counts"], s["lengths"], s["page_table"], c["page"], s["ring"], s["state"],
                            s["new_state"], s["offsets"], s["new_lengths"], s["slots"], s["positions"])
        return {k: s[k] for k in _RESERVED}
    cache = s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"]
    if c["op"] == "append":
        sdi.dlrm_kv8_append(s["k"], s["v"], s["offsets"], s["lengths"], s["page_table"], *cache)
        return {k: s[k] for k in _STORED}
    ws = _workspace(s, sdi.dlrm_kv8_attn_workspace_size(c["S"], s["n"], c["hq"], c["hk"], c["d"], s["max_new"],
                                                        s["max_len"]))
    sdi.dlrm_kv8_attn_fwd(s["q"], s["offsets"], s["lengths"], s["page_table"], *cache, s["out"], s["scale"], ws,
                          s["max_new"], s["max_len"], causal=c["causal"], window=c["window"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _run_plain(s):
    return {"reserve": _reserve, "append": _append, "attn": _attention}[s["case"]["op"]](s)


def _reserve(s):
    """Whole numbers: every user's pages by prefix sums of what each needs."""
    page, counts, before, table, ring = s["case"]["page"], s["counts"], s["lengths"], s["page_table"], s["ring"]
    (S, width), pages, n = table.shape, ring.numel(), s["n"]
    head, tail = s["state"][0], s["state"][1]
    take, stays = counts.clamp(min=0), counts >= 0
    held, wanted = -(-before // page), -(-(before + take) // page)
    fits = stays & (wanted <= width)
    need = torch.where(fits, wanted - held, 0)
    prefix = need.cumsum(0)
    granted = fits & ((need == 0) | (prefix <= tail - head))
    s["offsets"][0] = 0
    torch.cumsum(take, 0, out=s["offsets"][1:])
    s["new_lengths"].copy_(torch.where(granted, before + take, torch.where(stays, ~before, 0)))
    # the pages of users who have left go to the ring's end
    gone = torch.where(stays, 0, held)
    seq = torch.repeat_interleave(torch.arange(S, device="cuda"), gone, output_size=s["gone"])
    k = torch.arange(s["gone"], device="cuda")
    freed = table[seq, k - (gone.cumsum(0) - gone)[seq]]
    # every token's page, from the table or from the ring's start
    seq = torch.repeat_interleave(torch.arange(S, device="cuda"), take, output_size=n)
    at = before[seq] + torch.arange(n, device="cuda") - s["offsets"][seq]
    number = at // page
    fresh = ring[(head + (prefix - need - held)[seq] + number) % pages]
    mine = torch.where(number < held[seq], table[seq, number.clamp(max=width - 1)], fresh).long()
    got = granted[seq]
    s["slots"][:n] = torch.where(got, mine * page + at % page, -1)
    s["positions"][:n] = torch.where(got, at, -1)
    first = got & (at % page == 0)
    table[seq[first], number[first]] = fresh[first]
    ring[(tail + k) % pages] = freed
    s["new_state"][0] = head + torch.where(granted & (need > 0), prefix, 0).max()
    s["new_state"][1] = tail + s["gone"]
    return {k: s[k] for k in _RESERVED}


def _places(s):
    """Sequence, number in its chunk and place in its history of each new token."""
    counts = s["offsets"][1:] - s["offsets"][:-1]
    seq = torch.repeat_interleave(torch.arange(counts.numel(), device="cuda"), counts, output_size=s["n"])
    i = torch.arange(s["n"], device="cuda") - s["offsets"][seq]
    return seq, i, (s["lengths"] - counts)[seq] + i


def _append(s):
    """A block's exponent covers its new tokens and, where it holds older ones, the exponent it had; older codes
    are rounded again where it grows."""
    c = s["case"]
    page, block = c["page"], c["block"]
    seq, _, at = _places(s)
    number = s["page_table"][seq, at // page].long()
    cell = number * (page // block) + at % page // block  # the block that each new token enters
    before = s["lengths"] - (s["offsets"][1:] - s["offsets"][:-1])
    seen = before[seq]  # tokens stored before the call
    older = seen > at // block * block
    for name in ("k", "v"):
        x, codes, exps = s[name].float(), s[name + "_cache"].view(torch.uint8), s[name + "_exp"]
        flat = exps.view(-1, c["hk"])
        # the largest magnitude of each block's new tokens, through its first new token
        tops = torch.zeros_like(flat, dtype=torch.float32)
        tops.index_reduce_(0, cell, x.abs().amax(2), "amax")
        old = flat[cell].int()
        new = torch.maximum(_exponents(tops[cell]), torch.where(older[:, None], old, 0))
        # older tokens of the blocks that hold some: slots of the block before the call's first token of it
        j = torch.arange(block, device="cuda")
        lead = older & (at == seen)
        slot = (at % page // block * block)[:, None] + j
        mine = lead[:, None] & ((at // block * block)[:, None] + j < seen[:, None])
        held = codes[number[:, None].expand_as(slot)[mine], slot[mine]].view(CODE).float()
        o, e = (t[:, None].expand(-1, block, -1)[mine] for t in (old, new))
        held = held * torch.exp2((o - e).double()).float()[..., None]
        codes[number[:, None].expand_as(slot)[mine], slot[mine]] = held.to(CODE).view(torch.uint8)
        codes[number, at % page] = _encoded(x, new[..., None])
        flat[cell] = new.to(torch.uint8)
    return {k: s[k] for k in _STORED}


def _values(s, name):
    """The cache's values in 32 bits: codes times their blocks' powers of two."""
    codes, block = s[name + "_cache"].view(torch.uint8), s["case"]["block"]
    pages = s["page_table"].long().clamp(min=0)
    power = _power(s[name + "_exp"])[pages].repeat_interleave(block, 2)
    return codes[pages].view(CODE).float() * power[..., None]


def _attention(s):
    c = s["case"]
    S, hk, d, C, L = c["S"], c["hk"], c["d"], s["max_new"], s["max_len"]
    G = c["hq"] // hk
    seq, i, _ = _places(s)
    counts = s["offsets"][1:] - s["offsets"][:-1]
    j = torch.arange(L, device="cuda")
    stored = (j[None, :] < s["lengths"][:, None])[:, :, None, None]
    k, v = (torch.where(stored, _values(s, t).flatten(1, 2)[:, :L], 0.0) for t in ("k", "v"))
    q = torch.zeros((S, C, hk * G, d), device="cuda")
    q[seq, i] = s["q"].float()
    q = q.view(S, C, hk, G, d).permute(0, 2, 3, 1, 4).reshape(S, hk, G * C, d)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    hi = s["lengths"][:, None].expand(S, C)
    if c["causal"]:
        hi = (s["lengths"] - counts)[:, None] + torch.arange(C, device="cuda") + 1
    lo = (hi - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(hi)
    seen = (j >= lo[..., None]) & (j < torch.minimum(hi, s["lengths"][:, None])[..., None])
    scores = scores.view(S, hk, G, C, L).masked_fill(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, hk, G * C, L), v.permute(0, 2, 1, 3)).view(S, hk, G, C, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + torch.log(total)).squeeze(-1)
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(S, C, hk * G, d)[seq, i].to(DTYPES[c["dtype"]]),
            "lse": lse.permute(0, 3, 1, 2).reshape(S, C, hk * G)[seq, i]}


# ---------------------------------------------------------------- in 64 bits

def _code64(x):
    """x rounded to the nearest E4M3 value, ties to even, in 64 bits."""
    size = torch.frexp(x.abs().clamp(min=2.0 ** -6)).exponent - 1  # normal from 2^-6 on
    step = torch.exp2((size - 3).double())
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "reserve":
        return None  # whole numbers
    counts, lens = _lengths(c)
    table, page, block = s["page_table"].cpu(), c["page"], c["block"]
    slots = [table[b, :-(-length // page)].long() if length else table[b, :0].long() for b, length in enumerate(lens)]
    first = [0]
    for n in counts:
        first.append(first[-1] + n)
    if c["op"] == "append":
        return _append64(c, s, counts, lens, slots, first)
    G = c["hq"] // c["hk"]
    o = torch.zeros((s["n"], c["hq"], c["d"]), dtype=torch.float64, device="cuda")
    lse = torch.full((s["n"], c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, (n, length) in enumerate(zip(counts, lens)):
        if n == 0 or length == 0:
            continue
        at = slots[b].cuda()
        k, v = ((s[t + "_cache"].view(torch.uint8)[at].view(CODE).double().reshape(len(at), -1, block, c["hk"], c["d"])
                 * torch.exp2(s[t + "_exp"][at].double() - BIAS)[:, :, None, :, None]).reshape(-1, c["hk"], c["d"])[:length]
                for t in ("k", "v"))
        row = torch.arange(n, device="cuda")
        end = length - n + row + 1 if c["causal"] else torch.full_like(row, length)
        begin = (end - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(end)
        j = torch.arange(length, device="cuda")
        off = (j < begin[:, None]) | (j >= end[:, None])
        q = s["q"][first[b]:first[b] + n].double() * s["scale"]
        for h in range(c["hq"]):
            score = (q[:, h] @ k[:, h // G].T).masked_fill_(off, -math.inf)
            lse[first[b]:first[b] + n, h] = torch.logsumexp(score, -1)
            o[first[b]:first[b] + n, h] = torch.softmax(score, -1).nan_to_num_(0.0) @ v[:, h // G]
    return {"out": o, "lse": lse}


def _append64(c, s, counts, lens, slots, first):
    page, block, blocks = c["page"], c["block"], c["page"] // c["block"]
    out = {}
    for name in ("k", "v"):
        codes = s[name + "_cache"].view(torch.uint8).contiguous().view(CODE).double()
        cells = codes.view(-1, block, c["hk"], c["d"])  # every block of the cache
        exps = s[name + "_exp"].long().view(-1, c["hk"])
        x = s[name].double()
        # the batch's blocks, each with the row of its first slot's token (before the first new token: below it)
        rows, cell, olds = [], [], []
        for b, (n, length) in enumerate(zip(counts, lens)):
            p = torch.arange((length - n) // block, -(-length // block)) if n else torch.zeros(0, dtype=torch.int64)
            rows.append(p * block - (length - n))
            cell.append(slots[b][p * block // page] * blocks + p % blocks)
            olds.append((torch.stack([rows[-1]], 1) + torch.arange(block) >= n).long() * 2
                        + (torch.stack([rows[-1]], 1) + torch.arange(block) < 0).long())
            rows[-1] = rows[-1] + first[b]
        rows, cell, olds = (torch.cat(t).cuda() for t in (rows, cell, olds))
        take = (rows[:, None] + torch.arange(block, device="cuda")).clamp(0, max(s["n"] - 1, 0))
        for part in range(0, cell.numel(), 65536):
            at, kind = cell[part:part + 65536], olds[part:part + 65536, :, None, None]  # 0 new, 1 older, 2 unused
            new = x[take[part:part + 65536]]
            top = torch.where(kind == 0, new.abs(), 0.0).amax((1, 3))
            m, e = torch.frexp(top / 448)  # top <= 448 * 2^e, of m 0.5 the smaller
            e = torch.where(top > 0, (e - (m == 0.5).int() + BIAS).clamp(min=1), 0).long()
            e = torch.where((olds[part:part + 65536] == 1).any(1)[:, None], torch.maximum(e, exps[at]), e)
            held = cells[at]
            again = _code64(held * torch.exp2((exps[at] - e).double())[:, None, :, None])
            fresh = _code64(new * torch.exp2((BIAS - e).double())[:, None, :, None])
            cells[at] = torch.where(kind == 0, fresh, torch.where(kind == 1, again, held))
            exps[at] = e
        out[name + "_cache"] = codes
        out[name + "_exp"] = exps.view(s[name + "_exp"].shape)
    return out
