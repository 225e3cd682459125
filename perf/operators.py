"""Workloads of the event-history operators: head norms with rotation, the
paged key/value cache's append, and attention over that cache.

A user's stored events are a paged cache of keys and values.  New events are
normed, rotated and appended; new events (causal) or candidate items (not
causal, not stored) attend over the cache.  Each case is a dict of plain
values; ``prepare`` makes its inputs, ``run`` makes one pass through one
operator: with ``own`` true by the package's calls, else in elementary torch
operations in 32 bits.  ``exact`` gives the same outputs in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
ROPE_BASE = 10000.0


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one request's few events through the query/key norms: the launch is what counts
        dict(name="norm rotation, few tokens", op="norm_fwd", n=48, hq=8, hk=2, d=64, rot=64, interleaved=False,
             dtype="f16", rope_len=4096),
        # a training batch of event rows (65536, the multi-hot batch) of 128-wide heads, shared key heads
        dict(name="norm rotation, batch", op="norm_fwd", n=65536, hq=16, hk=4, d=128, rot=128, interleaved=False,
             dtype="bf16", rope_len=8192),
        # its gradient
        dict(name="norm rotation gradient, batch", op="norm_bwd", n=65536, hq=16, hk=4, d=128, rot=128,
             interleaved=False, dtype="bf16", rope_len=8192),
        # full-precision training with a ragged row count, 64-wide heads, half of each rotated, neighbouring pairs
        dict(name="norm rotation gradient, f32", op="norm_bwd", n=8193, hq=4, hk=4, d=64, rot=32, interleaved=True,
             dtype="f32", rope_len=16384),
        # one new event of each of 2048 users (the one-hot batch) enters the cache
        dict(name="append, one event each", op="append", S=2048, new=1, len=1000, hq=8, hk=2, d=64, rot=64, page=16,
             ragged=True, heads_first=False, norm=True, dtype="f16"),
        # whole histories on first sight: ragged prompts
        dict(name="append, prompts", op="append", S=48, new=2047, len=4096, hq=16, hk=4, d=128, rot=128, page=64,
             ragged=True, heads_first=True, norm=True, dtype="bf16"),
        # serving at low load: one event of a few users, short histories
        dict(name="attention, few users", op="attn", S=4, new=1, len=300, hq=8, hk=2, d=64, page=16, ragged=True,
             heads_first=False, causal=True, window=0, dtype="f16"),
        # serving at high load: one event of each of 256 users, histories of every length up to 8192
        dict(name="attention, many users", op="attn", S=256, new=1, len=8192, hq=16, hk=4, d=128, page=64,
             ragged=True, heads_first=True, causal=True, window=0, dtype="bf16"),
        # one user with a very long history: the long axis is split
        dict(name="attention, one long history", op="attn", S=1, new=1, len=262143, hq=16, hk=4, d=128, page=16,
             ragged=False, heads_first=False, causal=True, window=0, dtype="bf16"),
        # long chunks of new events on long histories: the largest
        dict(name="attention, long chunks", op="attn", S=4, new=2048, len=8192, hq=16, hk=4, d=128, page=64,
             ragged=False, heads_first=True, causal=True, window=0, dtype="bf16"),
        # ranking: up to 200 candidate items of each of 64 users attend over the user's history, no shared heads
        dict(name="attention, candidates", op="attn", S=64, new=200, len=2000, hq=8, hk=8, d=64, page=32,
             ragged=True, heads_first=False, causal=False, window=0, dtype="f16"),
        # full precision, a few new events each, only the last 512 events seen
        dict(name="attention, f32 window", op="attn", S=128, new=4, len=1500, hq=4, hk=2, d=64, page=32, ragged=True,
             heads_first=False, causal=True, window=512, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_MOST = {}  # per operator, the largest listed case's bytes and flops


def _most(op):
    if not _MOST:
        for c in listed():
            w, key = work(c), c["op"][:4]
            b, f = _MOST.get(key, (0, 0))
            _MOST[key] = (max(b, w["bytes"]), max(f, w["flops"]))
    return _MOST[op[:4]]


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "append", "append", "attn", "attn", "attn", "attn"])
    d = rng.choice([32, 64, 64, 80, 96, 128, 128, 128])
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("norm"):
        c = dict(op=op, n=_log(rng, 1, 65536), hq=hq, hk=hk, d=d, rot=rng.choice([d, d, d // 2]),
                 interleaved=rng.random() < 0.3, dtype=dtype, rope_len=_log(rng, 256, 16384))
        shrink = ("n",)
    elif op == "append":
        c = dict(op=op, S=_log(rng, 1, 2048), new=_log(rng, 1, 2048), len=_log(rng, 16, 8192), hq=hq, hk=hk, d=d,
                 rot=rng.choice([d, d, d // 2]), page=rng.choice([8, 16, 24, 32, 64]), ragged=rng.random() < 0.8,
                 heads_first=rng.random() < 0.5, norm=rng.random() < 0.7, dtype=dtype)
        shrink = ("S", "new", "len")
    else:
        dtype = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
        new = rng.choice([1, 1, _log(rng, 2, 2048), _log(rng, 16, 2048)])
        if dtype == "f32":  # full precision serves short chunks
            new = min(new, 16)
        c = dict(op=op, S=_log(rng, 1, 512), new=new, len=_log(rng, 16, 262144), hq=hq, hk=hk, d=d,
                 page=rng.choice([8, 16, 24, 32, 64, 128]), ragged=rng.random() < 0.8,
                 heads_first=rng.random() < 0.5, causal=rng.random() < 0.7,
                 window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]), dtype=dtype)
        shrink = ("S", "len")
    if "len" in c:
        c["len"] = max(c["len"], c["new"])
    k = 0
    while _cost(c) > 1 and k < 200:  # no dearer than the largest listed case
        key = shrink[k % len(shrink)]
        c[key] = max(1, c[key] * 2 // 3)
        if "len" in c:
            c["len"] = max(c["len"], c["new"])
        k += 1
    return c


def _cost(c):
    """A case's work over the largest listed one's; a batch is also held to the padded size of the plain form."""
    b, f = _most(c["op"])
    w = work(c)
    cost = max(w["bytes"] / b, w["flops"] / f)
    if c["op"] == "append":
        cost = max(cost, c["S"] * c["len"] * c["hk"] * c["d"] / (2048 * 1000 * 2 * 64))
    if c["op"] == "attn":
        cost = max(cost, c["S"] * c["len"] * c["hk"] * c["d"] / (256 * 8192 * 4 * 128),
                   c["S"] * c["len"] * c["hq"] * c["new"] / (4 * 8192 * 16 * 2048))
    return cost


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
    c, es = case, SIZES[case["dtype"]]
    if c["op"].startswith("norm"):
        el = c["n"] * (c["hq"] + c["hk"]) * c["d"]
        rows = min(c["n"], c["rope_len"]) * c["rot"] * 4 + 8 * c["n"]
        if c["op"] == "norm_fwd":
            return {"bytes": 2 * el * es + rows, "flops": 8 * el}
        return {"bytes": 3 * el * es + rows, "flops": 18 * el}
    n = sum(_lengths(c)[0])
    if c["op"] == "append":
        el = n * (c["hq"] + c["hk"]) * c["d"]
        return {"bytes": 2 * el * es + 2 * n * c["hk"] * c["d"] * es + min(n, c["len"]) * c["rot"] * 4 + 20 * c["S"],
                "flops": 8 * el}
    pairs, seen = _visible(c)
    return {"bytes": 2 * n * c["hq"] * c["d"] * es + 4 * n * c["hq"] + 2 * seen * c["hk"] * c["d"] * es
            + 4 * seen // c["page"] + 16 * c["S"],
            "flops": 4 * c["d"] * c["hq"] * pairs}


# ---------------------------------------------------------------- the inputs

def _randn(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _rope(length, rot):
    """cos of the rot/2 angles of every position, then their sins, in 32 bits."""
    f = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _cache(gen, pages, c, dtype):
    """A cache whose every page holds some user's tokens; seen as [pages][page][heads][d]."""
    if c["heads_first"]:
        return _randn(gen, (pages, c["hk"], c["page"], c["d"]), dtype).transpose(1, 2)
    return _randn(gen, (pages, c["page"], c["hk"], c["d"]), dtype)


def prepare(case, seed):
    c, dtype = case, DTYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    hq, hk, d = c["hq"], c["hk"], c["d"]
    if c["op"] != "attn":
        # weights as they are after some training: around one
        s["q_weight"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda")
        s["k_weight"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda")
    if c["op"].startswith("norm"):
        n = c["n"]
        # queries, keys and values come out of one projection: heads of one row, side by side
        qkv = _randn(gen, (n, hq + 2 * hk, d), dtype, 1.5)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["rope"] = _rope(c["rope_len"], c["rot"])
        s["positions"] = torch.randint(0, c["rope_len"], (n,), generator=gen, device="cuda")
        if c["op"] == "norm_bwd":
            s["dq_out"], s["dk_out"] = _randn(gen, (n, hq, d), dtype), _randn(gen, (n, hk, d), dtype)
            s["dq_weight"], s["dk_weight"] = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
        s["out"] = torch.empty((n, hq, d), dtype=dtype, device="cuda"), torch.empty((n, hk, d), dtype=dtype, device="cuda")
        return s
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
    s["k_cache"], s["v_cache"] = _cache(gen, pages, c, dtype), _cache(gen, pages, c, dtype)
    if c["op"] == "append":
        qkv = _randn(gen, (n, hq + 2 * hk, d), dtype, 1.5)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["rope"] = _rope(c["len"], c["rot"])
        s["q_out"] = torch.empty((n, hq, d), dtype=dtype, device="cuda")
        return s
    s["q"] = _randn(gen, (n, hq, d), dtype, 1.5)
    s["scale"] = 1 / math.sqrt(d)
    s["out"] = torch.empty((n, hq, d), dtype=dtype, device="cuda")
    s["lse"] = torch.empty((n, hq), device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def _workspace(s, size):
    """A program keeps its workspace from call to call."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s["workspace"]


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import sparse_dense_interaction_gb300 as sdi
    c = s["case"]
    if c["op"] == "norm_fwd":
        sdi.dlrm_qk_norm_rope_fwd(s["q"], s["k"], s["q_weight"], s["k_weight"], EPS, s["rope"], s["positions"],
                                  *s["out"], interleaved=c["interleaved"])
        return {"q": s["out"][0], "k": s["out"][1]}
    if c["op"] == "norm_bwd":
        ws = _workspace(s, sdi.dlrm_qk_norm_rope_bwd_workspace_size(c["n"], c["hq"], c["hk"], c["d"]))
        sdi.dlrm_qk_norm_rope_bwd(s["dq_out"], s["dk_out"], s["q"], s["k"], s["q_weight"], s["k_weight"], EPS,
                                  s["rope"], s["positions"], *s["out"], s["dq_weight"], s["dk_weight"], ws,
                                  interleaved=c["interleaved"])
        return {"dq": s["out"][0], "dk": s["out"][1], "dq_weight": s["dq_weight"], "dk_weight": s["dk_weight"]}
    if c["op"] == "append":
        norm = c["norm"]
        sdi.dlrm_kv_append(s["k"], s["v"], s["offsets"], s["lengths"], s["page_table"], s["k_cache"], s["v_cache"],
                           k_weight=s["k_weight"] if norm else None, eps=EPS, rope=s["rope"], q=s["q"],
                           q_weight=s["q_weight"] if norm else None, q_out=s["q_out"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    ws = _workspace(s, sdi.dlrm_kv_attn_workspace_size(c["S"], s["n"], c["hq"], c["hk"], c["d"], s["max_new"],
                                                       s["max_len"]))
    sdi.dlrm_kv_attn_fwd(s["q"], s["offsets"], s["lengths"], s["page_table"], s["k_cache"], s["v_cache"], s["out"],
                         s["scale"], ws, s["max_new"], s["max_len"], causal=c["causal"], window=c["window"],
                         lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _rotated(z, rope, positions, rot, interleaved, back=False):
    """z[n][heads][d] rotated by its positions' angles (back: by their negatives)."""
    row = rope[positions][:, None]
    cos, sin = row[..., :rot // 2], row[..., rot // 2:]
    sin = -sin if back else sin
    if interleaved:
        a, b = z[..., 0:rot:2], z[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = z[..., :rot // 2], z[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, z[..., rot:]], -1)


def _normed(x, weight):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def _places(s):
    """Sequence, number in its chunk and place in its history of each new token."""
    counts = s["offsets"][1:] - s["offsets"][:-1]
    seq = torch.repeat_interleave(torch.arange(counts.numel(), device="cuda"), counts, output_size=s["n"])
    i = torch.arange(s["n"], device="cuda") - s["offsets"][seq]
    return seq, i, (s["lengths"] - counts)[seq] + i


def _run_plain(s):
    c = s["case"]
    dtype, rot = DTYPES[c["dtype"]], c.get("rot")
    if c["op"] == "norm_fwd":
        q, k = (_rotated(_normed(x, w), s["rope"], s["positions"], rot, c["interleaved"])
                for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])))
        return {"q": q.to(dtype), "k": k.to(dtype)}
    if c["op"] == "norm_bwd":
        dq, dqw = _norm_gradient(s["dq_out"], s["q"], s["q_weight"], s)
        dk, dkw = _norm_gradient(s["dk_out"], s["k"], s["k_weight"], s)
        return {"dq": dq.to(dtype), "dk": dk.to(dtype), "dq_weight": dqw, "dk_weight": dkw}
    if c["op"] == "append":
        seq, _, at = _places(s)
        q = _normed(s["q"], s["q_weight"]) if c["norm"] else s["q"].float()
        k = _normed(s["k"], s["k_weight"]) if c["norm"] else s["k"].float()
        page, slot = s["page_table"][seq, at // c["page"]].long(), at % c["page"]
        s["k_cache"][page, slot] = _rotated(k, s["rope"], at, rot, False).to(dtype)
        s["v_cache"][page, slot] = s["v"]
        return {"q": _rotated(q, s["rope"], at, rot, False).to(dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return _attention(s)


def _norm_gradient(dy, x, weight, s):
    c = s["case"]
    dz = _rotated(dy.float(), s["rope"], s["positions"], c["rot"], c["interleaved"], back=True)
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    unit, g = x * r, dz * weight
    return r * (g - unit * (g * unit).mean(-1, keepdim=True)), (dz * unit).sum((0, 1))


def _attention(s):
    c = s["case"]
    S, hk, d, C, L = c["S"], c["hk"], c["d"], s["max_new"], s["max_len"]
    G = c["hq"] // hk
    seq, i, _ = _places(s)
    counts = s["offsets"][1:] - s["offsets"][:-1]
    j = torch.arange(L, device="cuda")
    stored = (j[None, :] < s["lengths"][:, None])[:, :, None, None]
    pages = s["page_table"].long().clamp(min=0)
    k, v = (torch.where(stored, t[pages].flatten(1, 2)[:, :L].float(), 0.0) for t in (s["k_cache"], s["v_cache"]))
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

def _turn64(z, rope, positions, rot, interleaved):
    """The rotation as a product of complex numbers."""
    row = rope.double()[positions]
    turn = torch.complex(row[:, :rot // 2], row[:, rot // 2:])[:, None]
    z = z.clone()
    if interleaved:
        w = torch.view_as_complex(z[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn
        z[..., :rot] = torch.view_as_real(w).flatten(-2)
    else:
        w = torch.complex(z[..., :rot // 2].contiguous(), z[..., rot // 2:rot].contiguous()) * turn
        z[..., :rot // 2], z[..., rot // 2:rot] = w.real, w.imag
    return z


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] in ("norm_fwd", "norm_bwd"):
        got = []
        for name in ("q", "k"):
            x = s[name].double().requires_grad_(c["op"] == "norm_bwd")
            w = s[name + "_weight"].double().requires_grad_(c["op"] == "norm_bwd")
            z = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * w
            if c["op"] == "norm_fwd":
                got.append(_turn64(z, s["rope"], s["positions"], c["rot"], c["interleaved"]))
                continue
            # the gradient of sum(dy * y), by torch's own differentiation in 64 bits
            back = s["rope"].clone()
            back[:, c["rot"] // 2:].neg_()
            dz = _turn64(s["d%s_out" % name].double(), back, s["positions"], c["rot"], c["interleaved"])
            (z * dz).sum().backward()
            got.append((x.grad, w.grad))
        if c["op"] == "norm_fwd":
            return {"q": got[0], "k": got[1]}
        return {"dq": got[0][0], "dk": got[1][0], "dq_weight": got[0][1], "dk_weight": got[1][1]}
    counts, lens = _lengths(c)
    table = s["page_table"].cpu()
    slots = [table[b, :-(-length // c["page"])].long() if length else table[b, :0].long() for b, length in enumerate(lens)]
    first = [0]
    for n in counts:
        first.append(first[-1] + n)
    if c["op"] == "append":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        at = torch.cat([torch.arange(length - n, length) for n, length in zip(counts, lens)]).cuda()
        page = torch.cat([slots[b][torch.arange(lens[b] - n, lens[b]) // c["page"]] for b, n in enumerate(counts)]).cuda()
        out = {}
        for name in ("q", "k"):
            x = s[name].double()
            if c["norm"]:
                x = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * s[name + "_weight"].double()
            out[name] = _turn64(x, s["rope"], at, c["rot"], False)
        kc[page, at % c["page"]] = out["k"]
        vc[page, at % c["page"]] = s["v"].double()
        return {"q": out["q"], "k_cache": kc, "v_cache": vc}
    G = c["hq"] // c["hk"]
    o = torch.zeros((s["n"], c["hq"], c["d"]), dtype=torch.float64, device="cuda")
    lse = torch.full((s["n"], c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, (n, length) in enumerate(zip(counts, lens)):
        if n == 0 or length == 0:
            continue
        at = slots[b].cuda()
        k, v = (t[at].flatten(0, 1)[:length].double() for t in (s["k_cache"], s["v_cache"]))
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
