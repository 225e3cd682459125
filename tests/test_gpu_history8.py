"""The event history in 8 bits on the GPU against 64-bit formulas: codes bit
for bit, attention within tolerances of its roundings; pages given out against
one-by-one bookkeeping."""
import numpy as np
import pytest
import torch

import sparse_dense_interaction_gb300 as sdi
from sparse_dense_interaction_gb300 import _native
from tests import _history8_ref as R8
from tests import _history_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_dense_interaction_gb300 import build
    build.build()


def randn(seed, shape, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DT[dtype]).to(DEV)


def flag():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def np64(t):
    return t.double().cpu().numpy()


def as64(x):
    return torch.tensor(x, dtype=torch.int64, device=DEV)


def table_of(lengths, page, seed=0, spare=2, width=2):
    """A page table of random pages, and how many there are."""
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + spare
    order = iter(np.random.RandomState(seed).permutation(pages))
    table = np.full((len(lengths), max(need + [1]) + width), -1, np.int32)
    for s, n in enumerate(need):
        table[s, :n] = [next(order) for _ in range(n)]
    return table, pages


def tensors8(codes, exps, first=False):
    """float8 codes (heads before slots in memory, if `first`) and uint8 exponents on the GPU."""
    c = torch.from_numpy(codes).to(DEV)
    if first:
        c = c.transpose(1, 2).contiguous().transpose(1, 2)
    return c.view(torch.float8_e4m3fn), torch.from_numpy(exps).to(DEV)


def cache8(seed, pages, page, block, heads, d, low=118, high=125):
    """Random finite codes and exponents."""
    r = np.random.RandomState(seed)
    codes = r.randint(0, 0x7F, (pages, page, heads, d)).astype(np.uint8)
    # sizes as encoded values have them: near the largest more often than far below it
    codes = np.where(r.rand(*codes.shape) < 0.9, np.maximum(codes, 0x58), codes)
    codes = (codes | r.randint(0, 2, codes.shape) << 7).astype(np.uint8)
    return codes, r.randint(low, high, (pages, page // block, heads)).astype(np.uint8)


def bytes_of(t):
    return t.view(torch.uint8).cpu().numpy()


# ---------------------------------------------------------------- append

APPEND = [
    # counts, lengths, heads, d, page, block, heads first, dtype
    ([1], [1], 1, 64, 16, 16, False, "f16"),
    ([1, 1, 1, 1], [1, 16, 17, 40], 2, 64, 16, 16, False, "f16"),
    ([5, 0, 40, 7], [9, 3, 40, 300], 4, 128, 64, 16, True, "bf16"),
    ([1] * 70, [1 + 13 * i for i in range(70)], 2, 64, 16, 8, False, "bf16"),
    ([300, 2], [301, 2], 8, 128, 64, 64, True, "bf16"),
    ([33, 100], [60, 133], 3, 96, 24, 8, False, "f32"),
    ([7, 19], [50, 19], 2, 80, 32, 1, False, "f16"),
    ([13, 4], [13, 29], 2, 17, 5, 5, False, "f32"),
    ([9, 70], [100, 71], 1, 256, 128, 128, True, "f16"),
    ([9, 70], [100, 71], 2, 30, 6, 3, False, "bf16"),
    ([1000], [1500], 1, 8, 1000, 500, False, "f32"),
    ([i % 4 for i in range(200)], [i % 4 + (i * 7) % 90 for i in range(200)], 1, 32, 8, 4, False, "bf16"),
]


@pytest.mark.parametrize("case", APPEND)
@pytest.mark.parametrize("sizes", ["alike", "wild"])
def test_append_bit_for_bit(case, sizes):
    counts, lengths, heads, d, page, block, first, dtype = case
    table, pages = table_of(lengths, page)
    n = sum(counts)
    k, v = (randn(s, (n, heads + 1, d), dtype, 1.5)[:, 1:] for s in (1, 2))
    if sizes == "wild":  # from token to token over most of fp16's range, whole rows of zeros, values not finite
        spread = torch.exp2(torch.randint(-20, 9, (n, heads, 1), generator=torch.Generator().manual_seed(3)).float())
        k, v = ((x.float() * spread.to(DEV)).to(DT[dtype]) for x in (k, v))
        k[::3] = 0
        v.view(-1)[::101] = float("inf")
        k.view(-1)[::77] = float("nan")
    caches = [cache8(10 + i, pages, page, block, heads, d) for i in (0, 1)]
    (kc, ke), (vc, ve) = (tensors8(*c, first) for c in caches)
    f = flag()
    sdi.dlrm_kv8_append(k, v, as64([0] + list(np.cumsum(counts))), as64(lengths), torch.from_numpy(table).to(DEV),
                        kc, vc, ke, ve, err_flag=f)
    assert sdi.dlrm_read_error(f) == 0
    for x, (codes, exps), c, e in ((k, caches[0], kc, ke), (v, caches[1], vc, ve)):
        R8.append(np64(x), codes, exps, counts, lengths, table, block)
        assert np.array_equal(e.cpu().numpy(), exps)
        got = bytes_of(c)
        nan = codes & 0x7F == 0x7F  # NaN's sign is free
        assert np.array_equal(np.where(nan, got & 0x7F, got), np.where(nan, codes & 0x7F, codes))


def test_append_one_token_at_a_time():
    # as serving does: exponents grow from step to step, older codes are rounded again
    page, block, heads, d = 16, 16, 2, 64
    table, pages = table_of([40], page)
    k, v = (randn(s, (40, heads, d), "bf16") for s in (4, 5))
    k *= torch.exp2(torch.randint(-8, 8, (40, 1, 1), generator=torch.Generator().manual_seed(6)).float()).to(DEV)
    caches = [cache8(10 + i, pages, page, block, heads, d) for i in (0, 1)]
    (kc, ke), (vc, ve) = (tensors8(*c) for c in caches)
    for i in range(40):
        sdi.dlrm_kv8_append(k[i:i + 1], v[i:i + 1], as64([0, 1]), as64([i + 1]), torch.from_numpy(table).to(DEV), kc, vc,
                            ke, ve)
        for x, c in ((k, caches[0]), (v, caches[1])):
            R8.append(np64(x[i:i + 1]), *c, [1], [i + 1], table, block)
    for (codes, exps), c, e in ((caches[0], kc, ke), (caches[1], vc, ve)):
        assert np.array_equal(bytes_of(c), codes) and np.array_equal(e.cpu().numpy(), exps)


def test_append_leaves_out_what_contradicts_itself():
    heads, d, page, block = 2, 64, 16, 8
    k, v = randn(1, (9, heads, d), "f16"), randn(2, (9, heads, d), "f16")
    for counts, lengths, bad, want in [
            ([3, 3, 3], [3, 2, 5], {1}, _native.ERR_BAD_OFFSETS),     # more new than stored
            ([3, 3, 3], [3, -1, 5], {1}, _native.ERR_BAD_OFFSETS),
            ([3, 3, 3], [3, 1000, 5], {1}, _native.ERR_BAD_OFFSETS),  # beyond the table
            ([3, 3, 3], [3, 20, 5], {2}, _native.ERR_INDEX_OOB)]:     # a page that is none
        table, pages = table_of([20, 20, 20], page)
        if bad == {2}:
            table[2, 0] = pages
        caches = [cache8(10 + i, pages, page, block, heads, d) for i in (0, 1)]
        (kc, ke), (vc, ve) = (tensors8(*c) for c in caches)
        f = flag()
        sdi.dlrm_kv8_append(k, v, as64([0, 3, 6, 9]), as64(lengths), torch.from_numpy(table).to(DEV), kc, vc, ke, ve,
                            err_flag=f)
        assert sdi.dlrm_read_error(f) == want
        for x, (codes, exps), c, e in ((k, caches[0], kc, ke), (v, caches[1], vc, ve)):
            for s in {0, 1, 2} - bad:
                R8.append(np64(x[3 * s:3 * s + 3]), codes, exps, [3], [lengths[s]], table[s:s + 1], block)
            assert np.array_equal(bytes_of(c), codes) and np.array_equal(e.cpu().numpy(), exps)


# ---------------------------------------------------------------- attention

ATTN = [
    # counts, lengths, q heads, kv heads, d, page, block, heads first, causal, window, dtype
    ([1], [1], 1, 1, 64, 16, 16, False, True, 0, "f16"),
    ([1, 1, 1], [0, 1, 33], 8, 2, 64, 16, 16, False, False, 0, "f16"),  # no history: empty rows
    ([1, 1, 1, 1, 1], [1, 15, 16, 17, 700], 4, 1, 128, 16, 8, True, True, 0, "bf16"),
    ([1, 1], [3000, 5], 6, 2, 128, 64, 64, True, True, 0, "bf16"),
    ([1], [5001], 8, 8, 64, 32, 16, False, True, 0, "f16"),
    ([1, 1], [900, 2000], 32, 2, 128, 8, 8, False, True, 0, "bf16"),  # 16 heads share one
    ([1, 1], [900, 2000], 40, 2, 64, 8, 1, False, True, 0, "f16"),  # 20 heads share one
    ([1, 1, 1], [777, 64, 65], 3, 1, 80, 24, 12, False, True, 100, "bf16"),
    ([2, 0, 4, 3], [40, 7, 4, 129], 4, 2, 96, 48, 16, True, True, 0, "f16"),
    ([3, 5], [2, 3], 2, 1, 64, 16, 16, False, True, 0, "bf16"),  # more new than stored: the first rows see nothing
    ([33, 70], [33, 200], 4, 4, 64, 16, 16, False, True, 0, "f16"),
    ([130, 1, 129], [130, 300, 515], 2, 1, 128, 64, 32, True, True, 0, "bf16"),
    ([64], [1000], 12, 4, 128, 16, 16, False, False, 0, "bf16"),
    ([200, 17], [400, 0], 3, 1, 128, 128, 128, True, False, 0, "f16"),
    ([150], [600], 4, 2, 64, 8, 8, False, True, 37, "bf16"),
    ([90, 260], [90, 700], 2, 2, 128, 32, 8, True, True, 200, "f16"),
    ([300], [300], 8, 1, 128, 256, 256, False, True, 0, "bf16"),
    ([50], [9000], 2, 1, 128, 64, 16, False, True, 0, "bf16"),  # few rows, long: split
    ([20], [9000], 4, 2, 64, 16, 16, True, False, 1500, "f16"),
    ([40, 3], [77, 500], 4, 2, 32, 16, 4, False, True, 0, "f16"),
    ([40, 3], [77, 500], 4, 2, 40, 1, 1, False, True, 0, "bf16"),
    ([1, 9, 2], [50, 90, 333], 4, 2, 64, 32, 32, False, True, 64, "f32"),
    ([1], [4000], 2, 1, 128, 16, 2, True, True, 0, "f32"),
    ([1, 30], [100, 260], 2, 2, 17, 5, 5, False, True, 0, "f32"),
    ([1, 30], [100, 260], 2, 2, 17, 5, 1, False, True, 0, "bf16"),
    ([3, 20], [100, 200], 2, 1, 256, 16, 16, False, True, 0, "bf16"),
    ([3, 20], [100, 200], 2, 1, 208, 16, 16, True, False, 50, "f32"),
    ([5 + i % 30 for i in range(270)], [3 + 37 * i % 200 for i in range(270)], 4, 2, 64, 16, 16, False, True, 0, "f16"),
    ([300], [5000], 2, 1, 64, 16, 16, True, True, 0, "bf16"),
    ([200, 5], [333, 64], 2, 1, 128, 7, 7, False, True, 0, "f16"),  # pages that end inside a tile, two query tiles
    ([140], [3001], 3, 1, 56, 3, 1, False, False, 700, "bf16"),
    ([1] * 40, [(i * i * 7) % 3001 for i in range(40)], 8, 2, 64, 16, 8, False, True, 0, "bf16"),
    ([i % 3 for i in range(300)], [(i * 61) % 1300 for i in range(300)], 2, 1, 64, 64, 32, True, False, 0, "f16"),
    ([16, 3], [1500, 2000], 1, 1, 128, 24, 8, False, True, 0, "bf16"),
    ([60, 1], [1100, 700], 3, 1, 64, 16, 16, True, True, 0, "f32"),
    ([1, 1, 1], [5000, 0, 77], 8, 2, 256, 16, 16, False, True, 0, "bf16"),
    ([3, 16], [900, 3300], 2, 2, 192, 24, 24, True, False, 0, "f16"),
    ([4, 2], [2500, 900], 4, 2, 256, 64, 16, True, True, 0, "f32"),
    ([260, 31], [260, 900], 2, 1, 256, 32, 32, False, True, 0, "f16"),
    ([180], [900], 2, 1, 80, 40, 8, False, False, 0, "f16"),
    # chunks of many rows, whose codes are converted once
    ([300, 40, 0], [700, 1000, 33], 16, 4, 64, 16, 8, False, True, 0, "bf16"),
    ([520], [1300], 4, 2, 128, 24, 24, True, True, 333, "bf16"),
    ([130, 2], [200, 0], 16, 2, 96, 7, 7, False, False, 0, "bf16"),
    # heads above 128 in tiles: parts, a window, pages that end inside a tile
    ([50, 0, 9], [3000, 5, 400], 4, 2, 256, 32, 16, True, True, 0, "bf16"),
    ([40, 33], [500, 700], 2, 2, 144, 7, 1, False, False, 90, "bf16"),
    ([20], [20000], 2, 1, 192, 64, 8, False, True, 0, "f16"),
]


def attention_inputs(case, seed=0, low=118, high=125):
    """Slots that nothing sees hold NaN codes, blocks that nothing sees exponents of 255; page numbers past the
    histories are -1, before the window -7."""
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, pages = table_of(lengths, page, seed)
    live = np.zeros((pages, page), bool)
    given = table.copy()
    for s, (c, n) in enumerate(zip(counts, lengths)):
        lo = 0
        if c == 0:
            lo = n
        elif window:
            hi = max(0, n - c + 1) if causal else n
            lo = max(0, hi - window)
        at = np.arange(lo, n)
        live[table[s, at // page], at % page] = True
        if lo >= page:  # pages before the window have been given back
            given[s, :lo // page] = -7
    caches = []
    for i in (0, 1):
        codes, exps = cache8(31 + i + seed, pages, page, block, hk, d, low, high)
        codes[~live] = 0x7F
        exps[~live.reshape(pages, page // block, block).any(2)] = 255
        caches.append((codes, exps))
    q = randn(41 + seed, (sum(counts), hq, d), dtype, 0.5)
    return table, given, caches, q


def attend(case, given, caches, q, scale, f=None, **kw):
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    n = sum(counts)
    out = torch.full((n, hq, d), 7, dtype=DT[dtype], device=DEV)
    lse = torch.full((n, hq), 7.0, device=DEV)
    sizes = (len(counts), n, hq, hk, d, max(counts), max(lengths))
    ws = torch.full((sdi.dlrm_kv8_attn_workspace_size(*sizes),), 255, dtype=torch.uint8, device=DEV)  # NaNs
    (kc, ke), (vc, ve) = (tensors8(*c, first) for c in caches)
    sdi.dlrm_kv8_attn_fwd(q, as64([0] + list(np.cumsum(counts))), as64(lengths), torch.from_numpy(given).to(DEV), kc, vc,
                          ke, ve, out, scale, ws, max(counts), max(lengths), causal=causal, window=window, lse=lse,
                          err_flag=f, **kw)
    return out, lse


def close(got, want, tol, what):
    got = np64(got)
    bad = ~(np.abs(got - want) <= tol) & ~(np.isneginf(got) & np.isneginf(want))
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4], np.broadcast_to(tol, got.shape)[bad][:4])


# The cache's values are exact in every kernel, so the formula's tolerance is that of the 16-bit cache,
# with products that are exact in fp32 and sums of as many.  Weights of 16-bit queries are rounded to fp16 in
# tiles (2^-11; no query type is finer), which the type's own rounding of the weight covers.  They are held
# relative to the largest weight times the largest power of two that the row's warp or tile has seen: down to
# 2^-25 of 2^15 (16 rows), 2^-25 of 2^11 (tiles), so what falls below is off by 2^-36 of the largest
# magnitude seen, for each of the row's weights.
def check_attention(case, table, caches, q, scale, out, lse, what="attention"):
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    with np.errstate(over="ignore", invalid="ignore"):
        k, v = (np.nan_to_num(R8.values(*c), nan=0.0, posinf=0.0, neginf=0.0) for c in caches)
    want, wl, absout, smax, flat = R.attention(np64(q), counts, lengths, table, k, v, scale, causal, window)
    tol = R.attention_tolerance(want, absout, smax, flat, d, dtype)
    largest = np.abs(v).max()
    tol = tol + 2.0 ** -36 * largest * max(lengths + [1])
    close(out, want, tol, (case, what))
    close(lse, wl, R.lse_tolerance(wl, smax, d), (case, what, "lse"))


@pytest.mark.parametrize("case", ATTN)
def test_attention(case):
    table, given, caches, q = attention_inputs(case)
    scale, f = 1 / case[4] ** 0.5, flag()
    out, lse = attend(case, given, caches, q, scale, f)
    assert sdi.dlrm_read_error(f) == 0
    check_attention(case, table, caches, q, scale, out, lse)
    again = attend(case, given, caches, q, scale)  # the same bits again
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


# ---------------------------------------------------------------- pages

RESERVE = [
    # sequences, most new, most stored, page, share that ends, pages free (of those wanted), seed
    (1, 1, 0, 16, 0.0, 1.0, 0), (1, 5000, 100, 16, 0.0, 2.0, 1), (8, 1, 300, 16, 0.1, 1.0, 2),
    (300, 40, 500, 8, 0.1, 0.6, 3), (2048, 1, 1000, 16, 0.05, 1.5, 4), (2049, 3, 100, 7, 0.3, 0.9, 5),
    (5000, 2, 64, 1, 0.2, 0.5, 6), (60, 900, 4000, 64, 0.2, 0.8, 7), (64, 900, 40, 100, 0.0, 0.0, 8),
    (700, 100, 300, 20, 0.0, 3.0, 9),
]


def reserve_inputs(case):
    S, new, stored, page, ends, share, seed = case
    r = np.random.RandomState(seed)
    lengths = r.randint(0, stored + 1, S)
    counts = np.where(r.rand(S) < ends, -1 - r.randint(0, 3, S), r.randint(0 if S > 1 else new, new + 1, S))
    held = -(-lengths // page)
    want = -(-(lengths + np.maximum(counts, 0)) // page) - held
    free, width = int(want.sum() * share), int((held + want).max()) + 1
    pages = max(int(held.sum()) + free, 1)
    order = r.permutation(pages).astype(np.int32)
    table = np.full((S, width), -1, np.int32)
    for s, at in enumerate(np.cumsum(held) - held):
        table[s, :held[s]] = order[at:at + held[s]]
    ring, head = np.full(pages, -3, np.int32), int(r.randint(0, 10 * pages))
    ring[(head + np.arange(free)) % pages] = order[held.sum():held.sum() + free]
    return counts, lengths, table, ring, [head, head + free]


@pytest.mark.parametrize("case", RESERVE)
@pytest.mark.parametrize("in_place", [False, True])
def test_reserve(case, in_place):
    page = case[3]
    counts, lengths, table, ring, state = reserve_inputs(case)
    n = int(np.maximum(counts, 0).sum())
    want = R8.reserve(counts.tolist(), lengths.tolist(), table, page, ring, state, n)
    gpu = [torch.from_numpy(np.asarray(x)).to(DEV) for x in (counts, lengths, table, ring)]
    c, l, t, r = gpu[0].long(), gpu[1].long(), gpu[2], gpu[3]
    st = as64(state)
    new_l, new_st = (l, st) if in_place else (torch.empty_like(l), torch.empty_like(st))
    offsets = torch.empty(len(counts) + 1, dtype=torch.int64, device=DEV)
    slots, positions = (torch.full((n + 3,), -9, dtype=torch.int64, device=DEV) for _ in range(2))
    f = flag()
    sdi.dlrm_kv_reserve(c, l, t, page, r, st, new_st, offsets, new_l, slots[:n], positions[:n], err_flag=f)
    assert sdi.dlrm_read_error(f) == (_native.ERR_CAPACITY if want[7] else 0)
    for got, w in zip((offsets, new_l, t, r, new_st, slots[:n], positions[:n]), want):
        assert np.array_equal(got.cpu().numpy(), np.asarray(w))
    assert (slots[n:] == -9).all() and (positions[n:] == -9).all()
