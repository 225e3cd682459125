"""Event-history calls where a type's range, a NaN or a batch's own numbers
meet their edges, against the 64-bit formulas."""
import numpy as np
import pytest
import torch

import sparse_dense_interaction_gb300 as sdi
from sparse_dense_interaction_gb300 import _native
from tests import _history_ref as R
from tests.test_gpu_history import (
    APPEND, DEV, DT, EPS, NORM, attend, attention_inputs, check_attention, close, flag, heads_of, make_batch, make_cache, norm_inputs,
    np64, randn, rope_table)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_dense_interaction_gb300 import build
    build.build()


# (counts, lengths, q heads, kv heads, d, page, heads first, causal, window, dtype) as the calls take them: rows of
# 16, whole and shared out, bulk copies and rows; tiles of 128 and 256, one part and several; the general kernel
WEIGHTS = [
    ([1], [1000], 4, 1, 64, 16, False, True, 0, "f16"), ([1, 1], [700, 1000], 2, 1, 128, 7, False, True, 0, "f16"),
    ([1], [40000], 4, 1, 128, 16, True, True, 0, "f16"), ([4], [3000], 4, 1, 256, 16, False, False, 0, "f16"),
    ([9], [700], 4, 1, 64, 16, False, False, 0, "f16"), ([9], [20000], 4, 1, 128, 64, True, True, 0, "f16"),
    ([70], [1500], 4, 1, 128, 24, False, True, 0, "f16"), ([20], [3000], 1, 1, 64, 5, False, False, 0, "f16"),
    ([2], [3000], 2, 1, 20, 5, False, True, 0, "f16"), ([9], [20000], 4, 1, 128, 64, True, True, 0, "bf16"),
    ([1], [1000], 4, 1, 64, 16, False, True, 0, "bf16"), ([1], [1000], 4, 1, 64, 16, False, True, 0, "f32"),
]


@pytest.mark.parametrize("strong", ["first", "every 16th"])
@pytest.mark.parametrize("gap", [17.5, 17.25, 10.5])
@pytest.mark.parametrize("case", WEIGHTS)
def test_attention_weights_far_below_the_strongest(case, gap, strong):
    """Strong keys of value 0 and many weak ones: all that is gathered comes
    from weights 2^-25 of the strongest (2^-15), below f16's own range.

    A weight is rounded to the type: by U of itself, or, where a 16-bit type's range
    ends, by half of its smallest step, which is 2^-33 of the strongest weight at
    most."""
    counts, lengths, hq, hk, d, page, first, causal, window, dtype = case
    table, table_d, offsets, lens, kc, vc, q = attention_inputs(case, stale=0.0)
    q.zero_()
    q[..., 0] = 4
    kc.zero_()
    vc.uniform_(0.5, 1.5, generator=torch.Generator(device=DEV).manual_seed(1))
    for s, length in enumerate(lengths):
        at = np.arange(1) if strong == "first" else np.arange(0, length // 2, 16)
        page_of, slot = (torch.from_numpy(a).long().to(DEV) for a in (table[s, at // page], at % page))
        kc[page_of, slot, :, 0] = gap / 4
        vc[page_of, slot] = 0
    out, lse = attend(case, q, offsets, lens, table_d, kc, vc, 1.0)
    want, wl, absout, smax, flat = R.attention(np64(q), counts, lengths, table, np64(kc), np64(vc), 1.0, causal, window)
    score = (d + 4) * 2.0 ** -23 * smax[..., None]
    weight = 0.0 if dtype == "f32" else R.U[dtype]
    tol = (2 * score + 2.0 ** -18 + weight) * absout + R.U[dtype] * np.abs(want) * 1.01 + R.TINY[dtype]
    close(out, want, tol + (flat * 2.0 ** -33 if dtype == "f16" else 0), case)
    close(lse, wl, R.lse_tolerance(wl, smax, d), (case, "lse"))


@pytest.mark.parametrize("case", [
    ([1, 1], [300, 40], 4, 2, 64, 16, False, True, 0, "f16"), ([1, 1], [40000, 40], 4, 2, 128, 16, True, True, 0, "bf16"),
    ([3, 2], [3000, 40], 4, 2, 64, 16, True, True, 0, "f32"), ([40, 9], [100, 40], 4, 2, 64, 16, False, False, 0, "bf16"),
    ([40, 9], [9000, 40], 4, 2, 128, 16, False, True, 0, "f16"), ([40, 9], [900, 40], 4, 2, 128, 5, False, True, 64, "f16"),
    ([1, 3], [3000, 40], 4, 2, 20, 5, False, True, 0, "f32"), ([1, 3], [40, 90], 4, 2, 20, 5, False, True, 0, "bf16"),
])
def test_a_query_of_nan_gives_nan(case):
    # and not the zeros of a row that sees nothing; no other row knows of it
    hq = case[2]
    table, table_d, offsets, lens, kc, vc, q = attention_inputs(case)
    out, lse = attend(case, q, offsets, lens, table_d, kc, vc, 0.125)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    bad[0, 1] = bad[-1, hq - 1] = True
    q[bad, 5] = float("nan")
    got, got_lse = attend(case, q, offsets, lens, table_d, kc, vc, 0.125)
    assert got[bad].isnan().all() and got_lse[bad].isnan().all()
    assert torch.equal(got[~bad], out[~bad]) and torch.equal(got_lse[~bad], lse[~bad])


# an idle sequence in the middle: rows of 16, whole and shared out; tiles, ranked and in the batch's order; general
CONTRADICTED = [
    ([2, 0, 2], [60, 40, 50], 4, 2, 64, 16, False, True, 0, "bf16"), ([2, 0, 2], [9000, 40, 50], 4, 2, 64, 16, True, True, 0, "f16"),
    ([2, 0, 2], [60, 40, 50], 4, 2, 64, 16, False, True, 0, "f32"), ([40, 0, 40], [60, 40, 50], 4, 2, 64, 16, False, True, 0, "f16"),
    ([20] + [0] * 300 + [20], [60] + [40] * 300 + [50], 4, 2, 128, 16, True, True, 0, "bf16"),
    ([2, 0, 2], [60, 40, 50], 4, 2, 20, 7, False, True, 0, "f32"), ([2, 0, 2], [60, 40, 50], 4, 2, 20, 7, False, True, 0, "bf16"),
]


@pytest.mark.parametrize("what", ["idle and negative", "idle and beyond its table", "first token", "last token"])
@pytest.mark.parametrize("case", CONTRADICTED)
def test_contradictions_of_a_batch_are_flagged_by_every_call(case, what):
    counts, lengths, hq, hk, d, page, first, causal, window, dtype = case
    table, table_d, offsets, lens, kc, vc, q = attention_inputs(case, stale=0.0)
    n, c, S = q.shape[0], counts[0], len(counts)
    good, good_lse = attend(case, q, offsets, lens, table_d, kc, vc, 0.125, f := flag())
    assert sdi.dlrm_read_error(f) == 0
    k, v = q[:, :hk].contiguous(), q[:, hk:2 * hk].contiguous()
    kc1, vc1 = kc.clone(), vc.clone()
    sdi.dlrm_kv_append(k, v, offsets, lens, table_d, kc1, vc1, err_flag=(f := flag()))
    assert sdi.dlrm_read_error(f) == 0
    same, left_out = slice(0, n), slice(0, 0)
    if what == "idle and negative":
        lens[1] = -1
    elif what == "idle and beyond its table":
        lens[1] = table_d.shape[1] * page + 1
    elif what == "first token":
        offsets[0], same, left_out = 1, slice(c, n), slice(0, 1)
    else:
        offsets[S], same, left_out = n - 1, slice(0, c), slice(n - 1, n)
    out, lse = attend(case, q, offsets, lens, table_d, kc, vc, 0.125, f := flag())
    assert sdi.dlrm_read_error(f) == _native.ERR_BAD_OFFSETS
    assert torch.equal(out[same], good[same]) and torch.equal(lse[same], good_lse[same])
    assert (out[left_out] == 7).all() and (lse[left_out] == 7).all()
    kc2, vc2 = kc.clone(), vc.clone()
    sdi.dlrm_kv_append(k, v, offsets, lens, table_d, kc2, vc2, err_flag=(f := flag()))
    assert sdi.dlrm_read_error(f) == _native.ERR_BAD_OFFSETS
    at = np.concatenate([np.arange(m - e, m) for e, m in zip(counts, lengths)])
    pages = table[np.repeat(np.arange(S), counts), at // page]
    for got, want, before in ((kc2, kc1, kc), (vc2, vc1, vc)):
        if what.startswith("idle"):
            assert torch.equal(got, want)
        else:  # the other sequences' tokens are stored, the token of nobody is not
            assert np.array_equal(np64(got)[pages[same], at[same] % page], np64(want)[pages[same], at[same] % page])


def idle_batch(busy, idle, where, length, dtype):
    """`busy` users with up to `length` events and one new among `idle` slots without."""
    S = busy + idle
    at = {"ends": np.linspace(0, S - 1, busy).astype(int), "last": np.arange(idle, S),
          "anywhere": np.sort(np.random.default_rng(S).permutation(S)[:busy])}[where]
    counts, lengths = np.zeros(S, int), np.full(S, 5)
    counts[at] = 1
    lengths[at] = length - np.arange(busy) * (length // (busy + 1))
    return counts.tolist(), lengths.tolist(), 4, 1, 64, 16, True, True, 0, dtype


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["ends", "last", "anywhere"])
@pytest.mark.parametrize("busy,idle,length", [(2, 1, 20000), (2, 31, 20000), (3, 127, 9000), (9, 1500, 9000), (2, 3000, 30000)])
def test_attention_among_idle_users(busy, idle, length, where, dtype):
    case = idle_batch(busy, idle, where, length, dtype)
    table, table_d, offsets, lens, kc, vc, q = attention_inputs(case)
    f = flag()
    out, lse = attend(case, q, offsets, lens, table_d, kc, vc, 0.125, f)
    assert sdi.dlrm_read_error(f) == 0
    check_attention(case, q, table, kc, vc, 0.125, out, lse)


def test_idle_users_cost_little():
    # 3000 slots between two long histories: 47 us beside 36 without them, 1231 when they were passed one by one
    def best(idle):
        case = idle_batch(2, idle, "ends", 200000, "bf16")
        _, table_d, offsets, lens, kc, vc, q = attention_inputs(case)
        out = torch.empty_like(q)
        ws = torch.empty(sdi.dlrm_kv_attn_workspace_size(2 + idle, 2, 4, 1, 64, 1, 200000), dtype=torch.uint8, device=DEV)
        times = []
        for _ in range(30):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            sdi.dlrm_kv_attn_fwd(q, offsets, lens, table_d, kc, vc, out, 0.125, ws, 1, 200000)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)
    assert best(3000) < 5 * best(0)


@pytest.mark.parametrize("case", NORM)
@pytest.mark.parametrize("normed", [True, False])
def test_norm_rope_and_gradient_in_place(case, normed):
    n, hq, hk, d, rot, inter, dtype, pad = case
    x, w, table, at = norm_inputs(case)
    if not normed:
        w = {"q": None, "k": None}
    copy = lambda t: {a: None if u is None else heads_of(9, n, u.shape[1], d, dtype, pad).copy_(u) for a, u in t.items()}
    run = lambda x, out: sdi.dlrm_qk_norm_rope_fwd(x["q"], x["k"], w["q"], w["k"], EPS, table, at, out["q"], out["k"],
                                                   interleaved=inter)
    want, got = copy(x), copy(x)
    run(x, want)
    run(got, got)
    for a in x:
        assert x[a] is None or torch.equal(got[a], want[a])
    dy = {a: heads_of(11, n, t.shape[1], d, dtype, pad, 1.0) if t is not None else None for a, t in x.items()}
    ws = torch.empty(sdi.dlrm_qk_norm_rope_bwd_workspace_size(n, hq, hk, d), dtype=torch.uint8, device=DEV)

    def back(dy, x, dx):
        dw = {a: torch.empty(d, device=DEV) if normed and x[a] is not None else None for a in x}
        sdi.dlrm_qk_norm_rope_bwd(dy["q"], dy["k"], x["q"], x["k"], w["q"], w["k"], EPS, table, at, dx["q"], dx["k"],
                                  dw["q"], dw["k"], ws, interleaved=inter)
        return dw

    want, over_dy, over_x = copy(x), copy(dy), copy(x)
    results = [back(dy, x, want), back(over_dy, x, over_dy), back(dy, over_x, over_x)]
    for a in x:
        if x[a] is not None:
            assert torch.equal(over_dy[a], want[a]) and torch.equal(over_x[a], want[a])
            assert not normed or all(torch.equal(r[a], results[0][a]) for r in results)


@pytest.mark.parametrize("case", [c for c in APPEND if c[2]])
def test_append_turns_its_queries_in_place(case):
    counts, lengths, hq, hk, d, rot, page, first, normed, inter, dtype = case
    n = sum(counts)
    _, table_d, offsets, lens, pages = make_batch(counts, lengths, page)
    kc, vc = (make_cache(s, pages, page, hk, d, dtype, first) for s in (21, 22))
    qkv = randn(23, (n, hq + 2 * hk, d), dtype, 1.5)
    weight = 1 + 0.3 * randn(3, (d,), "f32") if normed else None

    def run(q, q_out):
        sdi.dlrm_kv_append(qkv[:, hq:hq + hk], qkv[:, hq + hk:], offsets, lens, table_d, kc, vc, k_weight=weight, eps=EPS,
                           rope=rope_table(max(lengths), rot), interleaved=inter, q=q, q_weight=weight, q_out=q_out)
        return q_out

    want = run(qkv[:, :hq], torch.empty((n, hq, d), dtype=DT[dtype], device=DEV))
    assert torch.equal(run(qkv[:, :hq], qkv[:, :hq]), want)


@pytest.mark.parametrize("bad", [[0, 3, 1, 2, 4], [4, 3, 2, 1, 0], [-5, 1, 2, 1 << 40, 4], [1, 1, 1, 1, 1], [0, 1, 2, 1, 4],
                                 [0, 4, 0, 4, 4], [2, 3, 0, 1, 2], [-(1 << 62), 1 << 62, 0, 1, 2]])
@pytest.mark.parametrize("c,length,d,dtype", [(1, 40, 64, "bf16"), (1, 9000, 64, "f16"), (40, 40, 64, "f16"), (40, 9000, 128, "bf16"),
                                              (2, 40, 64, "f32"), (2, 40, 20, "f32"), (1, 5000, 20, "bf16"), (5, 300, 200, "f16")])
def test_offsets_that_fall_touch_only_what_a_sound_sequence_owns(c, length, d, dtype, bad):
    """Rows and slots hold what their sequence gives them, or what they held."""
    hq, hk, page, S, n = 4, 2, 16, 4, 4 * c
    case = ([c] * S, [length] * S, hq, hk, d, page, False, True, 0, dtype)
    table, table_d, _, lens, kc, vc, q = attention_inputs(case, stale=0.0)
    offsets = [o * c if abs(o) <= 5 else o for o in bad]
    offsets_d = torch.tensor(offsets, device=DEV)
    guard, size = 1024, n * hq * d
    buf, lse_buf = torch.full((size + 2 * guard,), 7, dtype=DT[dtype], device=DEV), torch.full((n * hq + 2 * guard,), 7.0, device=DEV)
    out, lse = buf[guard:guard + size].view(n, hq, d), lse_buf[guard:guard + n * hq].view(n, hq)
    ws = torch.full((sdi.dlrm_kv_attn_workspace_size(S, n, hq, hk, d, c, length),), 255, dtype=torch.uint8, device=DEV)
    sdi.dlrm_kv_attn_fwd(q, offsets_d, lens, table_d, kc, vc, out, 0.125, ws, c, length, lse=lse, err_flag=(f := flag()))
    assert sdi.dlrm_read_error(f) == _native.ERR_BAD_OFFSETS
    for b in (buf, lse_buf):
        assert (b[:guard] == 7).all() and (b[-guard:] == 7).all()
    sound = [s for s in range(S) if 0 <= offsets[s] <= offsets[s + 1] <= n]
    right = torch.zeros((n, hq), dtype=torch.bool, device=DEV)
    for s in sound:
        a, e = offsets[s], offsets[s + 1]
        if not 0 < e - a <= c:
            continue
        want, wl, absout, smax, flat = R.attention(np64(q[a:e]), [e - a], [length], table[s:s + 1], np64(kc), np64(vc), 0.125, True, 0)
        tol = R.attention_tolerance(want, absout, smax, flat, d, dtype)
        right[a:e] |= torch.from_numpy((np.abs(np64(out[a:e]) - want) <= tol).all(-1) &
                                       (np.abs(np64(lse[a:e]) - wl) <= R.lse_tolerance(wl, smax, d))).to(DEV)
    assert (right | ((out == 7).all(-1) & (lse == 7))).all()

    # the append: a slot may hold a token of a sound sequence that has its place there, or what it held
    k, v = q[:, :hk].contiguous(), q[:, hk:].contiguous()
    kc2, vc2 = kc.clone(), vc.clone()
    sdi.dlrm_kv_append(k, v, offsets_d, lens, table_d, kc2, vc2, err_flag=(f := flag()))
    assert sdi.dlrm_read_error(f) == _native.ERR_BAD_OFFSETS
    same = (kc2 == kc).flatten(2).all(-1) & (vc2 == vc).flatten(2).all(-1)
    for s in sound:
        a, e = offsets[s], offsets[s + 1]
        if e - a <= length:
            at = np.arange(length - (e - a), length)
            pages, slots = (torch.from_numpy(x).long().to(DEV) for x in (table[s, at // page], at % page))
            same[pages, slots] |= (kc2[pages, slots] == k[a:e]).flatten(1).all(-1) & (vc2[pages, slots] == v[a:e]).flatten(1).all(-1)
    assert same.all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts,lengths,hq,hk,d,page", [
    ([1] * 20, list(range(10, 2010, 100)), 4, 2, 64, 16), ([1], [20000], 8, 1, 128, 16), ([1] * 6, list(range(50, 350, 50)), 4, 1, 256, 8),
    ([2, 1], [900, 300], 4, 1, 96, 7), ([4] * 9, [700] * 9, 2, 1, 40, 32)])
def test_attention_of_few_rows_rounds_its_output_once(counts, lengths, hq, hk, d, page, dtype):
    """Up to 8 rows carry their weights in two parts: of U of a weight, U is left.

    The sum of p |v| is off by the scores' roundings and by U^2; the output is then
    rounded to the type (small scores, so that theirs do not hide it)."""
    case = (counts, lengths, hq, hk, d, page, True, True, 0, dtype)
    table, table_d, offsets, lens, kc, vc, q = attention_inputs(case)
    scale = 0.1 / d ** 0.5
    out, _ = attend(case, q, offsets, lens, table_d, kc, vc, scale)
    k, v = (np.nan_to_num(np64(t), nan=0.0) for t in (kc, vc))
    want, _, absout, smax, flat = R.attention(np64(q), counts, lengths, table, k, v, scale, True, 0)
    score = (d + 4) * 2.0 ** -23 * smax[..., None]
    close(out, want, (2 * score + 2.0 ** -18 + 2 * R.U[dtype] ** 2) * absout + R.U[dtype] * np.abs(want) * 1.01 + R.TINY[dtype], case)


FORMS = [
    # fp32 bulk copies of columns that reach past the head's width
    ([3, 1], [300, 77], 4, 2, 40, 16, False, True, 0, "f32"), ([1, 2], [900, 50], 2, 2, 96, 8, True, False, 0, "f32"),
    ([5], [200], 3, 1, 24, 32, False, True, 30, "f32"), ([2], [3000], 4, 1, 100, 16, True, True, 0, "f32"),
    ([1, 1], [40, 90], 2, 1, 4, 8, False, True, 0, "f32"), ([9], [500], 4, 2, 124, 24, False, True, 0, "f32"),
    # the same in 16 bits, rows of 16 and tiles
    ([2, 1], [300, 77], 4, 2, 8, 16, False, True, 0, "bf16"), ([1], [5000], 4, 1, 72, 16, True, True, 0, "f16"),
    ([70, 3], [300, 77], 2, 2, 24, 16, False, True, 0, "f16"), ([40], [1000], 4, 1, 104, 32, True, False, 0, "bf16"),
    # prompts in fp32 and of 16-bit heads above 128
    ([300], [300], 2, 1, 64, 16, False, True, 0, "f32"), ([150, 200], [900, 200], 2, 2, 128, 32, True, True, 70, "f32"),
    ([150, 7], [150, 400], 2, 1, 256, 16, False, True, 0, "bf16"), ([200], [700], 3, 1, 192, 7, True, True, 40, "f16"),
    ([130], [400], 2, 2, 136, 8, False, False, 0, "bf16"),
    # tiles in the batch's order by their number: more than five for each place
    ([9] * 200, [9 + (i * 37) % 120 for i in range(200)], 16, 4, 128, 16, False, True, 0, "bf16"),
    ([6] * 200, [6 + (i * 37) % 90 for i in range(200)], 32, 8, 64, 16, False, True, 0, "f16"),
]


@pytest.mark.parametrize("case", FORMS)
def test_attention_of_further_forms(case):
    table, table_d, offsets, lens, kc, vc, q = attention_inputs(case)
    f = flag()
    out, lse = attend(case, q, offsets, lens, table_d, kc, vc, case[4] ** -0.5, f)
    assert sdi.dlrm_read_error(f) == 0
    check_attention(case, q, table, kc, vc, case[4] ** -0.5, out, lse)
    again = attend(case, q, offsets, lens, table_d, kc, vc, case[4] ** -0.5)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
