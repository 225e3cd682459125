"""Event-history operators on the GPU against 64-bit formulas: types, head
layouts, odd widths and lengths, empty rows, stale and invalid pages."""
import numpy as np
import pytest
import torch

import sparse_dense_interaction_gb300 as sdi
from sparse_dense_interaction_gb300 import _native
from tests import _history_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_dense_interaction_gb300 import build
    build.build()


def np64(t):
    return t.double().cpu().numpy()


def randn(seed, shape, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DT[dtype]).to(DEV)


def rope_table(length, rot, base=1000.0):
    a = torch.arange(length, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([a.cos(), a.sin()], 1).float().to(DEV)


def flag():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def close(got, want, tol, what):
    got = np64(got) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - want) <= tol) & ~(np.isneginf(got) & np.isneginf(want))
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4], np.broadcast_to(tol, got.shape)[bad][:4])


# (n, q heads, k heads, d, rot, interleaved, dtype, pad): pad elements between rows of heads
NORM = [
    (1, 1, 1, 64, 64, False, "f16", 0), (7, 3, 1, 128, 128, False, "bf16", 0), (33, 8, 2, 128, 64, False, "bf16", 8),
    (65, 4, 4, 64, 32, True, "f32", 0), (130, 2, 1, 96, 96, False, "f16", 16), (5, 2, 2, 80, 40, False, "bf16", 0),
    (9, 1, 1, 256, 256, True, "f16", 0), (12, 2, 1, 32, 32, False, "f32", 0), (31, 2, 3, 17, 16, False, "f32", 0),
    (4, 2, 1, 1, 0, False, "f32", 0), (6, 1, 2, 250, 6, True, "bf16", 1), (40, 2, 2, 64, 48, False, "bf16", 3),
    (300, 5, 0, 128, 128, True, "bf16", 0), (3, 40, 5, 64, 64, False, "f16", 0), (17, 1, 1, 8, 8, True, "f32", 0),
    (23, 6, 2, 24, 16, False, "f16", 0), (2051, 3, 1, 64, 64, False, "bf16", 0), (19, 2, 1, 200, 160, False, "f32", 0),
]


def heads_of(seed, n, heads, d, dtype, pad, scale=1.5):
    return randn(seed, (n, heads, d + pad), dtype, scale)[:, :, :d]


def norm_inputs(case):
    n, hq, hk, d, rot, _, dtype, pad = case
    x = {"q": heads_of(1, n, hq, d, dtype, pad), "k": heads_of(2, n, hk, d, dtype, pad) if hk else None}
    w = {a: (1 + 0.3 * randn(s, (d,), "f32")) for a, s in (("q", 3), ("k", 4))}
    table = rope_table(50, rot) if rot else None
    at = torch.randint(0, 50, (n,), generator=torch.Generator().manual_seed(5)).to(DEV)
    return x, w, table, at


@pytest.mark.parametrize("case", NORM)
@pytest.mark.parametrize("normed", [True, False])
def test_norm_rope(case, normed):
    n, hq, hk, d, rot, inter, dtype, pad = case
    x, w, table, at = norm_inputs(case)
    out = {a: torch.full_like(heads_of(9, n, t.shape[1], d, dtype, pad), 7) if t is not None else None
           for a, t in x.items()}
    f = flag()
    sdi.dlrm_qk_norm_rope_fwd(x["q"], x["k"], w["q"] if normed else None, w["k"] if normed else None, EPS, table, at,
                              out["q"], out["k"], interleaved=inter, err_flag=f)
    assert sdi.dlrm_read_error(f) == 0
    for a in ("q", "k") if hk else ("q",):
        y, mag = R.norm_rope(np64(x[a]), np64(w[a]) if normed else None, EPS, None if table is None else np64(table),
                             at.cpu().numpy(), inter)
        close(out[a], y, R.rows_tolerance(y, mag, dtype), (case, a))


@pytest.mark.parametrize("case", NORM)
@pytest.mark.parametrize("normed", [True, False])
def test_norm_rope_gradient(case, normed):
    n, hq, hk, d, rot, inter, dtype, pad = case
    x, w, table, at = norm_inputs(case)
    dy = {a: heads_of(11, n, t.shape[1], d, dtype, pad, 1.0) if t is not None else None for a, t in x.items()}
    dx = {a: torch.full_like(t, 7) if t is not None else None for a, t in x.items()}
    dw = {a: torch.full((d,), 7.0, device=DEV) if normed and x[a] is not None else None for a in x}
    ws = torch.full((sdi.dlrm_qk_norm_rope_bwd_workspace_size(n, hq, hk, d),), 255, dtype=torch.uint8, device=DEV)
    f = flag()
    call = lambda dx, dw: sdi.dlrm_qk_norm_rope_bwd(
        dy["q"], dy["k"], x["q"], x["k"], w["q"] if normed else None, w["k"] if normed else None, EPS, table, at,
        dx["q"], dx["k"], dw["q"], dw["k"], ws, interleaved=inter, err_flag=f)
    call(dx, dw)
    assert sdi.dlrm_read_error(f) == 0
    for a in ("q", "k") if hk else ("q",):
        want, mag, wsum, wmag = R.norm_rope_bwd(np64(dy[a]), np64(x[a]), np64(w[a]) if normed else None, EPS,
                                                None if table is None else np64(table), at.cpu().numpy(), inter)
        close(dx[a], want, R.rows_tolerance(want, mag, dtype, 32), (case, a))
        if normed:
            close(dw[a], wsum, R.weight_tolerance(wmag, 64 + n * x[a].shape[1] // 64), (case, a, "weight"))
    again = ({a: None if t is None else torch.empty_like(t) for a, t in dx.items()},
             {a: None if t is None else torch.empty_like(t) for a, t in dw.items()})
    call(*again)  # the same bits again
    for a in dx:
        assert dx[a] is None or torch.equal(dx[a], again[0][a])
        assert dw[a] is None or torch.equal(dw[a], again[1][a])


def test_norm_rope_gradient_against_differences():
    # the GPU's gradient in f32 against second-order differences of the 64-bit
    # forward: off by the GPU's roundings and by h^2 of the third derivative
    case = (3, 2, 1, 16, 8, False, "f32", 0)
    x, w, table, at = norm_inputs(case)
    dy = {a: heads_of(11, 3, t.shape[1], 16, "f32", 0, 1.0) for a, t in x.items()}
    dx, dw = {a: torch.empty_like(t) for a, t in x.items()}, {a: torch.empty_like(w[a]) for a in x}
    ws = torch.empty(sdi.dlrm_qk_norm_rope_bwd_workspace_size(3, 2, 1, 16), dtype=torch.uint8, device=DEV)
    sdi.dlrm_qk_norm_rope_bwd(dy["q"], dy["k"], x["q"], x["k"], w["q"], w["k"], EPS, table, at, dx["q"], dx["k"],
                              dw["q"], dw["k"], ws)
    for a in x:
        x64, w64, dy64 = np64(x[a]), np64(w[a]), np64(dy[a])
        f = lambda x, w: (R.norm_rope(x, w, EPS, np64(table), at.cpu().numpy())[0] * dy64).sum()
        for base, got, which in ((x64, np64(dx[a]), 0), (w64, np64(dw[a]), 1)):
            for i in np.ndindex(base.shape):
                e = np.zeros_like(base)
                e[i] = 1e-5
                args = ((x64 + e, w64), (x64 - e, w64)) if which == 0 else ((x64, w64 + e), (x64, w64 - e))
                assert abs((f(*args[0]) - f(*args[1])) / 2e-5 - got[i]) < 2e-5, (a, which, i)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 17)])
def test_norm_rope_positions_outside_the_table(dtype, d):
    x = randn(1, (6, 2, d), dtype)
    w, table = torch.ones(d, device=DEV), rope_table(10, 16)
    at = torch.tensor([0, -1, 9, 10, 1 << 40, 3], device=DEV)
    out, f = torch.full_like(x, 7), flag()
    sdi.dlrm_qk_norm_rope_fwd(x, None, w, None, EPS, table, at, out, None, err_flag=f)
    assert sdi.dlrm_read_error(f) == _native.ERR_INDEX_OOB
    bad = torch.tensor([False, True, False, True, True, False], device=DEV)
    assert not out[bad].any()
    good = (~bad).cpu().numpy()
    y, mag = R.norm_rope(np64(x)[good], np64(w), EPS, np64(table), at.cpu().numpy()[good])
    close(out[~bad], y, R.rows_tolerance(y, mag, dtype), "good rows")
    # in the gradient they add nothing
    dy, dx, dw = randn(2, x.shape, dtype), torch.full_like(x, 7), torch.empty(d, device=DEV)
    ws = torch.empty(sdi.dlrm_qk_norm_rope_bwd_workspace_size(6, 2, 0, d), dtype=torch.uint8, device=DEV)
    sdi.dlrm_qk_norm_rope_bwd(dy, None, x, None, w, None, EPS, table, at, dx, None, dw, None, ws)
    assert not dx[bad].any()
    want, mag, ws_, wm = R.norm_rope_bwd(np64(dy)[good], np64(x)[good], np64(w), EPS, np64(table), at.cpu().numpy()[good])
    close(dx[~bad], want, R.rows_tolerance(want, mag, dtype, 32), "good gradients")
    close(dw, ws_, R.weight_tolerance(wm, 64), "weight")


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 18)])
def test_norm_rope_of_broadcast_inputs(dtype, d):
    # one row for all heads, one gradient for all tokens: strides of 0
    n, h = 9, 3
    row, dy = randn(1, (n, 1, d), dtype, 1.5), randn(2, (1, h, d), dtype)
    x, dyx = row.expand(n, h, d), dy.expand(n, h, d)
    w, table, at = 1 + 0.3 * randn(3, (d,), "f32"), rope_table(20, 16), torch.arange(n, device=DEV)
    out, dx, dw = torch.empty((n, h, d), dtype=DT[dtype], device=DEV), torch.empty((n, h, d), dtype=DT[dtype], device=DEV), torch.empty(d, device=DEV)
    sdi.dlrm_qk_norm_rope_fwd(x, None, w, None, EPS, table, at, out, None)
    y, mag = R.norm_rope(np64(x), np64(w), EPS, np64(table), at.cpu().numpy())
    close(out, y, R.rows_tolerance(y, mag, dtype), "broadcast rows")
    ws = torch.empty(sdi.dlrm_qk_norm_rope_bwd_workspace_size(n, h, 0, d), dtype=torch.uint8, device=DEV)
    sdi.dlrm_qk_norm_rope_bwd(dyx, None, x, None, w, None, EPS, table, at, dx, None, dw, None, ws)
    want, mag, wsum, wmag = R.norm_rope_bwd(np64(dyx), np64(x), np64(w), EPS, np64(table), at.cpu().numpy())
    close(dx, want, R.rows_tolerance(want, mag, dtype, 32), "broadcast gradients")
    close(dw, wsum, R.weight_tolerance(wmag, 64 + n * h // 64), "weight")


@pytest.mark.parametrize("n,hq,hk,d,dtype", [(5, 3, 1, 64, "f32"), (11, 1, 3, 32, "bf16"), (33, 2, 1, 24, "f16"),
                                             (70, 5, 1, 32, "f32"), (9, 1, 1, 128, "bf16")])
def test_norm_gradient_without_an_epsilon(n, hq, hk, d, dtype):
    # lanes and rows that hold nothing must not turn into 0 * infinity
    x, dy = randn(1, (n, hq + hk, d), dtype, 1.5), randn(2, (n, hq + hk, d), dtype)
    w = [1 + 0.3 * randn(3 + i, (d,), "f32") for i in (0, 1)]
    dx, dw = torch.empty_like(x), [torch.empty(d, device=DEV) for _ in range(2)]
    ws = torch.full((sdi.dlrm_qk_norm_rope_bwd_workspace_size(n, hq, hk, d),), 255, dtype=torch.uint8, device=DEV)
    sdi.dlrm_qk_norm_rope_bwd(dy[:, :hq], dy[:, hq:], x[:, :hq], x[:, hq:], w[0], w[1], 0.0, None, None, dx[:, :hq],
                              dx[:, hq:], dw[0], dw[1], ws)
    for i, part in enumerate((slice(0, hq), slice(hq, hq + hk))):
        want, mag, wsum, wmag = R.norm_rope_bwd(np64(dy[:, part]), np64(x[:, part]), np64(w[i]), 0.0, None, None)
        close(dx[:, part], want, R.rows_tolerance(want, mag, dtype, 32), "inputs")
        close(dw[i], wsum, R.weight_tolerance(wmag, 64 + n * max(hq, hk)), "weight")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_of_many_empty_sequences(dtype):
    # tokens whose sequences lie more than 32 apart, and several in one
    counts = [1] + [0] * 40 + [2] + [0] * 100 + [1, 1] + [0] * 7 + [3, 0]
    lengths = [c + 4 * (c > 0) for c in counts]
    table, table_d, offsets, lens, pages = make_batch(counts, lengths, 8)
    d, hk, n = 64, 2, sum(counts)
    kc, vc = (make_cache(s, pages, 8, hk, d, dtype, False) for s in (1, 2))
    k, v = randn(3, (n, hk, d), dtype), randn(4, (n, hk, d), dtype)
    f = flag()
    sdi.dlrm_kv_append(k, v, offsets, lens, table_d, kc, vc, err_flag=f)
    assert sdi.dlrm_read_error(f) == 0
    at = np.concatenate([np.arange(m - c, m) for c, m in zip(counts, lengths)])
    pg = table[np.repeat(np.arange(len(counts)), counts), at // 8]
    assert np.array_equal(np64(kc)[pg, at % 8], np64(k)) and np.array_equal(np64(vc)[pg, at % 8], np64(v))


@pytest.mark.parametrize("dtype,c", [("bf16", 1), ("f16", 40), ("f32", 2)])
def test_offsets_that_are_not_monotone_do_no_harm(dtype, c):
    # whatever the offsets say, only the batch's own rows and slots are touched
    case = ([c] * 4, [40] * 4, 4, 2, 64, 16, False, True, 0, dtype)
    table, table_d, offsets, lens, kc, vc, q = attention_inputs(case, stale=0.0)
    good_out, _ = attend(case, q, offsets, lens, table_d, kc, vc, 0.125)
    for bad in ([0, 3 * c, c, 2 * c, 4 * c], [4 * c, 3 * c, 2 * c, c, 0], [-5, c, 2 * c, 1 << 40, 4 * c], [1, 1, 1, 1, 1]):
        o, f = torch.tensor(bad, device=DEV), flag()
        out, _ = attend(case, q, o, lens, table_d, kc, vc, 0.125, f)
        kc2, vc2 = kc.clone(), vc.clone()
        sdi.dlrm_kv_append(q[:, :2], q[:, 2:], o, lens, table_d, kc2, vc2, err_flag=f)
        torch.cuda.synchronize()
        if bad != [1, 1, 1, 1, 1]:
            assert sdi.dlrm_read_error(f) == _native.ERR_BAD_OFFSETS
        live = torch.from_numpy(table[:, :3]).long().to(DEV).flatten()
        other = torch.ones(kc.shape[0], dtype=torch.bool, device=DEV)
        other[live] = False
        assert torch.equal(kc2[other], kc[other])


def test_norm_rope_of_no_tokens_and_zero_rows():
    x = torch.zeros(0, 2, 64, device=DEV)
    w, dw = torch.ones(64, device=DEV), torch.full((64,), 7.0, device=DEV)
    ws = torch.empty(max(1, sdi.dlrm_qk_norm_rope_bwd_workspace_size(0, 2, 0, 64)), dtype=torch.uint8, device=DEV)
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    sdi.dlrm_qk_norm_rope_fwd(x, None, w, None, EPS, rope_table(4, 64), none, x.clone(), None)
    sdi.dlrm_qk_norm_rope_bwd(x, None, x, None, w, None, EPS, rope_table(4, 64), none, x.clone(), None, dw, None, ws)
    assert not dw.any()
    z = torch.zeros(3, 2, 64, device=DEV, dtype=torch.bfloat16)
    out = torch.full_like(z, 7)
    sdi.dlrm_qk_norm_rope_fwd(z, None, w, None, EPS, None, None, out, None)
    assert not out.any()


# ---------------------------------------------------------------- the cache

def make_cache(seed, pages, page, hk, d, dtype, heads_first, fill=None):
    shape = (pages, hk, page, d) if heads_first else (pages, page, hk, d)
    t = randn(seed, shape, dtype) if fill is None else torch.full(shape, fill, dtype=DT[dtype], device=DEV)
    return t.transpose(1, 2) if heads_first else t


def make_batch(counts, lengths, page, spare=2, seed=0, width=0):
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + spare
    order = np.random.default_rng(seed).permutation(pages)[:sum(need)]
    table = np.full((len(counts), max(max(need), width, 1)), -1, np.int32)
    k = 0
    for s, m in enumerate(need):
        table[s, :m] = order[k:k + m]
        k += m
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return table, dev(table), dev(offsets), dev(np.asarray(lengths, np.int64)), pages


APPEND = [
    # counts, lengths, q heads, kv heads, d, rot, page, heads first, normed, interleaved, dtype
    ([1], [1], 1, 1, 64, 64, 16, False, True, False, "f16"),
    ([1, 1, 1, 1], [5, 16, 17, 300], 8, 2, 128, 128, 16, True, True, False, "bf16"),
    ([3, 0, 40, 1], [3, 9, 41, 100], 4, 4, 64, 32, 8, False, True, False, "bf16"),
    ([7, 2], [20, 2], 6, 3, 96, 96, 24, True, False, True, "f32"),
    ([5, 6], [5, 60], 2, 1, 17, 16, 7, False, True, False, "f32"),
    ([130], [513], 0, 2, 80, 40, 32, False, True, False, "f16"),
    ([2] * 70, list(range(2, 72)), 4, 2, 32, 32, 1, True, True, True, "bf16"),
    ([9], [90], 2, 2, 256, 128, 64, False, False, False, "bf16"),
]


@pytest.mark.parametrize("case", APPEND)
def test_append(case):
    counts, lengths, hq, hk, d, rot, page, first, normed, inter, dtype = case
    n = sum(counts)
    table, table_d, offsets, lens, pages = make_batch(counts, lengths, page)
    kc, vc = (make_cache(s, pages, page, hk, d, dtype, first) for s in (21, 22))
    kc0, vc0 = np64(kc), np64(vc)
    qkv = randn(23, (n, hq + 2 * hk, d), dtype, 1.5)  # heads of one projection
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    qw, kw = (1 + 0.3 * randn(s, (d,), "f32") for s in (3, 4))
    rope = rope_table(max(lengths), rot)
    qo = torch.full((n, hq, d), 7, dtype=DT[dtype], device=DEV) if hq else None
    f = flag()
    sdi.dlrm_kv_append(k, v, offsets, lens, table_d, kc, vc, k_weight=kw if normed else None, eps=EPS, rope=rope,
                       interleaved=inter, q=q if hq else None, q_weight=qw if normed and hq else None, q_out=qo,
                       err_flag=f)
    assert sdi.dlrm_read_error(f) == 0
    at = np.concatenate([np.arange(m - c, m) for c, m in zip(counts, lengths)])
    seq = np.repeat(np.arange(len(counts)), counts)
    if hq:
        y, mag = R.norm_rope(np64(q), np64(qw) if normed else None, EPS, np64(rope), at, inter)
        close(qo, y, R.rows_tolerance(y, mag, dtype), "queries")
    y, mag = R.norm_rope(np64(k), np64(kw) if normed else None, EPS, np64(rope), at, inter)
    pg, sl = table[seq, at // page], at % page
    close(np64(kc)[pg, sl], y, R.rows_tolerance(y, mag, dtype), "keys")
    kc0[pg, sl], vc0[pg, sl] = np64(kc)[pg, sl], np64(v)
    assert np.array_equal(np64(kc), kc0) and np.array_equal(np64(vc), vc0)  # nothing else written


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 20)])
def test_append_leaves_out_what_does_not_fit(dtype, d):
    page, hk = 8, 2
    counts, lengths = [2, 3, 2, 2, 1], [10, 2, 12, 40, 5]  # 1: more new than stored; 3: beyond the table
    n = sum(counts)
    table, table_d, offsets, lens, pages = make_batch(counts, [16, 16, 16, 16, 16], page)
    table_d[2, 1] = pages  # an invalid page under both of its new tokens
    kc, vc = (make_cache(s, pages, page, hk, d, dtype, False) for s in (21, 22))
    kc0, vc0 = kc.clone(), vc.clone()
    k, v, q = (randn(s, (n, hk, d), dtype) for s in (5, 6, 7))
    lens = torch.tensor(lengths, device=DEV)
    qo, f = torch.full_like(q, 7), flag()
    at = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, 8, 99], device=DEV)
    # given positions: the last token's is outside the table
    sdi.dlrm_kv_append(k, v, offsets, lens, table_d, kc, vc, rope=rope_table(20, 16), positions=at, q=q, q_out=qo,
                       err_flag=f)
    assert int(f.item()) == _native.FLAG_INDEX_OOB | _native.FLAG_BAD_OFFSETS
    pg = table[0, 1]
    want, mag = R.norm_rope(np64(k[:2]), None, 0, np64(rope_table(20, 16)), np.array([0, 1]))
    close(kc[pg, :2], want, R.rows_tolerance(want, mag, dtype), "the good sequence")
    kc0[pg, :2], vc0[pg, :2] = kc[pg, :2], v[:2]
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)
    assert (qo[2:5] == 7).all() and (qo[7:9] == 7).all()  # left out
    assert not qo[9].any() and (qo[5:7] != 7).any()


# ---------------------------------------------------------------- attention

ATTN = [
    # counts, lengths, q heads, kv heads, d, page, heads first, causal, window, dtype
    ([1], [1], 1, 1, 64, 16, False, True, 0, "f16"),
    ([1, 1, 1], [0, 1, 33], 8, 2, 64, 16, False, False, 0, "f16"),  # no history: empty rows
    ([1, 1, 1, 1, 1], [1, 15, 16, 17, 700], 4, 1, 128, 16, True, True, 0, "bf16"),
    ([1, 1], [3000, 5], 6, 2, 128, 64, True, True, 0, "bf16"),
    ([1], [5001], 8, 8, 64, 32, False, True, 0, "f16"),
    ([1, 1], [900, 2000], 32, 2, 128, 8, False, True, 0, "bf16"),  # 16 heads share one
    ([1, 1], [900, 2000], 40, 2, 64, 8, False, True, 0, "f16"),  # 20 heads share one
    ([1, 1, 1], [777, 64, 65], 3, 1, 80, 24, False, True, 100, "bf16"),
    ([2, 0, 4, 3], [40, 7, 4, 129], 4, 2, 96, 48, True, True, 0, "f16"),
    ([3, 5], [2, 3], 2, 1, 64, 16, False, True, 0, "bf16"),  # more new than stored: the first rows see nothing
    ([33, 70], [33, 200], 4, 4, 64, 16, False, True, 0, "f16"),
    ([130, 1, 129], [130, 300, 515], 2, 1, 128, 64, True, True, 0, "bf16"),
    ([64], [1000], 12, 4, 128, 16, False, False, 0, "bf16"),
    ([200, 17], [400, 0], 3, 1, 128, 128, True, False, 0, "f16"),
    ([150], [600], 4, 2, 64, 8, False, True, 37, "bf16"),
    ([90, 260], [90, 700], 2, 2, 128, 32, True, True, 200, "f16"),
    ([300], [300], 8, 1, 128, 256, False, True, 0, "bf16"),
    ([50], [9000], 2, 1, 128, 64, False, True, 0, "bf16"),  # few rows, long: split
    ([20], [9000], 4, 2, 64, 16, True, False, 1500, "f16"),
    ([40, 3], [77, 500], 4, 2, 32, 16, False, True, 0, "f16"),
    ([40, 3], [77, 500], 4, 2, 40, 1, False, True, 0, "bf16"),
    ([1, 9, 2], [50, 90, 333], 4, 2, 64, 32, False, True, 64, "f32"),
    ([1], [4000], 2, 1, 128, 16, True, True, 0, "f32"),
    ([1, 30], [100, 260], 2, 2, 17, 5, False, True, 0, "f32"),
    ([1, 30], [100, 260], 2, 2, 17, 5, False, True, 0, "bf16"),
    ([3, 20], [100, 200], 2, 1, 256, 16, False, True, 0, "bf16"),
    ([3, 20], [100, 200], 2, 1, 200, 16, True, False, 50, "f32"),
    ([5 + i % 30 for i in range(270)], [3 + 37 * i % 200 for i in range(270)], 4, 2, 64, 16, False, True, 0, "f16"),
    ([300], [5000], 2, 1, 64, 16, True, True, 0, "bf16"),
    ([200, 5], [333, 64], 2, 1, 128, 7, False, True, 0, "f16"),  # pages that end inside a tile, two query tiles
    ([140], [3001], 3, 1, 56, 3, False, False, 700, "bf16"),
    ([1] * 40, [(i * i * 7) % 3001 for i in range(40)], 8, 2, 64, 16, False, True, 0, "bf16"),
    ([i % 3 for i in range(300)], [(i * 61) % 1300 for i in range(300)], 2, 1, 64, 64, True, False, 0, "f16"),
    ([16, 3], [1500, 2000], 1, 1, 128, 24, False, True, 0, "bf16"),
    ([2, 1], [2500, 3], 2, 1, 20, 5, False, True, 0, "f32"),
    ([60, 1], [1100, 700], 3, 1, 64, 16, True, True, 0, "f32"),
    ([1, 1, 1], [5000, 0, 77], 8, 2, 256, 16, False, True, 0, "bf16"),
    ([3, 16], [900, 3300], 2, 2, 192, 24, True, False, 0, "f16"),
    ([30, 5], [400, 5], 3, 1, 160, 7, False, True, 100, "bf16"),
    ([5, 1], [700, 200], 4, 2, 136, 8, False, True, 0, "f16"),
    ([5], [700], 2, 1, 132, 8, False, True, 0, "f16"),
]


def attention_inputs(case, seed=0, stale=float("nan")):
    """Slots that nothing sees hold `stale`; page numbers past the histories are -1."""
    counts, lengths, hq, hk, d, page, first, causal, window, dtype = case
    table, table_d, offsets, lens, pages = make_batch(counts, lengths, page, seed=seed, width=2)
    kc, vc = (make_cache(31 + i + seed, pages, page, hk, d, dtype, first) for i in (0, 1))
    live = np.zeros((pages, page), bool)
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
            table_d[s, :lo // page] = -7
    dead = torch.from_numpy(~live).to(DEV)
    kc[dead], vc[dead] = stale, stale
    q = randn(41 + seed, (sum(counts), hq, d), dtype, 1.5)
    return table, table_d, offsets, lens, kc, vc, q


def attend(case, q, offsets, lens, table_d, kc, vc, scale, f=None, **kw):
    counts, lengths, hq, hk, d, page, first, causal, window, dtype = case
    n = sum(counts)
    out = torch.full((n, hq, d), 7, dtype=DT[dtype], device=DEV)
    lse = torch.full((n, hq), 7.0, device=DEV)
    sizes = (len(counts), n, hq, hk, d, max(counts), max(lengths))
    ws = torch.full((sdi.dlrm_kv_attn_workspace_size(*sizes),), 255, dtype=torch.uint8, device=DEV)  # NaNs
    sdi.dlrm_kv_attn_fwd(q, offsets, lens, table_d, kc, vc, out, scale, ws, max(counts), max(lengths), causal=causal,
                         window=window, lse=lse, err_flag=f, **kw)
    return out, lse


def check_attention(case, q, table, kc, vc, scale, out, lse, what="attention"):
    counts, lengths, hq, hk, d, page, first, causal, window, dtype = case
    k, v = (np.nan_to_num(np64(t), nan=0.0, posinf=0.0, neginf=0.0) for t in (kc, vc))
    want, wl, absout, smax, flat = R.attention(np64(q), counts, lengths, table, k, v, scale, causal, window)
    close(out, want, R.attention_tolerance(want, absout, smax, flat, d, dtype), (case, what))
    close(lse, wl, R.lse_tolerance(wl, smax, d), (case, what, "lse"))


@pytest.mark.parametrize("case", ATTN)
def test_attention(case):
    table, table_d, offsets, lens, kc, vc, q = attention_inputs(case)
    scale, f = 1 / case[4] ** 0.5, flag()
    out, lse = attend(case, q, offsets, lens, table_d, kc, vc, scale, f)
    assert sdi.dlrm_read_error(f) == 0
    check_attention(case, q, table, kc, vc, scale, out, lse)
    again = attend(case, q, offsets, lens, table_d, kc, vc, scale)  # the same bits again
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("case", [c for c in ATTN if sum(c[0]) <= 130][::3])
def test_attention_of_sharp_scores_and_strided_queries(case):
    # scores of a few hundred: the maximum moves by much from tile to tile
    counts, lengths, hq, hk, d, page, first, causal, window, dtype = case
    table, table_d, offsets, lens, kc, vc, q = attention_inputs(case, stale=float("inf"))
    wide = torch.full((sum(counts), hq + 3, d + 8), 9, dtype=DT[dtype], device=DEV)
    wide[:, 1:hq + 1, :d] = q
    scale = 8 / d ** 0.5
    out, lse = attend(case, wide[:, 1:hq + 1, :d], offsets, lens, table_d, kc, vc, scale)
    check_attention(case, q, table, kc, vc, scale, out, lse)


@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("case", [([1], [3000], 4, 1, 128, 16, False, True, 0, "bf16"),
                                  ([60], [900], 4, 2, 64, 16, True, False, 0, "f16")])
def test_attention_of_scores_that_rise_or_fall(case, rising):
    # every later tile beats the running maximum by much, or none does
    counts, lengths, hq, hk, d, page, first, causal, window, dtype = case
    table, table_d, offsets, lens, kc, vc, q = attention_inputs(case)
    q.zero_()
    q[..., 0] = 4
    at = np.arange(lengths[0])
    slope = torch.from_numpy(np.linspace(-20, 20, lengths[0]) * (1 if rising else -1)).to(DEV).to(DT[dtype])
    kc[torch.from_numpy(table[0, at // page]).long().to(DEV), torch.from_numpy(at % page).to(DEV), :, 0] = slope[:, None]
    out, lse = attend(case, q, offsets, lens, table_d, kc, vc, 1.0)
    check_attention(case, q, table, kc, vc, 1.0, out, lse)


@pytest.mark.parametrize("case", [([1, 1], [100, 40], 4, 2, 64, 16, False, True, 0, "f16"),
                                  ([60, 40], [100, 40], 4, 2, 128, 16, False, True, 0, "bf16"),
                                  ([2, 3], [100, 40], 4, 2, 64, 16, False, True, 0, "f32")])
def test_attention_invalid_page_reads_as_zeros(case):
    table, table_d, offsets, lens, kc, vc, q = attention_inputs(case)
    for bad in (-1, kc.shape[0], 0x7fffffff):
        table[0, 2] = table_d[0, 2] = bad
        f = flag()
        out, lse = attend(case, q, offsets, lens, table_d, kc, vc, 0.1, f)
        assert sdi.dlrm_read_error(f) == _native.ERR_INDEX_OOB
        check_attention(case, q, table, kc, vc, 0.1, out, lse)


@pytest.mark.parametrize("dtype,c", [("bf16", 1), ("f16", 40), ("f32", 2)])
def test_attention_leaves_out_bad_sequences(dtype, c):
    case = ([c] * 4, [300] * 4, 4, 2, 64, 16, False, True, 0, dtype)
    table, table_d, offsets, lens, kc, vc, q = attention_inputs(case)
    good_out, good_lse = attend(case, q, offsets, lens, table_d, kc, vc, 0.125)
    lens[1] = 301  # beyond max_len
    lens[2] = -1
    f = flag()
    out, lse = attend(case, q, offsets, lens, table_d, kc, vc, 0.125, f)
    assert sdi.dlrm_read_error(f) == _native.ERR_BAD_OFFSETS
    for s in range(4):
        rows = slice(s * c, (s + 1) * c)
        if s in (1, 2):
            assert (out[rows] == 7).all() and (lse[rows] == 7).all()
        else:
            assert torch.equal(out[rows], good_out[rows]) and torch.equal(lse[rows], good_lse[rows])
    lens[1:3] = 300
    offsets[3] += 1  # one sequence has more new tokens than max_new, the next fewer
    f = flag()
    out, _ = attend(case, q, offsets, lens, table_d, kc, vc, 0.125, f)
    assert sdi.dlrm_read_error(f) == _native.ERR_BAD_OFFSETS
    assert torch.equal(out[:2 * c], good_out[:2 * c]) and (out[2 * c:3 * c] == 7).all()


@pytest.mark.parametrize("dtype,c", [("bf16", 1), ("f16", 70), ("f32", 2)])
def test_attention_on_another_stream_and_in_a_graph(dtype, c):
    case = ([c, c], [2000, 333], 4, 2, 64, 16, False, True, 0, dtype)
    table, table_d, offsets, lens, kc, vc, q = attention_inputs(case)
    out, lse = attend(case, q, offsets, lens, table_d, kc, vc, 0.125)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = attend(case, q, offsets, lens, table_d, kc, vc, 0.125)
    side.synchronize()
    assert torch.equal(out, other[0]) and torch.equal(lse, other[1])
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    ws = torch.empty(sdi.dlrm_kv_attn_workspace_size(2, 2 * c, 4, 2, 64, c, 2000), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdi.dlrm_kv_attn_fwd(q, offsets, lens, table_d, kc, vc, o2, 0.125, ws, c, 2000, lse=l2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("dtype,c", [("bf16", 1), ("bf16", 40), ("f32", 1)])
def test_attention_and_append_past_32_bit_offsets(dtype, c):
    # pages a long way apart: element offsets beyond 2^32
    page, hk, d, pages, stride = 16, 2, 64, 4, 3 << 29
    cell = torch.zeros(2 * stride * pages, dtype=torch.bfloat16, device=DEV) if dtype == "bf16" else torch.zeros(
        2 * stride * pages, device=DEV)
    kc, vc = (cell[i * hk * page * d:].as_strided((pages, page, hk, d), (stride, hk * d, d, 1),
                                                  i * stride * pages) for i in (0, 1))
    case = ([c], [60], 4, 2, d, page, False, True, 0, dtype)
    table = np.array([[3, 0, 2, 1]], np.int32)
    table_d = torch.from_numpy(table).to(DEV)
    offsets, lens = torch.tensor([0, 60], device=DEV), torch.tensor([60], device=DEV)
    k, v = randn(1, (60, hk, d), dtype), randn(2, (60, hk, d), dtype)
    sdi.dlrm_kv_append(k, v, offsets, lens, table_d, kc, vc)
    at = torch.arange(60, device=DEV)
    pg = table_d[0].long()[at // page]
    assert torch.equal(kc[pg, at % page], k) and torch.equal(vc[pg, at % page], v)
    q, offsets = randn(3, (c, 4, d), dtype), torch.tensor([0, c], device=DEV)
    out, lse = attend(case, q, offsets, lens, table_d, kc, vc, 0.125)
    check_attention(case, q, table, kc, vc, 0.125, out, lse)


def test_norm_append_attend_together():
    """Histories appended in pieces and attended give what one full pass gives."""
    hq, hk, d, page, n = 4, 2, 64, 16, 90
    qkv = randn(50, (n, hq + 2 * hk, d), "f32")
    qw, kw, rope = 1 + 0.2 * randn(51, (d,), "f32"), 1 + 0.2 * randn(52, (d,), "f32"), rope_table(n, d)
    kc, vc = (make_cache(53, 8, page, hk, d, "f32", True, 0.0) for _ in range(2))
    table = np.array([[5, 1, 7, 0, 2, 3]], np.int32)
    table_d = torch.from_numpy(table).to(DEV)
    outs, done = [], 0
    for c in (40, 1, 1, 30, 18):
        part = qkv[done:done + c]
        done += c
        offsets, lens = torch.tensor([0, c], device=DEV), torch.tensor([done], device=DEV)
        q = torch.empty((c, hq, d), device=DEV)
        sdi.dlrm_kv_append(part[:, hq:hq + hk], part[:, hq + hk:], offsets, lens, table_d, kc, vc, k_weight=kw,
                           eps=EPS, rope=rope, q=part[:, :hq], q_weight=qw, q_out=q)
        case = ([c], [done], hq, hk, d, page, True, True, 0, "f32")
        outs.append(attend(case, q, offsets, lens, table_d, kc, vc, 0.125)[0])
    at = np.arange(n)
    qn, _ = R.norm_rope(np64(qkv[:, :hq]), np64(qw), EPS, np64(rope), at)
    kn, _ = R.norm_rope(np64(qkv[:, hq:hq + hk]), np64(kw), EPS, np64(rope), at)
    want, _, absout, smax, flat = R.attention(qn, [n], [n], np.arange(1)[None], kn[None], np64(qkv[None, :, hq + hk:]),
                                              0.125, True, 0)
    # the stored keys and the queries carry the row tolerance, which moves a score by 2 * 17 roundings more
    tol = R.attention_tolerance(want, absout, smax * (1 + 34 / (d + 4)), flat, d, "f32")
    close(torch.cat(outs), want, tol, "appended in pieces")
