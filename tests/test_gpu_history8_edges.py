"""The event history in 8 bits where a batch, a type or a wait meets its edge:
sharp and rising scores, powers that differ by much, pages that are none, NaN,
contradictions, waits that run out, streams and captured graphs; and a run of
all its calls together."""
import time

import numpy as np
import pytest
import torch

import sparse_dense_interaction_gb300 as sdi
from sparse_dense_interaction_gb300 import _native
from tests import _history8_ref as R8
from tests import _history_ref as R
from tests.test_gpu_history8 import (
    ATTN, DEV, DT, as64, attend, attention_inputs, bytes_of, cache8, check_attention, flag, np64, randn, table_of,
    tensors8)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_dense_interaction_gb300 import build
    build.build()


@pytest.fixture(autouse=True)
def _reset_hooks():
    yield
    sdi.dlrm_set_wait_test_hooks()


# one of each kernel and variant: (counts, lengths, q heads, kv heads, d, page, block, heads first, causal, window, dtype)
KINDS = [
    ([1, 1, 1], [300, 5, 90], 4, 2, 64, 16, 8, False, True, 0, "f16"), ([1, 1], [9000, 3], 4, 1, 128, 16, 16, True, True, 0, "bf16"),
    ([3, 1], [900, 4000], 4, 1, 128, 8, 8, True, True, 0, "bf16"), ([1, 4], [700, 5000], 4, 2, 256, 16, 4, True, True, 0, "f16"),
    ([2, 1], [700, 3000], 4, 2, 64, 32, 16, False, True, 100, "f32"), ([1], [3000], 4, 2, 128, 16, 1, True, True, 0, "f32"),
    ([40], [333], 4, 2, 64, 16, 16, True, True, 0, "f16"), ([150], [2000], 4, 2, 64, 16, 2, True, False, 0, "bf16"),
    ([9], [20000], 4, 1, 128, 64, 64, True, True, 0, "bf16"), ([300], [900], 3, 1, 128, 32, 8, False, True, 200, "f16"),
    ([200, 5], [333, 64], 2, 1, 128, 7, 7, False, True, 0, "f16"), ([300, 30], [400, 700], 4, 1, 128, 128, 32, True, True, 0, "bf16"),
    ([40, 3], [1000, 50], 4, 2, 256, 32, 8, True, True, 0, "bf16"), ([70], [900], 2, 2, 160, 12, 4, False, False, 0, "f16"),
    ([2, 30], [100, 260], 2, 2, 17, 5, 5, False, True, 0, "f32"), ([3], [700], 2, 1, 20, 5, 1, False, True, 0, "bf16"),
    # chunks for which the codes are converted once
    ([300, 5], [900, 700], 12, 2, 128, 32, 8, False, True, 0, "f16"), ([700, 1], [1500, 90], 8, 2, 64, 16, 16, True, True, 300, "f16"),
    ([260, 40], [400, 500], 12, 2, 96, 12, 3, False, True, 0, "bf16"), ([520], [600], 4, 1, 48, 64, 1, True, False, 0, "f16"),
]


@pytest.mark.parametrize("case", KINDS)
def test_sharp_scores_and_strided_queries(case):
    # scores of a hundred or so: the maximum moves by much from tile to tile
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, given, caches, q = attention_inputs(case, seed=7)
    wide = torch.full((sum(counts), hq + 3, d + 8), 9, dtype=DT[dtype], device=DEV)
    wide[:, 1:hq + 1, :d] = q
    out, lse = attend(case, given, caches, wide[:, 1:hq + 1, :d], 8 / d ** 0.5)
    check_attention(case, table, caches, q, 8 / d ** 0.5, out, lse)


@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("case", KINDS)
def test_powers_that_rise_or_fall_along_a_history(case, rising):
    # each page's values are larger, or smaller, than the one's before it: by 2^24 in all, and keys by 2^8
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, given, caches, q = attention_inputs(case, seed=3)
    for s, n in enumerate(lengths):
        own = -(-n // page)
        for i in range(own):
            share = (i if rising else own - 1 - i) / max(own - 1, 1)
            caches[0][1][table[s, i]] = 114 + int(8 * share)
            caches[1][1][table[s, i]] = 104 + int(24 * share)
    out, lse = attend(case, given, caches, q, 1 / d ** 0.5)
    check_attention(case, table, caches, q, 1 / d ** 0.5, out, lse)


@pytest.mark.parametrize("case", KINDS)
def test_blocks_of_zeros_count_for_the_weights(case):
    # every other page's values are zeros (exponent 0), its keys too in some: their weights count all the same
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, given, caches, q = attention_inputs(case, seed=4)
    pages = np.arange(caches[0][0].shape[0])
    for i, every in ((0, 3), (1, 2)):
        codes, exps = caches[i]
        codes[pages % every == 0] = 0
        exps[pages % every == 0] = 0
    out, lse = attend(case, given, caches, q, 1 / d ** 0.5)
    check_attention(case, table, caches, q, 1 / d ** 0.5, out, lse)


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** 60])
@pytest.mark.parametrize("case", [c for c in KINDS if c[-1] != "f16"])
def test_queries_far_from_one(case, size):
    # bf16 and fp32 rows of any size: the scale takes it back
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, given, caches, q = attention_inputs(case, seed=5)
    q = (q.double() * size).to(DT[dtype])
    q[0] = 0
    scale = 1 / d ** 0.5 / size
    scale = min(scale, 2e38)
    out, lse = attend(case, given, caches, q, scale)
    check_attention(case, table, caches, q, scale, out, lse)


@pytest.mark.parametrize("case", KINDS)
def test_a_page_that_is_none_reads_as_zeros(case):
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, given, caches, q = attention_inputs(case)
    at = (lengths[0] - 1) // page  # seen whatever the window
    for bad in (-1, caches[0][0].shape[0], 0x7FFFFFFF):
        table[0, at] = given[0, at] = bad
        f = flag()
        out, lse = attend(case, given, caches, q, 0.1, f)
        assert sdi.dlrm_read_error(f) == _native.ERR_INDEX_OOB
        check_attention(case, table, caches, q, 0.1, out, lse)


@pytest.mark.parametrize("case", KINDS)
def test_a_query_of_nan_gives_nan(case):
    hq = case[2]
    table, given, caches, q = attention_inputs(case)
    out, lse = attend(case, given, caches, q, 0.125)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    bad[0, 1] = bad[-1, hq - 1] = True
    q[bad, 5] = float("nan")
    got, got_lse = attend(case, given, caches, q, 0.125)
    assert got[bad].isnan().all() and got_lse[bad].isnan().all()
    assert torch.equal(got[~bad], out[~bad]) and torch.equal(got_lse[~bad], lse[~bad])


@pytest.mark.parametrize("what", ["negative", "beyond its table", "first token", "last token"])
@pytest.mark.parametrize("case", [
    ([2, 0, 2], [60, 40, 50], 4, 2, 64, 16, 16, False, True, 0, "bf16"), ([2, 0, 2], [9000, 40, 50], 4, 2, 64, 16, 8, True, True, 0, "f16"),
    ([2, 0, 2], [60, 40, 50], 4, 2, 64, 16, 4, False, True, 0, "f32"), ([40, 0, 40], [60, 40, 50], 4, 2, 64, 16, 16, False, True, 0, "f16"),
    ([300, 0, 40], [600, 40, 50], 4, 1, 128, 16, 16, True, True, 0, "bf16"), ([2, 0, 2], [60, 40, 50], 4, 2, 20, 7, 7, False, True, 0, "bf16"),
])
def test_contradictions_are_flagged(case, what):
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, given, caches, q = attention_inputs(case)
    n, S = sum(counts), len(counts)
    good, _ = attend(case, given, caches, q, 0.125)
    offsets, lens = [0] + list(np.cumsum(counts)), list(lengths)
    same, left_out = slice(0, n), slice(0, 0)
    if what == "negative":
        lens[1] = -1
    elif what == "beyond its table":
        lens[1] = given.shape[1] * page + 1
    elif what == "first token":
        offsets[0], same, left_out = 1, slice(counts[0], n), slice(0, 1)
    else:
        offsets[S], same, left_out = n - 1, slice(0, counts[0]), slice(n - 1, n)
    sizes = (S, n, hq, hk, d, max(counts), given.shape[1] * page + 9)
    ws = torch.full((sdi.dlrm_kv8_attn_workspace_size(*sizes),), 255, dtype=torch.uint8, device=DEV)
    out, f = torch.full_like(q, 7), flag()
    (kc, ke), (vc, ve) = (tensors8(*c, first) for c in caches)
    sdi.dlrm_kv8_attn_fwd(q, as64(offsets), as64(lens), torch.from_numpy(given).to(DEV), kc, vc, ke, ve, out, 0.125, ws,
                          max(counts), sizes[-1], causal=causal, window=window, err_flag=f)
    assert sdi.dlrm_read_error(f) == _native.ERR_BAD_OFFSETS
    # another max_len may share the positions out otherwise: the last bits are free
    assert (out[same].float() - good[same].float()).abs().max() <= 2 * R.U[dtype] * good[same].float().abs().max() + 1e-5
    assert (out[left_out] == 7).all()


@pytest.mark.parametrize("polls", [0, 1, 40])
@pytest.mark.parametrize("case", KINDS[:14])
def test_waits_that_run_out(case, polls):
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, given, caches, q = attention_inputs(case)
    n, guard = sum(counts), 4096
    size = sdi.dlrm_kv8_attn_workspace_size(len(counts), n, hq, hk, d, max(counts), max(lengths))
    bufs = [torch.full((2 * guard + m,), fill, dtype=t, device=DEV)
            for m, fill, t in ((n * hq * d, 7, DT[dtype]), (n * hq, 7, torch.float32), (size, 0xA5, torch.uint8))]
    out, lse, ws = (b[guard:b.numel() - guard] for b in bufs)
    out, lse = out.view(n, hq, d), lse.view(n, hq)
    (kc, ke), (vc, ve) = (tensors8(*c, first) for c in caches)
    offsets, lens, pages = as64([0] + list(np.cumsum(counts))), as64(lengths), torch.from_numpy(given).to(DEV)

    def call(f):
        sdi.dlrm_kv8_attn_fwd(q, offsets, lens, pages, kc, vc, ke, ve, out, d ** -0.5, ws, max(counts), max(lengths),
                              causal=causal, window=window, lse=lse, err_flag=f)
        return sdi.dlrm_read_error(f)

    assert call(flag()) == 0
    want = out.clone(), lse.clone()
    sdi.dlrm_set_wait_test_hooks(copy_wait_polls=polls)
    start = time.perf_counter()
    status = call(flag())
    took = time.perf_counter() - start
    sdi.dlrm_set_wait_test_hooks()
    assert took < 2, f"{took:.3f} s"
    assert status in (0, _native.ERR_WAIT_TIMEOUT)
    if polls == 0:
        assert status == _native.ERR_WAIT_TIMEOUT
    if status == 0:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for buf, fill in zip(bufs, (7, 7, 0xA5)):
        assert (buf[:guard] == fill).all() and (buf[buf.numel() - guard:] == fill).all()
    assert call(flag()) == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("case", KINDS[:2] + KINDS[6:7] + KINDS[11:])
def test_views_of_larger_caches(case):
    # codes whose rows, slots and pages lie apart, exponents of heads in another order: same values, same bits
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, given, caches, q = attention_inputs(case)
    want, want_lse = attend(case, given, caches, q, 0.125)
    views = []
    for codes, exps in caches:
        big = torch.full((codes.shape[0], page + 3, hk + 1, (d + 31) // 16 * 16), 0x7F, dtype=torch.uint8, device=DEV)
        big[:, :page, :hk, :d] = torch.from_numpy(codes).to(DEV)
        e = torch.full((hk + 2, exps.shape[1], codes.shape[0]), 255, dtype=torch.uint8, device=DEV).permute(2, 1, 0)
        e[:, :, 1:hk + 1] = torch.from_numpy(exps).to(DEV)
        views.append((big[:, :page, :hk, :d], e[:, :, 1:hk + 1]))
    n = sum(counts)
    sizes = (len(counts), n, hq, hk, d, max(counts), max(lengths))
    ws = torch.full((sdi.dlrm_kv8_attn_workspace_size(*sizes),), 255, dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(n, hq, device=DEV)
    (kc, ke), (vc, ve) = views
    sdi.dlrm_kv8_attn_fwd(q, as64([0] + list(np.cumsum(counts))), as64(lengths), torch.from_numpy(given).to(DEV), kc, vc,
                          ke, ve, out, 0.125, ws, max(counts), max(lengths), causal=causal, window=window, lse=lse)
    # an aligned view may take another kernel than an odd one: the last bits are free
    close = lambda a, b, u: (a.double() - b.double()).abs() <= u * b.double().abs() + 1e-5
    assert close(out, want, 2 * R.U[dtype]).all() and (close(lse, want_lse, 1e-5) | (lse == want_lse)).all()
    if d % 16 == 0:
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_offsets_past_32_bits():
    # pages 2^32 codes apart: the last one's slots lie behind 4 GB
    page, hk, d, hq = 16, 1, 64, 4
    stride = (1 << 31) + 4096
    store = torch.zeros(2 * stride + page * d, dtype=torch.uint8, device=DEV)
    exps = torch.zeros((3, 1, hk), dtype=torch.uint8, device=DEV)
    view = store.as_strided((3, page, hk, d), (stride, d, d, 1))
    v_store = store.clone()
    v_view, v_exps = v_store.as_strided((3, page, hk, d), (stride, d, d, 1)), exps.clone()
    k, v = randn(1, (20, hk, d), "bf16"), randn(2, (20, hk, d), "bf16")
    table = torch.tensor([[2, 1]], dtype=torch.int32, device=DEV)
    sdi.dlrm_kv8_append(k, v, as64([0, 20]), as64([20]), table, view, v_view, exps, v_exps)
    codes, e = np.zeros((3, page, hk, d), np.uint8), np.zeros((3, 1, hk), np.uint8)
    R8.append(np64(k), codes, e, [20], [20], np.array([[2, 1]]), page)
    assert np.array_equal(view.cpu().numpy(), codes) and np.array_equal(exps.cpu().numpy(), e)
    q = randn(3, (1, hq, d), "bf16", 0.5)
    ws = torch.empty(sdi.dlrm_kv8_attn_workspace_size(1, 1, hq, hk, d, 1, 20), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    sdi.dlrm_kv8_attn_fwd(q, as64([0, 1]), as64([20]), table, view, v_view, exps, v_exps, out, 0.125, ws, 1, 20)
    small = [t.clone() for t in (view, v_view)]
    want = torch.empty_like(q)
    sdi.dlrm_kv8_attn_fwd(q, as64([0, 1]), as64([20]), table, small[0].contiguous(), small[1].contiguous(), exps, v_exps,
                          want, 0.125, ws, 1, 20)
    assert torch.equal(out, want)


# ---------------------------------------------------------------- the calls together

class Store:
    """Users' histories in 8 bits, kept by the calls alone."""

    def __init__(self, users, pages, page, block, hk, d, width):
        self.page, self.hk, self.d = page, hk, d
        self.codes = [torch.zeros((pages, page, hk, d), dtype=torch.uint8, device=DEV) for _ in range(2)]
        self.exps = [torch.zeros((pages, page // block, hk), dtype=torch.uint8, device=DEV) for _ in range(2)]
        self.table = torch.full((users, width), -1, dtype=torch.int32, device=DEV)
        self.ring = torch.arange(pages, dtype=torch.int32, device=DEV).flip(0).contiguous()
        self.state = as64([0, pages])
        self.lengths, self.offsets = as64([0] * users), as64([0] * (users + 1))
        self.err = flag()

    def step(self, counts, q, k, v, q_weight, k_weight, rope, positions, out, ws, max_new, max_len):
        """Reserves, norms and turns, appends, attends: new events see those up to themselves."""
        sdi.dlrm_kv_reserve(counts, self.lengths, self.table, self.page, self.ring, self.state, self.state, self.offsets,
                            self.lengths, positions=positions, err_flag=self.err)
        sdi.dlrm_qk_norm_rope_fwd(q, k, q_weight, k_weight, 1e-6, rope, positions, q, k, err_flag=self.err)
        batch = self.offsets, self.lengths, self.table, *self.codes, *self.exps
        sdi.dlrm_kv8_append(k, v, *batch, err_flag=self.err)
        sdi.dlrm_kv8_attn_fwd(q, *batch, out, self.d ** -0.5, ws, max_new, max_len, err_flag=self.err)


def rope_table(length, rot):
    a = torch.arange(length, dtype=torch.float64)[:, None] * 1000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([a.cos(), a.sin()], 1).float().to(DEV)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_steps_of_a_server(dtype):
    """Prompts, then events one at a time, users who leave and their pages given to others; every step's attention
    against the formula over the codes that the cache holds."""
    users, page, block, hq, hk, d = 5, 16, 8, 4, 2, 64
    store = Store(users, 40, page, block, hk, d, 12)
    w = [1 + 0.2 * randn(s, (d,), "f32") for s in (1, 2)]
    rope = rope_table(200, d)
    want_lengths = [0] * users
    seed = 10
    for counts in ([40, 3, 0, 17, 100], [1] * 5, [1, 0, 30, 1, 0], [-1, 1, 1, 1, -1], [60, 1, 0, 1, 20], [1] * 5):
        new = [max(c, 0) for c in counts]
        n, seed = sum(new), seed + 10
        want_lengths = [0 if c < 0 else length + c for c, length in zip(counts, want_lengths)]
        q, k, v = (randn(seed + i, (n, h, d), dtype, 1.5) for i, h in enumerate((hq, hk, hk)))
        q0, k0, v0 = np64(q), np64(k), np64(v)
        out, positions = torch.empty_like(q), as64([0] * n)
        size = sdi.dlrm_kv8_attn_workspace_size(users, n, hq, hk, d, max(new), 200)
        store.step(as64(counts), q, k, v, *w, rope, positions, out, torch.empty(size, dtype=torch.uint8, device=DEV),
                   max(new), 192)
        assert sdi.dlrm_read_error(store.err) == 0
        assert store.lengths.tolist() == want_lengths
        at = np.concatenate([np.arange(length - c, length) for c, length in zip(new, want_lengths)])
        assert positions.tolist() == at.tolist()
        # what is stored lies within a code's rounding of the formula's keys, and within two where it was rounded again
        table = store.table.cpu().numpy()
        used = [int(table[s, i]) for s, length in enumerate(want_lengths) for i in range(-(-length // page))]
        assert len(set(used)) == len(used) and min(used) >= 0
        codes = [(bytes_of(c), e.cpu().numpy()) for c, e in zip(store.codes, store.exps)]
        keys, mag = R.norm_rope(k0, np64(w[1]), 1e-6, np64(rope), at)
        first = 0
        for s, c in enumerate(new):
            p = np.arange(want_lengths[s] - c, want_lengths[s])
            for x, (held, exps) in ((keys[first:first + c], codes[0]), (v0[first:first + c], codes[1])):
                got = R8.values(held, exps)[table[s, p // page], p % page]
                power = R8.power(exps.repeat(block, 1)[table[s, p // page], p % page])[..., None]
                assert (np.abs(got - x) <= 2.0 ** -4 * np.abs(x) * 1.01 + 2.0 ** -10 * power + R.U[dtype] * 2 * np.abs(x)
                        + 1e-5).all()
            first += c
        values = [R8.values(*c) for c in codes]
        want, _, absout, smax, flat = R.attention(np64(q), new, want_lengths, table, *values, d ** -0.5, True, 0)
        tol = R.attention_tolerance(want, absout, smax, flat, d, dtype) + 2.0 ** -36 * np.abs(values[1]).max() * 200
        assert (np.abs(np64(out) - want) <= tol).all()
    free = [int(store.ring[i % 40]) for i in range(*store.state.tolist())]
    assert sorted(free + used) == list(range(40))


def test_steps_captured_in_graphs_and_on_other_streams():
    """A step captured once and replayed for every event gives the bits of the same steps launched one by one."""
    users, page, hq, hk, d = 6, 8, 4, 2, 64
    w = [1 + 0.2 * randn(s, (d,), "f32") for s in (1, 2)]
    rope = rope_table(300, d)
    rows = [[randn(100 * t + i, (users, h, d), "bf16", 1.5) for i, h in enumerate((hq, hk, hk))] for t in range(30)]
    size = sdi.dlrm_kv8_attn_workspace_size(users, users, hq, hk, d, 1, 300)
    results = []
    for captured in (False, True):
        store = Store(users, 40, page, page, hk, d, 40)
        counts, positions = as64([1] * users), as64([0] * users)
        q, k, v = (torch.empty_like(x) for x in rows[0])
        out, ws = torch.empty_like(q), torch.empty(size, dtype=torch.uint8, device=DEV)
        step = lambda: store.step(counts, q, k, v, *w, rope, positions, out, ws, 1, 300)
        outs = []
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph = None
            for t in range(30):
                for to, x in zip((q, k, v), rows[t]):
                    to.copy_(x)
                if captured and graph is None:
                    graph = torch.cuda.CUDAGraph()
                    graph.capture_begin()
                    step()
                    graph.capture_end()
                graph.replay() if captured else step()
                outs.append(out.clone())
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert sdi.dlrm_read_error(store.err) == 0
        results.append((outs, *store.codes, *store.exps, store.lengths, store.table, store.state))
    for a, b in zip(results[0][0], results[1][0]):
        assert torch.equal(a, b)
    for a, b in zip(results[0][1:], results[1][1:]):
        assert torch.equal(a, b)


def test_reserve_without_rows_tries_again_and_refuses_a_bad_state():
    page, S = 8, 3
    lengths, counts = as64([5, 8, 0]), as64([4, 9, 1])
    table = torch.tensor([[0, -1, -1], [1, -1, -1], [-1, -1, -1]], dtype=torch.int32, device=DEV)
    ring = torch.tensor([2, 3, 4, -1, -1, -1], dtype=torch.int32, device=DEV)
    state, offsets, new = as64([0, 2]), as64([0] * 4), as64([0] * 3)
    call = lambda st, to, **kw: sdi.dlrm_kv_reserve(counts, lengths, table, page, ring, st, to, offsets, lengths, err_flag=f, **kw)
    f = flag()
    call(state, state, n=14)  # 1 + 2 + 1 pages are wanted, there are 2: the second gets none, nor does the third
    assert sdi.dlrm_read_error(f) == _native.ERR_CAPACITY
    assert lengths.tolist() == [9, ~8, ~0] and offsets.tolist() == [0, 4, 13, 14] and state.tolist() == [1, 2]
    assert table.tolist() == [[0, 2, -1], [1, -1, -1], [-1, -1, -1]]
    state[1], f = 4, flag()  # more pages: the next call tries again
    ring[3] = 5
    counts[0] = 0
    call(state, state, n=10)
    assert sdi.dlrm_read_error(f) == 0
    assert lengths.tolist() == [9, 17, 1] and state.tolist() == [4, 4]
    assert table.tolist() == [[0, 2, -1], [1, 3, 4], [5, -1, -1]]
    for bad in ([3, 2], [-1, 2], [0, 7]):
        before, f = (lengths.clone(), table.clone(), ring.clone()), flag()
        st, to = as64(bad), as64([9, 9])
        counts.copy_(as64([-1, 1, 8]))
        sdi.dlrm_kv_reserve(counts, lengths, table, page, ring, st, to, offsets, new, n=9, err_flag=f)
        assert sdi.dlrm_read_error(f) in (_native.ERR_BAD_OFFSETS, _native.ERR_CAPACITY)
        assert new.tolist() == [0, 18, ~1] and to.tolist() == bad  # 18 fits its pages, 1 + 8 does not
        assert torch.equal(table, before[1]) and torch.equal(ring, before[2])


def test_reserve_tokens_beyond_n_and_tables():
    page = 4
    table = torch.full((4, 2), -1, dtype=torch.int32, device=DEV)
    ring, offsets, new, to = torch.arange(9, dtype=torch.int32, device=DEV), as64([0] * 5), as64([0] * 4), as64([0, 0])
    slots = torch.full((6,), -9, dtype=torch.int64, device=DEV)
    f = flag()
    sdi.dlrm_kv_reserve(as64([3, 9, 2, 4]), as64([0, 0, 0, 0]), table, page, ring, as64([0, 9]), to, offsets, new,
                        slots=slots, err_flag=f)
    assert sdi.dlrm_read_error(f) == _native.ERR_BAD_OFFSETS  # 9 do not fit a row; the rest goes beyond 6 rows
    assert new.tolist() == [3, ~0, ~0, ~0] and offsets.tolist() == [0, 3, 12, 14, 18] and to.tolist() == [1, 9]
    assert slots.tolist() == [0, 1, 2, -1, -1, -1]


@pytest.mark.parametrize("page", [8, 16, 24, 40, 64, 128, 192])
@pytest.mark.parametrize("d,dtype", [(64, "f16"), (48, "bf16"), (64, "f32")])
def test_narrow_heads_on_pages_of_every_kind(page, d, dtype):
    """Pages shorter and longer than what a warp reads at a time, none of them dividing the other."""
    counts, lengths = [1, 2, 0, 1, 2, 1], [1, 63, 40, 64, 130, 1777]
    for window in (0, 70):
        case = (counts, lengths, 6, 2, d, page, 8, False, True, window, dtype)
        table, given, caches, q = attention_inputs(case, seed=page + window)
        out, lse = attend(case, given, caches, q, 1 / d ** 0.5)
        check_attention(case, table, caches, q, 1 / d ** 0.5, out, lse)


@pytest.mark.parametrize("case", KINDS)
def test_long_runs_of_zeros(case):
    """Runs longer than any tile whose values, or keys, are zeros: their weights count, wherever they come."""
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, given, caches, q = attention_inputs(case, seed=9)
    for s, n in enumerate(lengths):
        for i in range(-(-n // page)):
            for kind, run in ((0, 300), (1, 280)):
                if i * page // run % 2 == 0:
                    caches[kind][0][table[s, i]] = 0
                    caches[kind][1][table[s, i]] = 0
    out, lse = attend(case, given, caches, q, 1 / d ** 0.5)
    check_attention(case, table, caches, q, 1 / d ** 0.5, out, lse)
