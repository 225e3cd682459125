"""Long chunks, whose codes are converted once, beside single events and short
chunks in one batch of the event history in 8 bits."""
import numpy as np
import pytest
import torch

import sparse_dense_interaction_gb300 as sdi
from sparse_dense_interaction_gb300 import _native
from tests import _history_ref as R
from tests.test_gpu_history8 import DEV, as64, attend, attention_inputs, check_attention, flag, tensors8
from tests.test_gpu_history8_edges import _built, _reset_hooks  # noqa: F401

pytestmark = pytest.mark.gpu

# (counts, lengths, q heads, kv heads, d, page, block, heads first, causal, window, dtype)
MIXED = [
    # a prompt and single events, users without new ones, one without a history
    ([1, 390, 1, 0, 1, 1], [700, 400, 1, 33, 2500, 0], 8, 2, 128, 64, 16, True, True, 0, "bf16"),
    ([1, 390, 1, 0, 1, 4], [700, 400, 1, 33, 2500, 2], 8, 2, 128, 16, 8, False, True, 0, "f16"),
    # around 16 rows of a cache head
    ([4, 5, 384, 3, 17, 1], [900, 5, 390, 70, 17, 4000], 8, 2, 96, 32, 8, True, True, 0, "bf16"),
    ([16, 17, 2048, 15, 0], [300, 40, 2048, 15, 9], 1, 1, 64, 16, 16, False, True, 0, "bf16"),
    ([1, 520, 2, 40], [90, 600, 0, 333], 4, 1, 64, 64, 4, True, False, 0, "f16"),
    # a window, long histories that are shared out over CTAs
    ([1, 1, 400, 2], [9000, 5000, 900, 7000], 8, 2, 128, 128, 16, True, True, 700, "bf16"),
    ([1, 1, 400, 1], [40000, 30, 900, 77], 4, 1, 128, 16, 16, False, True, 0, "f16"),
    # 20 rows for one event; pages that rows of 16 do not take; many sequences
    ([1, 110, 2], [50, 200, 90], 20, 1, 128, 16, 16, False, True, 0, "bf16"),
    ([1, 390, 2, 1], [50, 400, 90, 640], 8, 2, 128, 7, 7, False, True, 0, "bf16"),
    ([i % 3 for i in range(300)] + [600], [(i * 61) % 900 for i in range(300)] + [700], 4, 1, 64, 32, 32, False, True, 0,
     "bf16"),
]


@pytest.mark.parametrize("case", MIXED)
def test_mixed_batches(case):
    table, given, caches, q = attention_inputs(case, seed=31)
    scale, f = 1 / case[4] ** 0.5, flag()
    out, lse = attend(case, given, caches, q, scale, f)
    assert sdi.dlrm_read_error(f) == 0
    check_attention(case, table, caches, q, scale, out, lse)
    again = attend(case, given, caches, q, scale)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_a_batch_without_any_long_chunk():
    # max_new is a bound: no sequence has as many
    case = ([1, 3, 20, 0, 100], [900, 3, 40, 7, 333], 8, 2, 128, 16, 16, False, True, 0, "bf16")
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, given, caches, q = attention_inputs(case, seed=32)
    wide = torch.zeros((2000, hq, d), dtype=q.dtype, device=DEV)  # n is one, too: rows that nobody owns
    wide[:q.shape[0]] = q
    out, f = torch.full_like(wide, 7), flag()
    sizes = (len(counts), 2000, hq, hk, d, 1500, 2000)
    ws = torch.full((sdi.dlrm_kv8_attn_workspace_size(*sizes),), 255, dtype=torch.uint8, device=DEV)
    lse = torch.full((2000, hq), 7.0, device=DEV)
    (kc, ke), (vc, ve) = (tensors8(*c, first) for c in caches)
    sdi.dlrm_kv8_attn_fwd(wide, as64([0] + list(np.cumsum(counts))), as64(lengths), torch.from_numpy(given).to(DEV), kc, vc,
                          ke, ve, out, d ** -0.5, ws, 1500, 2000, lse=lse, err_flag=f)
    assert sdi.dlrm_read_error(f) == _native.ERR_BAD_OFFSETS  # offsets[S] is not n
    n = sum(counts)
    check_attention(case, table, caches, q, d ** -0.5, out[:n], lse[:n])
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()


@pytest.mark.parametrize("what", ["negative", "beyond its table", "more than max_new", "a page that is none"])
def test_contradictions_in_mixed_batches(what):
    case = MIXED[0]
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    for bad in (0, 1):  # a single event; the long chunk
        table, given, caches, q = attention_inputs(case, seed=33)
        good, _ = attend(case, given, caches, q, 0.125)
        n, lens, max_new = sum(counts), list(lengths), max(counts)
        if what == "negative":
            lens[bad] = -1
        elif what == "beyond its table":
            lens[bad] = given.shape[1] * page + 1
        elif what == "more than max_new" and bad == 1:
            max_new -= 1
        else:
            given[bad, 0] = 0x7FFFFFFF
        wrong = _native.ERR_INDEX_OOB if given[bad, 0] == 0x7FFFFFFF else _native.ERR_BAD_OFFSETS
        sizes = (len(counts), n, hq, hk, d, max_new, given.shape[1] * page + 9)
        ws = torch.full((sdi.dlrm_kv8_attn_workspace_size(*sizes),), 255, dtype=torch.uint8, device=DEV)
        out, f = torch.full_like(q, 7), flag()
        (kc, ke), (vc, ve) = (tensors8(*c, first) for c in caches)
        offsets = [0] + list(np.cumsum(counts))
        sdi.dlrm_kv8_attn_fwd(q, as64(offsets), as64(lens), torch.from_numpy(given).to(DEV), kc, vc, ke, ve, out, 0.125, ws,
                              max_new, sizes[-1], causal=causal, window=window, err_flag=f)
        assert sdi.dlrm_read_error(f) == wrong
        own = torch.zeros(n, dtype=torch.bool, device=DEV)
        own[offsets[bad]:offsets[bad + 1]] = True
        same = (out[~own].float() - good[~own].float()).abs().max()
        assert same <= 2 * R.U[dtype] * good[~own].float().abs().max() + 1e-5
        assert wrong == _native.ERR_INDEX_OOB or (out[own] == 7).all()


@pytest.mark.parametrize("polls", [0, 1, 40])
@pytest.mark.parametrize("case", MIXED[:6])
def test_waits_that_run_out_in_mixed_batches(case, polls):
    table, given, caches, q = attention_inputs(case, seed=34)
    want = attend(case, given, caches, q, 0.125)
    sdi.dlrm_set_wait_test_hooks(copy_wait_polls=polls)
    f = flag()
    got = attend(case, given, caches, q, 0.125, f)
    status = sdi.dlrm_read_error(f)
    sdi.dlrm_set_wait_test_hooks()
    assert status in (0, _native.ERR_WAIT_TIMEOUT)
    assert polls > 0 or status == _native.ERR_WAIT_TIMEOUT
    again = attend(case, given, caches, q, 0.125)
    for a, b, c in zip(want, again, got):
        assert torch.equal(a, b) and (status != 0 or torch.equal(a, c))
