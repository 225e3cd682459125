"""Paths of the attention in 8 bits that sizes alone choose: tiles over the codes
with many rows, where a copy of them would be too large; waits of chunks whose
codes are converted; codes beyond 4 GB for every number of rows."""
import time

import numpy as np
import pytest
import torch

import sparse_dense_interaction_gb300 as sdi
from sparse_dense_interaction_gb300 import _native
from tests.test_gpu_history8 import (
    DEV, DT, as64, attend, attention_inputs, check_attention, flag, randn, tensors8)
from tests.test_gpu_history8_edges import KINDS, _built, _reset_hooks  # noqa: F401
from tests.test_gpu_history8_mixed import MIXED

pytestmark = pytest.mark.gpu

CONVERTED = KINDS[16:] + MIXED[:5]


@pytest.mark.parametrize("max_len", [1 << 21, 1 << 24])
@pytest.mark.parametrize("case", CONVERTED + [([2048], [2100], 1, 1, 64, 16, 16, False, True, 0, "bf16")])
def test_many_rows_in_tiles_over_the_codes(case, max_len):
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, given, caches, q = attention_inputs(case, seed=51)
    n = sum(counts)
    sizes = (len(counts), n, hq, hk, d, max(counts), max_len)
    # a copy of up to 2 GiB is made; beyond, no room for one is asked for
    copied = 4 * len(counts) * hk * d * max_len <= 1 << 31
    assert (sdi.dlrm_kv8_attn_workspace_size(*sizes) > sdi.dlrm_kv_attn_workspace_size(*sizes)) == copied
    ws = torch.full((sdi.dlrm_kv8_attn_workspace_size(*sizes),), 255, dtype=torch.uint8, device=DEV)
    out, lse, f = torch.full_like(q, 7), torch.full((n, hq), 7.0, device=DEV), flag()
    (kc, ke), (vc, ve) = (tensors8(*c, first) for c in caches)
    sdi.dlrm_kv8_attn_fwd(q, as64([0] + list(np.cumsum(counts))), as64(lengths), torch.from_numpy(given).to(DEV), kc, vc,
                          ke, ve, out, d ** -0.5, ws, max(counts), max_len, causal=causal, window=window, lse=lse, err_flag=f)
    assert sdi.dlrm_read_error(f) == 0
    check_attention(case, table, caches, q, d ** -0.5, out, lse)


@pytest.mark.parametrize("polls", [0, 1, 40])
@pytest.mark.parametrize("case", KINDS[14:])
def test_waits_that_run_out_after_a_conversion(case, polls):
    # (the general kernel, first two, waits for nothing)
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, given, caches, q = attention_inputs(case, seed=52)
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
    if polls == 0 and d % 8 == 0:
        assert status == _native.ERR_WAIT_TIMEOUT
    if status == 0:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for buf, fill in zip(bufs, (7, 7, 0xA5)):
        assert (buf[:guard] == fill).all() and (buf[buf.numel() - guard:] == fill).all()
    assert call(flag()) == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_codes_past_4_gb_for_every_number_of_rows(dtype):
    # pages 2^31 codes apart, so the last one's lie behind 4 GB
    page, hk, d, hq = 512, 1, 64, 4
    stride = (1 << 31) + 4096
    stores = [torch.zeros(2 * stride + page * d, dtype=torch.uint8, device=DEV) for _ in range(2)]
    views = [s.as_strided((3, page, hk, d), (stride, d, d, 1)) for s in stores]
    exps = [torch.zeros((3, page // 16, hk), dtype=torch.uint8, device=DEV) for _ in range(2)]
    table = torch.tensor([[2, 1]], dtype=torch.int32, device=DEV)
    k, v = randn(1, (700, hk, d), dtype), randn(2, (700, hk, d), dtype)
    sdi.dlrm_kv8_append(k, v, as64([0, 700]), as64([700]), table, *views, *exps)
    small = [t.clone().contiguous() for t in views]
    for rows in (1, 10, 40, 600):  # single tokens; one tile; many tiles, whose codes are converted
        q = randn(3, (rows, hq, d), dtype, 0.5)
        size = sdi.dlrm_kv8_attn_workspace_size(1, rows, hq, hk, d, rows, 700)
        got = []
        for codes in (views, small):
            ws, out = torch.empty(size, dtype=torch.uint8, device=DEV), torch.empty_like(q)
            sdi.dlrm_kv8_attn_fwd(q, as64([0, rows]), as64([700]), table, *codes, *exps, out, 0.125, ws, rows, 700)
            got.append(out)
        assert torch.equal(*got) and got[0].abs().max() > 0
