"""Waits inside the attention kernels that run out on purpose (through the
library's testing hook, never by a fault): the call is flagged, ends soon,
writes nothing but its rows, and the next call is right."""
import time

import pytest
import torch

import sparse_dense_interaction_gb300 as sdi
from sparse_dense_interaction_gb300 import _native
from tests.test_gpu_history import DEV, DT, attention_inputs, flag

pytestmark = pytest.mark.gpu

GUARD = 4096


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_dense_interaction_gb300 import build
    build.build()


@pytest.fixture(autouse=True)
def _reset_hooks():
    yield
    sdi.dlrm_set_wait_test_hooks()


def guarded(shape, dtype, fill):
    """A tensor of `fill` inside a buffer of it, and the buffer."""
    size = 1
    for n in shape:
        size *= n
    buf = torch.full((size + 2 * GUARD,), fill, dtype=dtype, device=DEV)
    return buf, buf[GUARD:GUARD + size].view(shape)


CASES = [
    # rows of 16: whole and shared-out items, stages of 2 and 3, keys and values in stages of their own
    ([1, 1, 1], [300, 5, 90], 4, 2, 64, 16, False, True, 0, "f16"), ([1], [9000], 4, 1, 128, 16, True, True, 0, "bf16"),
    ([3, 1], [900, 4000], 4, 1, 128, 8, True, True, 0, "bf16"), ([1, 4], [700, 5000], 4, 2, 256, 16, True, True, 0, "f16"),
    ([2, 1], [700, 3000], 4, 2, 64, 32, False, True, 100, "f32"), ([1], [3000], 4, 2, 128, 16, True, True, 0, "f32"),
    # tiles: one and two query tiles, parts, mended first and last tiles, queries row by row, all row by row
    ([40], [333], 4, 2, 64, 16, True, True, 0, "f16"), ([150], [2000], 4, 2, 64, 16, True, False, 0, "bf16"),
    ([9], [20000], 4, 1, 128, 64, True, True, 0, "bf16"), ([300], [900], 3, 1, 128, 32, False, True, 200, "f16"),
    ([200, 5], [333, 64], 2, 1, 128, 7, False, True, 0, "f16"), ([64, 30], [64, 2000], 4, 1, 128, 128, True, True, 0, "bf16"),
]


@pytest.mark.parametrize("polls", [0, 1, 40])
@pytest.mark.parametrize("case", CASES)
def test_waits_that_run_out(case, polls):
    counts, lengths, hq, hk, d, page, first, causal, window, dtype = case
    table, table_d, offsets, lens, kc, vc, q = attention_inputs(case, stale=0.0)
    n = sum(counts)
    size = sdi.dlrm_kv_attn_workspace_size(len(counts), n, hq, hk, d, max(counts), max(lengths))
    out_buf, out = guarded((n, hq, d), DT[dtype], 7.0)
    lse_buf, lse = guarded((n, hq), torch.float32, 7.0)
    ws_buf, ws = guarded((size,), torch.uint8, 0xA5)
    kc0, vc0 = kc.clone(), vc.clone()

    def call(f):
        sdi.dlrm_kv_attn_fwd(q, offsets, lens, table_d, kc, vc, out, d ** -0.5, ws, max(counts), max(lengths),
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
    for buf, size, fill in ((out_buf, out.numel(), 7.0), (lse_buf, lse.numel(), 7.0), (ws_buf, size, 0xA5)):
        assert (buf[:GUARD] == fill).all() and (buf[GUARD + size:] == fill).all()
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)
    assert call(flag()) == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
