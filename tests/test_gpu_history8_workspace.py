"""Workspace of the attention in 8 bits: calls that convert no codes do without
the room for their copy."""
import numpy as np
import pytest
import torch

import sparse_dense_interaction_gb300 as sdi
from sparse_dense_interaction_gb300 import _native
from tests.test_gpu_history8 import DEV, DT, as64, attention_inputs, check_attention, flag, tensors8
from tests.test_gpu_history8_edges import _built  # noqa: F401

pytestmark = pytest.mark.gpu

# (counts, lengths, q heads, kv heads, d, page, block, heads first, causal, window, dtype), elements between query heads
# beside d: chunks whose codes would be converted if type and strides allowed it (the first has too few rows for that)
CASES = [
    (([400, 1], [500, 70], 8, 2, 64, 16, 8, False, True, 0, "f32"), 0, True),
    (([600, 1], [700, 70], 4, 1, 64, 16, 8, False, True, 0, "f32"), 0, True),
    (([600], [700], 4, 1, 128, 32, 32, True, True, 0, "f32"), 0, True),
    (([600], [700], 4, 1, 64, 32, 32, True, True, 0, "bf16"), 1, True),
    (([600], [700], 4, 1, 128, 32, 32, True, True, 0, "f16"), 4, True),
    (([600], [700], 4, 1, 128, 32, 32, True, True, 0, "bf16"), 0, False),
    (([600], [700], 4, 1, 64, 32, 32, True, True, 0, "f16"), 8, False),
]


@pytest.mark.parametrize("case,gap,enough", CASES)
def test_calls_without_a_copy_need_no_room_for_it(case, gap, enough):
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, given, caches, q = attention_inputs(case, seed=41)
    n = sum(counts)
    wide = torch.zeros((n, hq, d + gap), dtype=DT[dtype], device=DEV)
    wide[..., :d] = q
    sizes = (len(counts), n, hq, hk, d, max(counts), max(lengths))
    size, guard = sdi.dlrm_kv_attn_workspace_size(*sizes), 4096
    assert (size < sdi.dlrm_kv8_attn_workspace_size(*sizes)) == (max(counts) * hq // hk >= (1536 if d > 64 else 2048))
    buf = torch.full((size + guard,), 0xA5, dtype=torch.uint8, device=DEV)
    out, lse, f = torch.full_like(wide, 7), torch.full((n, hq), 7.0, device=DEV), flag()
    (kc, ke), (vc, ve) = (tensors8(*c, first) for c in caches)
    call = lambda size: sdi.dlrm_kv8_attn_fwd(
        wide[..., :d], as64([0] + list(np.cumsum(counts))), as64(lengths), torch.from_numpy(given).to(DEV), kc, vc, ke, ve,
        out[..., :d], d ** -0.5, buf[:size], max(counts), max(lengths), causal=causal, window=window, lse=lse, err_flag=f)
    for short in [size - 1] if enough else [size - 1, size]:
        with pytest.raises(_native.DlrmError) as error:
            call(short)
        assert error.value.status == _native.ERR_WORKSPACE_TOO_SMALL
    if enough:
        call(size)
        assert sdi.dlrm_read_error(f) == 0
        check_attention(case, table, caches, q, d ** -0.5, out[..., :d], lse)
    assert (buf[size:] == 0xA5).all() and (out[..., d:] == 7).all()
