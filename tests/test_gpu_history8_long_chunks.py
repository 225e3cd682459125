"""Long chunks over the event history in 8 bits, whose codes are converted once:
the bits that their weights have."""
import numpy as np
import pytest
import torch

from tests import _history8_ref as R8
from tests import _history_ref as R
from tests.test_gpu_history8 import attend, attention_inputs, close, flag, np64
from tests.test_gpu_history8_edges import KINDS, _built  # noqa: F401

import sparse_dense_interaction_gb300 as sdi

pytestmark = pytest.mark.gpu

# (counts, lengths, q heads, kv heads, d, page, block, heads first, causal, window, dtype); 1535 rows and fewer are not
# converted, nor are heads above 128
CHUNKS = [
    ([400, 3], [400, 70], 8, 2, 96, 16, 8, False, True, 0, "bf16"), ([600], [601], 4, 1, 64, 32, 32, True, True, 0, "bf16"),
    ([383, 10], [390, 12], 8, 2, 128, 64, 16, True, True, 0, "bf16"), ([384], [384], 8, 2, 128, 64, 16, True, True, 0, "bf16"),
    ([400], [400], 8, 2, 128, 16, 1, False, True, 9, "f16"),
]


# A weight is rounded to fp16 (2^-11 of it), whatever the type; where values cancel, that is more than the rounding of
# the output.  The rest is the 16-bit cache's tolerance without its rounding of weights.  The rows that see few keys
# show it: the more keys, the more the roundings even out.
@pytest.mark.parametrize("case", CHUNKS)
def test_weights_have_eleven_bits(case):
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, given, caches, q = attention_inputs(case, seed=21)
    scale, f = 1 / d ** 0.5, flag()
    out, _ = attend(case, given, caches, q, scale, f)
    assert sdi.dlrm_read_error(f) == 0
    with np.errstate(over="ignore", invalid="ignore"):
        k, v = (np.nan_to_num(R8.values(*c), nan=0.0, posinf=0.0, neginf=0.0) for c in caches)
    want, _, absout, smax, flat = R.attention(np64(q), counts, lengths, table, k, v, scale, causal, window)
    tol = R.attention_tolerance(want, absout, smax, flat, d, "f32") + 2.0 ** -11 * 1.01 * absout
    tol = tol + R.U[dtype] * 1.01 * np.abs(want) + R.TINY[dtype] * (1 + flat)
    close(out, want, tol + 2.0 ** -36 * np.abs(v).max() * max(lengths), case)


# One row's scores grow by much along the history, those of the others by less than a maximum is let lag: with the one
# row gone (NaN) the others keep their bits.
@pytest.mark.parametrize("case", KINDS)
def test_bits_do_not_depend_on_other_rows(case):
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, given, caches, q = attention_inputs(case, seed=22)
    for s, n in enumerate(lengths):
        own = -(-n // page)
        for i in range(own):  # keys grow by 2^6 in all
            caches[0][1][table[s, i]] = 114 + int(6 * i / max(own - 1, 1))
    one = torch.zeros(q.shape[:2], dtype=torch.bool, device=q.device)
    one[-1, hq - 1] = True  # the last row of the batch
    q = q * 0.25
    q[one] *= 64
    with_one, lse_with = attend(case, given, caches, q, 0.5 / d ** 0.5)
    q[one] = float("nan")
    out, lse = attend(case, given, caches, q, 0.5 / d ** 0.5)
    assert out[one].isnan().all() and lse[one].isnan().all()
    assert torch.equal(out[~one], with_one[~one]) and torch.equal(lse[~one], lse_with[~one])
