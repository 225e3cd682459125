"""Event-history calls where a type's range, a NaN or a batch's own numbers
meet their edges, against the 64-bit formulas."""
import numpy as np
import pytest
import torch

from tests import _history_ref as R
from tests.test_gpu_history import DEV, attend, attention_inputs, close, np64

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
