"""The event history in 8 bits with keys, scales and queries near the ends of
fp32's range: scores that are finite stay so in every kernel."""
import numpy as np
import pytest

from tests import _history8_ref as R8
from tests import _history_ref as R
from tests.test_gpu_history8 import DT, attend, attention_inputs, check_attention, close, np64
from tests.test_gpu_history8_edges import KINDS, _built  # noqa: F401

pytestmark = pytest.mark.gpu


def lse_check(case, table, caches, q, scale, lse):
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    k, v = (np.nan_to_num(R8.values(*c), nan=0.0, posinf=0.0, neginf=0.0) for c in caches)
    _, want, _, smax, _ = R.attention(np64(q), counts, lengths, table, k, v, scale, causal, window)
    close(lse, want, R.lse_tolerance(want, smax, d), (case, "lse"))


# Keys of up to 2^8 * 2^(e - 127), queries of up to 4 or so and sums of 256: below 2^127 to e = 235.  Lifted
# queries (2^15) make that 2^141.  The scale takes the scores back to a few.
@pytest.mark.parametrize("low,high", [(228, 233), (150, 233), (2, 8)])
@pytest.mark.parametrize("case", KINDS)
def test_keys_near_the_ends_of_the_range(case, low, high):
    d = case[4]
    table, given, caches, q = attention_inputs(case, seed=11)
    r = np.random.RandomState(1)
    exps = caches[0][1]
    exps[exps < 255] = r.randint(low, high, int((exps < 255).sum()))
    scale = min(float(np.float32(2.0 ** (119 - high) / d ** 0.5)), 1e38)
    out, lse = attend(case, given, caches, q, scale)
    check_attention(case, table, caches, q, scale, out, lse)
    lse_check(case, table, caches, q, scale, lse)


# Queries at the other end from the keys: the product and the scale are ordinary, each factor is not.
@pytest.mark.parametrize("size,low,high", [(2.0 ** -100, 220, 226), (2.0 ** 90, 24, 30)])
@pytest.mark.parametrize("case", [c for c in KINDS if c[-1] != "f16"])
def test_queries_and_keys_at_opposite_ends(case, size, low, high):
    d, dtype = case[4], case[-1]
    table, given, caches, q = attention_inputs(case, seed=12)
    r = np.random.RandomState(2)
    exps = caches[0][1]
    exps[exps < 255] = r.randint(low, high, int((exps < 255).sum()))
    q = (q.double() * size).to(DT[dtype])
    q[0] = 0
    scale = float(np.float32(2.0 ** (119 - high) / size / d ** 0.5))
    out, lse = attend(case, given, caches, q, scale)
    check_attention(case, table, caches, q, scale, out, lse)


# A row of zeros scores 0 against every key, however large scale and keys are: the mean of the values.
@pytest.mark.parametrize("case", KINDS)
def test_a_query_of_zeros_under_a_large_scale(case):
    counts, lengths, hq, hk, d, page, block, first, causal, window, dtype = case
    table, given, caches, q = attention_inputs(case, seed=13)
    exps = caches[0][1]
    exps[exps < 255] = 200
    q[:] = 0
    out, lse = attend(case, given, caches, q, 1e38)
    check_attention(case, table, caches, q, 1e38, out, lse)
