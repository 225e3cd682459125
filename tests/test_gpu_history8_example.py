"""The event-history example with its histories in 8 bits: what is stored lies
within a code's rounding of the formula's keys and values, what the candidates
gather equals the formula over what is stored."""
import numpy as np
import pytest
import torch

from tests import _history8_ref as R8
from tests import _history_ref as R
from tests.test_gpu_history_example import example  # noqa: F401

pytestmark = pytest.mark.gpu


def test_candidates_gather_from_histories_in_8_bits(example):  # noqa: F811
    m = example.HistoryModel(dtype=torch.float32)
    store, past, counts, items, gathered, y = example.serve(m, kind=example.Histories8)
    lengths = [len(p) for p in past]
    assert lengths == store.lengths == store.stored.tolist()
    np64 = lambda t: t.double().cpu().numpy()
    table = store.pages.cpu().numpy()
    k, v = (R8.values(c.contiguous().cpu().numpy(), e.cpu().numpy()) for c, e in ((store.k, store.k_exp), (store.v, store.v_exp)))
    for u, ids in enumerate(past):
        _, ku, vu = (np64(t) for t in m.heads(ids))
        keys, _ = R.norm_rope(ku, np64(m.k_weight), m.eps, np64(m.rope), np.arange(lengths[u]))
        at = np.arange(lengths[u])
        for got, want, exps in ((k, keys, store.k_exp), (v, vu, store.v_exp)):
            power = R8.power(exps.cpu().numpy().repeat(16, 1)[table[u, at // 16], at % 16])[..., None]
            held = got[table[u, at // 16], at % 16]
            assert (np.abs(held - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * power + 1e-5).all()
    q, _ = R.norm_rope(np64(m.heads(items)[0]), np64(m.q_weight), m.eps, np64(m.rope), np.repeat(lengths, counts))
    want, _, absout, smax, flat = R.attention(q, counts, lengths, table, k, v, m.d ** -0.5, False, 0)
    # normed and rotated rows carry their own tolerance, which moves a score by 2 * 17 roundings more
    tol = R.attention_tolerance(want, absout, smax * (1 + 34 / (m.d + 4)), flat, m.d, "f32")
    assert (np.abs(np64(gathered) - want) <= tol + 2.0 ** -36 * np.abs(v).max() * max(lengths)).all()
    assert torch.isfinite(y).all()


def test_a_user_leaves_and_others_take_the_pages(example):  # noqa: F811
    m = example.HistoryModel(items=50)
    store = example.Histories8(m, 3, pages=7, pages_of_user=4)
    items = lambda n: torch.arange(n, device=m.device) % 50
    store.append([40, 20, 16], items(76))  # six of seven pages
    gone = store.pages.tolist()[0][:3]
    store.append([-1, 1, 0], items(1))
    store.append([20, 0, 30], items(50))  # the seventh, and the three of the user who left
    assert store.stored.tolist() == store.lengths == [20, 21, 46]
    held = [p for u, n in enumerate(store.lengths) for p in store.pages.tolist()[u][:-(-n // 16)]]
    assert sorted(held) == list(range(7)) and set(gone) <= set(held)
    assert m.err.item() == 0
