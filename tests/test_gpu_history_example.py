"""The event-history example: what its candidates gather equals the formula on
the same items, and its training step lowers the loss."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import _history_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from sparse_dense_interaction_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "user_history.py")
    spec = importlib.util.spec_from_file_location("user_history", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_candidates_gather_from_their_histories(example):
    m = example.HistoryModel(dtype=torch.float32)
    store, past, counts, items, gathered, y = example.serve(m)
    lengths = [len(p) for p in past]
    assert lengths == store.lengths
    np64 = lambda t: t.double().cpu().numpy()
    heads = lambda ids: [np64(t) for t in m.heads(ids)]
    width = max(lengths)
    k = np.zeros((len(past), width, m.kv_heads, m.d))
    v = np.zeros_like(k)
    for u, ids in enumerate(past):
        _, ku, vu = heads(ids)
        k[u, :lengths[u]], _ = R.norm_rope(ku, np64(m.k_weight), m.eps, np64(m.rope), np.arange(lengths[u]))
        v[u, :lengths[u]] = vu
    q, _ = R.norm_rope(heads(items)[0], np64(m.q_weight), m.eps, np64(m.rope), np.repeat(lengths, counts))
    # a page a user: as long as the longest history
    want, _, absout, smax, flat = R.attention(q, counts, lengths, np.arange(len(past))[:, None], k, v, m.d ** -0.5,
                                              False, 0)
    # normed and rotated rows carry their own tolerance, which moves a score by 2 * 17 roundings more
    tol = R.attention_tolerance(want, absout, smax * (1 + 34 / (m.d + 4)), flat, m.d, "f32")
    assert (np.abs(np64(gathered) - want) <= tol).all()
    # the first pair: the candidate's own vector with its user's pooled items
    own, user = np64(m.table[items]), np.repeat(np.arange(len(past)), counts)
    recent = np.stack([np64(m.table[ids[-20:]]) for ids in past])
    size = (np.abs(own) * np.abs(recent).sum(1)[user]).sum(1)
    assert np.array_equal(np64(y)[:, :own.shape[1]], own)
    assert (np.abs(np64(y)[:, own.shape[1]] - (own * recent.sum(1)[user]).sum(1)) <= 1e-5 * size).all()


def test_training_lowers_the_loss(example):
    losses = example.train(example.HistoryModel())
    assert losses[-1] < 0.1 * losses[0] and all(b <= a for a, b in zip(losses, losses[1:]))
