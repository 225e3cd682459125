"""Page numbers that are none do not enter the ring of free pages: one bad entry of
a user who leaves costs nobody else's events."""
import numpy as np
import pytest
import torch

import sparse_dense_interaction_gb300 as sdi
from sparse_dense_interaction_gb300 import _native
from tests import _history8_ref as R8
from tests.test_gpu_history8 import DEV, RESERVE, as64, flag, reserve_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_dense_interaction_gb300 import build
    build.build()


def reference(counts, lengths, table, page, ring, state, n):
    """The reservation by the one-by-one bookkeeping, with the sound pages of those who leave moved together."""
    pages, moved, less = len(ring), table.copy(), lengths.copy()
    for s in np.flatnonzero(counts < 0):
        held = table[s, :-(-lengths[s] // page)]
        sound = held[(held >= 0) & (held < pages)]
        moved[s, :len(sound)] = sound
        less[s] = len(sound) * page
    want = list(R8.reserve(counts.tolist(), less.tolist(), moved, page, ring, state, n))
    want[2][counts < 0] = table[counts < 0]  # rows of those who leave are not written
    return want


@pytest.mark.parametrize("case", [c for c in RESERVE if c[4] > 0 and c[0] > 8])
@pytest.mark.parametrize("in_place", [False, True])
def test_bad_pages_of_users_who_leave(case, in_place):
    page = case[3]
    counts, lengths, table, ring, state = reserve_inputs(case)
    r = np.random.RandomState(case[6])
    spoiled = 0
    for i, s in enumerate(np.flatnonzero(counts < 0)):
        held = -(-int(lengths[s]) // page)
        # some rows whole, some with a few bad numbers, some with nothing but those
        for k in range(held):
            if i % 3 == 2 or (i % 3 == 1 and r.rand() < 0.3):
                table[s, k] = (-1, len(ring), -7, 2 ** 31 - 1)[r.randint(4)]
                spoiled += 1
    assert spoiled
    n = int(np.maximum(counts, 0).sum())
    want = reference(counts, lengths, table, page, ring, state, n)
    c, l, t, g = (torch.from_numpy(np.asarray(x)).to(DEV) for x in (counts, lengths, table, ring))
    c, l, st = c.long(), l.long(), as64(state)
    new_l, new_st = (l, st) if in_place else (torch.empty_like(l), torch.empty_like(st))
    offsets = torch.empty(len(counts) + 1, dtype=torch.int64, device=DEV)
    slots, positions = (torch.full((n,), -9, dtype=torch.int64, device=DEV) for _ in range(2))
    f = flag()
    sdi.dlrm_kv_reserve(c, l, t, page, g, st, new_st, offsets, new_l, slots, positions, err_flag=f)
    assert sdi.dlrm_read_error(f) == _native.ERR_INDEX_OOB
    for got, w, what in zip((offsets, new_l, t, g, new_st, slots, positions), want,
                            ("offsets", "lengths", "table", "ring", "state", "slots", "positions")):
        assert np.array_equal(got.cpu().numpy(), np.asarray(w)), what
    head, tail = new_st.tolist()
    free = g.cpu().numpy()[np.arange(head, tail) % len(ring)]
    assert ((free >= 0) & (free < len(ring))).all()


def test_a_bad_page_costs_nobody_else_an_event():
    """A user whose older pages were given back by hand leaves; the others fill the pool afterwards."""
    page, pages = 4, 8
    table = torch.tensor([[-1, 3, -7, 5], [-1] * 4, [-1] * 4], dtype=torch.int32, device=DEV)
    ring = torch.tensor([0, 1, 2, 4, 6, 7, -1, -1], dtype=torch.int32, device=DEV)
    state, lengths, offsets = as64([0, 6]), as64([15, 0, 0]), as64([0] * 4)
    f = flag()
    step = lambda *c, n=32: sdi.dlrm_kv_reserve(as64(c), lengths, table, page, ring, state, state, offsets, lengths, n=n,
                                                err_flag=f)
    step(-1, 0, 0)
    assert sdi.dlrm_read_error(f) == _native.ERR_INDEX_OOB
    assert state.tolist() == [0, 8] and ring.tolist() == [0, 1, 2, 4, 6, 7, 3, 5]
    sdi.dlrm_clear_error(f)
    step(0, 16, 16)
    assert sdi.dlrm_read_error(f) == 0
    assert lengths.tolist() == [0, 16, 16] and state.tolist() == [8, 8]
    assert sorted(table[1:].flatten().tolist()) == list(range(8))


def test_a_bad_entry_of_the_ring_leaves_it_with_its_user():
    """The caller's own ring holds a number that is none: its tokens have no slots, and it is not given out again."""
    page = 4
    table = torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
    ring, state = torch.tensor([0, 9, 2, 1], dtype=torch.int32, device=DEV), as64([0, 4])
    lengths, offsets, slots = as64([0, 0]), as64([0] * 3), as64([-9] * 8)
    f = flag()
    sdi.dlrm_kv_reserve(as64([8, 0]), lengths, table, page, ring, state, state, offsets, lengths, slots=slots, err_flag=f)
    assert sdi.dlrm_read_error(f) == _native.ERR_INDEX_OOB
    assert slots.tolist() == [0, 1, 2, 3, -1, -1, -1, -1] and lengths.tolist() == [8, 0]
    sdi.dlrm_clear_error(f)
    sdi.dlrm_kv_reserve(as64([-1, 0]), lengths, table, page, ring, state, state, offsets, lengths, n=8, err_flag=f)
    assert sdi.dlrm_read_error(f) == _native.ERR_INDEX_OOB
    assert state.tolist() == [2, 5] and [int(ring[i % 4]) for i in range(2, 5)] == [2, 1, 0]
