"""The calls of the event history in 8 bits reject bad arguments on the host,
before anything is launched, in the library and in the binding (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_dense_interaction_gb300 as sdi
from sparse_dense_interaction_gb300 import _history8, _native, build
from tests import _history8_ref as R8
from tests.test_history_abi import BAD, FAKE, OK, SMALL, UNSUPPORTED, batch, heads, ref

_i32, _i64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class Cache8(ctypes.Structure):
    _fields_ = [(x, _vp) for x in ("k", "v", "k_exp", "v_exp")] + [
        (x, _i64) for x in ("pages", "page_stride", "slot_stride", "head_stride", "exp_page_stride",
                            "exp_block_stride", "exp_head_stride")] + [(x, _i32) for x in ("page_size", "heads", "block")]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.load()


@pytest.fixture(autouse=True)
def _nothing_is_launched(lib):
    before = lib.dlrm_kernel_launch_count()
    yield
    assert lib.dlrm_kernel_launch_count() == before


def cache8(k=FAKE, v=FAKE, ke=FAKE, ve=FAKE, pages=9, page=4096, slot=256, head=64, epage=16, eblock=4, ehead=1, size=16,
           n=4, block=4):
    return Cache8(k, v, ke, ve, pages, page, slot, head, epage, eblock, ehead, size, n, block)


CHECKS = [
    (BAD, dict(b=None)), (BAD, dict(b=batch(S=-1))), (BAD, dict(b=batch(S=0))), (BAD, dict(b=batch(lengths=None))),
    (UNSUPPORTED, dict(b=batch(S=(1 << 24) + 1))), (UNSUPPORTED, dict(b=batch(width=1 << 27))),
    (BAD, dict(c=None)), (BAD, dict(c=cache8(k=None))), (BAD, dict(c=cache8(v=None))), (BAD, dict(c=cache8(ke=None))),
    (BAD, dict(c=cache8(ve=None))), (BAD, dict(c=cache8(pages=0))), (UNSUPPORTED, dict(c=cache8(pages=1 << 31))),
    (BAD, dict(c=cache8(size=0))), (UNSUPPORTED, dict(c=cache8(size=1 << 17))), (BAD, dict(c=cache8(page=-1))),
    (BAD, dict(c=cache8(epage=-1))), (BAD, dict(c=cache8(eblock=-1))), (BAD, dict(c=cache8(ehead=-1))),
    (BAD, dict(c=cache8(block=0))), (BAD, dict(c=cache8(block=3))), (BAD, dict(c=cache8(block=32))),
    (UNSUPPORTED, dict(d=257)), (BAD, dict(d=0)), (BAD, dict(dtype=3)), (BAD, dict(dtype=-1)),
]


@pytest.mark.parametrize("want,kw", CHECKS + [
    (BAD, dict(k=None)), (BAD, dict(v=None)), (BAD, dict(k=heads(n=3))), (BAD, dict(v=heads(n=3))),
    (BAD, dict(k=heads(ptr=FAKE + 1))), (BAD, dict(c=cache8(page=63))), (BAD, dict(c=cache8(slot=63))),
    (BAD, dict(c=cache8(head=0))), (BAD, dict(c=cache8(epage=0))), (BAD, dict(c=cache8(eblock=0))),
    (BAD, dict(c=cache8(ehead=0))), (OK, dict(b=batch(n=0))),
])
def test_append_checks(lib, want, kw):
    a = dict(k=heads(), v=heads(), b=batch(), c=cache8(), d=64, dtype=1) | kw
    assert lib.dlrm_kv8_append(ref(a["k"]), ref(a["v"]), ref(a["b"]), ref(a["c"]), a["d"], a["dtype"], None, None) == want


@pytest.mark.parametrize("want,kw", CHECKS + [
    (BAD, dict(q=None)), (BAD, dict(out=None)), (BAD, dict(q=heads(n=6), out=heads(n=6))), (BAD, dict(out=heads(n=4))),
    (BAD, dict(out=heads(n=8, head=0))), (BAD, dict(scale=0.0)), (BAD, dict(scale=float("nan"))),
    (BAD, dict(scale=2.5e38)), (BAD, dict(causal=2)), (BAD, dict(window=-1)), (BAD, dict(max_new=0)),
    (BAD, dict(max_new=-1)), (BAD, dict(max_len=-1)), (UNSUPPORTED, dict(max_len=1 << 31)), (BAD, dict(lse=FAKE + 2)),
    (BAD, dict(ws=None)), (BAD, dict(ws=FAKE + 8)), (SMALL, dict(ws_bytes=-1)), (OK, dict(b=batch(n=0))),
])
def test_attention_checks(lib, want, kw):
    need = sdi.dlrm_kv8_attn_workspace_size(2, 8, 8, 4, 64, 8, 64)
    assert need > 0
    a = dict(q=heads(n=8), b=batch(), c=cache8(), d=64, dtype=1, scale=0.1, causal=1, window=0, max_new=8, max_len=64,
             out=heads(n=8), lse=FAKE, ws=FAKE, ws_bytes=0) | kw
    assert lib.dlrm_kv8_attn_fwd(ref(a["q"]), ref(a["b"]), ref(a["c"]), a["d"], a["dtype"], a["scale"], a["causal"],
                                 a["window"], a["max_new"], a["max_len"], ref(a["out"]), a["lse"], a["ws"],
                                 need + a["ws_bytes"], None, None) == want


@pytest.mark.parametrize("bad", [dict(S=-1), dict(S=(1 << 24) + 1), dict(n=-1), dict(n=1 << 31), dict(q_heads=6),
                                 dict(kv_heads=0), dict(d=0), dict(d=257), dict(max_new=-1), dict(max_len=1 << 31)])
def test_workspace_size_of_invalid_sizes(bad):
    assert sdi.dlrm_kv8_attn_workspace_size(**dict(S=2, n=8, q_heads=8, kv_heads=4, d=64, max_new=8, max_len=64) | bad) == 0


@pytest.mark.parametrize("want,kw", [
    (BAD, dict(S=-1)), (BAD, dict(n=-1)), (UNSUPPORTED, dict(S=(1 << 24) + 1)), (UNSUPPORTED, dict(n=1 << 31)),
    (BAD, dict(counts=None)), (BAD, dict(lengths=None)), (BAD, dict(new_lengths=None)), (BAD, dict(table=None)),
    (BAD, dict(ring=None)), (BAD, dict(state=None)), (BAD, dict(new_state=None)), (BAD, dict(offsets=None)),
    (BAD, dict(stride=7)), (BAD, dict(stride=-1)), (BAD, dict(width=-1)), (BAD, dict(page=0)),
    (UNSUPPORTED, dict(page=65537)), (BAD, dict(pages=0)), (UNSUPPORTED, dict(pages=1 << 31)),
    (UNSUPPORTED, dict(width=1 << 27, stride=1 << 27)), (BAD, dict(counts=FAKE + 4)), (BAD, dict(lengths=FAKE + 4)),
    (BAD, dict(slots=FAKE + 4)), (BAD, dict(positions=FAKE + 4)), (BAD, dict(table=FAKE + 2)), (BAD, dict(ring=FAKE + 2)),
    (BAD, dict(state=FAKE + 4)), (BAD, dict(offsets=FAKE + 4)),
])
def test_reserve_checks(lib, want, kw):
    a = dict(counts=FAKE, lengths=FAKE, S=2, n=8, table=FAKE, stride=8, width=8, page=16, ring=FAKE, pages=9, state=FAKE,
             new_state=FAKE, offsets=FAKE, new_lengths=FAKE, slots=FAKE, positions=FAKE) | kw
    assert lib.dlrm_kv_reserve(*a.values(), None, None) == want


class OnGpu:
    """A tensor that says it is on a GPU; nothing reads its memory."""
    is_cuda = True

    def __init__(self, tensor, device=0):
        self._tensor, self._device = tensor, device

    def get_device(self):
        return self._device

    def __getattr__(self, name):
        return getattr(self._tensor, name)


class Library:
    """Takes every call and remembers its name."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append(name) or 0


@pytest.fixture
def stub(monkeypatch):
    stub = Library()
    monkeypatch.setattr(_history8, "load", lambda: stub)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return stub


def arguments():
    z = lambda *shape, dtype=torch.float16: OnGpu(torch.zeros(*shape, dtype=dtype))
    code = torch.float8_e4m3fn
    return dict(k=z(4, 2, 8), v=z(4, 2, 8), offsets=OnGpu(torch.tensor([0, 4])), lengths=OnGpu(torch.tensor([4])),
                page_table=z(1, 1, dtype=torch.int32), k_cache=z(1, 16, 2, 8, dtype=code),
                v_cache=z(1, 16, 2, 8, dtype=code), k_exp=z(1, 4, 2, dtype=torch.uint8),
                v_exp=z(1, 4, 2, dtype=torch.uint8))


def append(**kw):
    sdi.dlrm_kv8_append(**arguments() | kw, stream=0)


def attend(**kw):
    a = arguments()
    q = a.pop("k")
    a.pop("v")
    sdi.dlrm_kv8_attn_fwd(**dict(q=q, out=q, scale=0.1, workspace=OnGpu(torch.zeros(64, dtype=torch.uint8)), max_new=4,
                                 max_len=4) | a | kw, stream=0)


def reserve(**kw):
    i = lambda *x: OnGpu(torch.zeros(*x, dtype=torch.int64))
    sdi.dlrm_kv_reserve(**dict(counts=i(3), lengths=i(3), page_table=OnGpu(torch.zeros(3, 4, dtype=torch.int32)),
                               page_size=16, ring=OnGpu(torch.zeros(9, dtype=torch.int32)), state=i(2), new_state=i(2),
                               offsets=i(4), new_lengths=i(3), slots=i(5)) | kw, stream=0)


t = lambda *shape, dtype=torch.uint8, device=0: OnGpu(torch.zeros(*shape, dtype=dtype), device)


@pytest.mark.parametrize("call,bad", [(c, b) for c in (append, attend) for b in [
    dict(k_cache=t(1, 16, 2, 8, dtype=torch.float16)), dict(k_cache=t(2, 16, 2, 8, dtype=torch.float8_e4m3fn)),
    dict(v_cache=t(1, 16, 2, 8)), dict(k_exp=t(1, 3, 2), v_exp=t(1, 3, 2)), dict(k_exp=t(1, 4, 3), v_exp=t(1, 4, 3)),
    dict(k_exp=t(2, 4, 2), v_exp=t(2, 4, 2)), dict(v_exp=t(1, 2, 2)), dict(k_exp=t(1, 4, 2, dtype=torch.int8)),
    dict(k_cache=t(1, 16, 2, 8, dtype=torch.float8_e4m3fn, device=1)), dict(lengths=torch.tensor([4])),
    dict(err_flag=t(1, dtype=torch.int64)), dict(page_table=t(2, 1, dtype=torch.int32)),
]] + [
    (append, dict(v=t(4, 2, 9, dtype=torch.float16))), (append, dict(v=t(4, 2, 8, dtype=torch.float32))),
    (attend, dict(out=t(4, 2, 8, dtype=torch.float32))), (attend, dict(lse=t(4, 3, dtype=torch.float32))),
    (attend, dict(workspace=torch.zeros(64, dtype=torch.uint8))),
    (reserve, dict(counts=t(3, dtype=torch.int32))), (reserve, dict(lengths=t(2, dtype=torch.int64))),
    (reserve, dict(page_table=t(3, 4, dtype=torch.int64))), (reserve, dict(page_table=t(2, 4, dtype=torch.int32))),
    (reserve, dict(ring=t(9, dtype=torch.int64))), (reserve, dict(state=t(3, dtype=torch.int64))),
    (reserve, dict(offsets=t(3, dtype=torch.int64))), (reserve, dict(positions=t(4, dtype=torch.int64))),
    (reserve, dict(slots=None)), (reserve, dict(new_lengths=t(3, dtype=torch.int64, device=1))),
])
def test_binding_refuses(stub, call, bad):
    call()
    assert len(stub.calls) == 1
    with pytest.raises(ValueError):
        call(**bad)
    assert len(stub.calls) == 1


def test_binding_takes_bytes_and_either_row(stub):
    append(k_cache=t(1, 16, 2, 8), v_cache=t(1, 16, 2, 8))
    reserve(slots=None, positions=t(5, dtype=torch.int64))
    reserve(slots=None, n=5)
    assert len(stub.calls) == 3


def test_reference_codes_are_torchs():
    r = np.random.RandomState(0)
    x = np.concatenate([r.randn(5000) * 2.0 ** r.randint(-12, 10, 5000), R8.POSITIVE, -R8.POSITIVE,
                        (R8.POSITIVE[1:] + R8.POSITIVE[:-1]) / 2, [0.0, -0.0]]).astype(np.float32)
    codes = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R8.encode(x), codes)
    assert np.array_equal(torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy(), R8.CODES,
                          equal_nan=True)


def test_reference_exponents():
    for top, e in [(0.0, 0), (448.0, 127), (448.0001, 128), (449, 128), (1.75, 119), (1.76, 120), (2.0 ** -149, 1),
                   (3.4e38, 247)]:
        assert R8.exponent(top) == e
