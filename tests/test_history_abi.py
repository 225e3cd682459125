"""The event-history calls reject bad arguments on the host, before anything is
launched (no GPU needed)."""
import ctypes

import pytest
import torch

import sparse_dense_interaction_gb300 as sdi
from sparse_dense_interaction_gb300 import _history, _native, build

FAKE = 0x10000  # never dereferenced: every call below fails its host checks first
BAD, UNSUPPORTED, SMALL, OK = (_native.ERR_INVALID_ARG, _native.ERR_UNSUPPORTED, _native.ERR_WORKSPACE_TOO_SMALL,
                               _native.OK)


_i32, _i64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class Heads(ctypes.Structure):
    _fields_ = [("ptr", _vp), ("token_stride", _i64), ("head_stride", _i64), ("heads", _i32)]


class Rope(ctypes.Structure):
    _fields_ = [("table", _vp), ("length", _i64), ("positions", _vp), ("rot", _i32), ("layout", _i32)]


class Cache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("pages", _i64), ("page_stride", _i64), ("slot_stride", _i64),
                ("head_stride", _i64), ("page_size", _i32), ("heads", _i32)]


class Batch(ctypes.Structure):
    _fields_ = [("S", _i64), ("n", _i64), ("offsets", _vp), ("lengths", _vp), ("page_table", _vp),
                ("table_stride", _i64), ("table_width", _i64)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.load()


@pytest.fixture(autouse=True)
def _nothing_is_launched(lib):
    before = lib.dlrm_kernel_launch_count()
    yield
    assert lib.dlrm_kernel_launch_count() == before


def heads(ptr=FAKE, token=256, head=64, n=4):
    return Heads(ptr, token, head, n)


def rope(table=FAKE, length=10, positions=FAKE, rot=64, layout=0):
    return Rope(table, length, positions, rot, layout)


def batch(S=2, n=8, offsets=FAKE, lengths=FAKE, table=FAKE, stride=4, width=4):
    return Batch(S, n, offsets, lengths, table, stride, width)


def cache(k=FAKE, v=FAKE, pages=9, page=4096, slot=256, head=64, size=16, n=4):
    return Cache(k, v, pages, page, slot, head, size, n)


ref = lambda x: None if x is None else ctypes.byref(x)


@pytest.mark.parametrize("want,kw", [
    (BAD, dict(n=-1)), (BAD, dict(d=0)), (UNSUPPORTED, dict(d=257)), (BAD, dict(dtype=3)), (BAD, dict(dtype=-1)),
    (UNSUPPORTED, dict(n=1 << 31)), (BAD, dict(q=None)), (BAD, dict(q=heads(ptr=None))), (BAD, dict(q=heads(n=0))),
    (BAD, dict(q=heads(ptr=FAKE + 1))), (BAD, dict(q=heads(token=-1))), (BAD, dict(q=heads(head=-64))),
    (BAD, dict(qo=None)), (BAD, dict(qo=heads(n=3))), (BAD, dict(k=None)), (BAD, dict(ko=None)),
    (UNSUPPORTED, dict(q=heads(n=65537), qo=heads(n=65537))),
    (BAD, dict(eps=-1.0)), (BAD, dict(eps=float("nan"))), (BAD, dict(eps=float("inf"))),
    (BAD, dict(qw=FAKE + 2)), (BAD, dict(rope=rope(rot=66))), (BAD, dict(rope=rope(rot=3))),
    (BAD, dict(rope=rope(rot=0))), (BAD, dict(rope=rope(table=None))), (BAD, dict(rope=rope(positions=None))),
    (BAD, dict(qo=heads(head=63))), (BAD, dict(ko=heads(token=0))), (BAD, dict(qo=heads(token=63))),  # rows overlap
    (BAD, dict(rope=rope(layout=2))), (BAD, dict(rope=rope(length=-1))), (BAD, dict(rope=rope(positions=FAKE + 4))),
    (OK, dict(n=0)), (OK, dict(n=0, k=None, ko=None)), (OK, dict(n=0, rope=None, qw=None, kw=None)),
])
def test_norm_rope_checks(lib, want, kw):
    a = dict(q=heads(), k=heads(), n=8, d=64, dtype=1, qw=FAKE, kw=FAKE, eps=1e-6, rope=rope(), qo=heads(),
             ko=heads()) | kw
    assert lib.dlrm_qk_norm_rope_fwd(ref(a["q"]), ref(a["k"]), a["n"], a["d"], a["dtype"], a["qw"], a["kw"], a["eps"],
                                     ref(a["rope"]), ref(a["qo"]), ref(a["ko"]), None, None) == want


@pytest.mark.parametrize("want,kw", [
    (BAD, dict(dq=None)), (BAD, dict(dqo=None)), (BAD, dict(dqo=heads(n=5))), (BAD, dict(dk=None)),
    (BAD, dict(dko=None)), (BAD, dict(dko=heads(n=3))), (BAD, dict(dq=heads(head=0))),
    (BAD, dict(qw=None)), (BAD, dict(kw=None)), (BAD, dict(dqw=FAKE + 1)), (BAD, dict(ws=None)),
    (BAD, dict(ws=FAKE + 8)), (SMALL, dict(ws_bytes=None)), (BAD, dict(rope=rope(rot=65))),
    (BAD, dict(k=None, dk=None, dko=None)),  # the keys' weight gradient without keys
    (OK, dict(n=0, dqw=None, dkw=None)),
])
def test_norm_rope_gradient_checks(lib, want, kw):
    need = sdi.dlrm_qk_norm_rope_bwd_workspace_size(8, 4, 4, 64)
    assert need > 0
    a = dict(dqo=heads(), dko=heads(), q=heads(), k=heads(), n=8, d=64, qw=FAKE, kw=FAKE, rope=rope(), dq=heads(),
             dk=heads(), dqw=FAKE, dkw=FAKE, ws=FAKE, ws_bytes=need) | kw
    ws_bytes = need - 1 if a["ws_bytes"] is None else a["ws_bytes"]
    assert lib.dlrm_qk_norm_rope_bwd(
        ref(a["dqo"]), ref(a["dko"]), ref(a["q"]), ref(a["k"]), a["n"], a["d"], 2, a["qw"], a["kw"], 1e-6,
        ref(a["rope"]), ref(a["dq"]), ref(a["dk"]), a["dqw"], a["dkw"], a["ws"], ws_bytes, None, None) == want


BATCH_CHECKS = [
    (BAD, dict(b=None)), (BAD, dict(b=batch(S=-1))), (BAD, dict(b=batch(n=-1))), (BAD, dict(b=batch(S=0))),
    (UNSUPPORTED, dict(b=batch(S=(1 << 24) + 1))), (BAD, dict(b=batch(offsets=None))),
    (BAD, dict(b=batch(lengths=None))), (BAD, dict(b=batch(table=None))), (BAD, dict(b=batch(stride=-1))),
    (BAD, dict(b=batch(offsets=FAKE + 4))), (BAD, dict(b=batch(table=FAKE + 2))),
    (UNSUPPORTED, dict(b=batch(width=1 << 27))),  # 2^31 positions
    (BAD, dict(c=None)), (BAD, dict(c=cache(k=None))), (BAD, dict(c=cache(v=None))), (BAD, dict(c=cache(pages=0))),
    (UNSUPPORTED, dict(c=cache(pages=1 << 31))), (BAD, dict(c=cache(size=0))), (UNSUPPORTED, dict(c=cache(size=65537))),
    (BAD, dict(c=cache(page=-1))), (BAD, dict(c=cache(n=0))), (BAD, dict(c=cache(k=FAKE + 1))),
    (UNSUPPORTED, dict(d=300)), (BAD, dict(d=-1)), (BAD, dict(dtype=7)),
]


@pytest.mark.parametrize("want,kw", BATCH_CHECKS + [
    (BAD, dict(k=None)), (BAD, dict(v=None)), (BAD, dict(k=heads(n=3))), (BAD, dict(v=heads(n=5))),
    (BAD, dict(qo=None)), (BAD, dict(q=None)), (BAD, dict(eps=-1.0)), (BAD, dict(rope=rope(rot=1))),
    (BAD, dict(c=cache(page=0))), (BAD, dict(c=cache(slot=32))), (BAD, dict(c=cache(head=0))),  # slots overlap
    (OK, dict(b=batch(n=0))), (OK, dict(b=batch(S=0, n=0))),
])
def test_append_checks(lib, want, kw):
    a = dict(k=heads(), v=heads(), b=batch(), c=cache(), d=64, dtype=2, kw=FAKE, eps=1e-6, rope=rope(positions=None),
             q=heads(n=8), qo=heads(n=8)) | kw
    assert lib.dlrm_kv_append(ref(a["k"]), ref(a["v"]), ref(a["b"]), ref(a["c"]), a["d"], a["dtype"], a["kw"],
                              a["eps"], ref(a["rope"]), ref(a["q"]), FAKE, ref(a["qo"]), None, None) == want


@pytest.mark.parametrize("want,kw", BATCH_CHECKS + [
    (BAD, dict(q=None)), (BAD, dict(out=None)), (BAD, dict(q=heads(n=6), out=heads(n=6))), (BAD, dict(out=heads())),
    (BAD, dict(scale=0.0)), (BAD, dict(scale=-1.0)), (BAD, dict(scale=float("nan"))), (BAD, dict(scale=float("inf"))),
    (BAD, dict(causal=2)), (BAD, dict(window=-1)), (BAD, dict(max_new=-1)), (BAD, dict(max_len=-1)),
    (BAD, dict(max_new=0)), (UNSUPPORTED, dict(max_len=1 << 31)), (BAD, dict(lse=FAKE + 2)), (BAD, dict(ws=None)),
    (BAD, dict(out=heads(n=8, token=0))), (BAD, dict(out=heads(n=8, head=0))),
    (BAD, dict(ws=FAKE + 8)), (SMALL, dict(short=1)), (OK, dict(b=batch(n=0))), (OK, dict(b=batch(S=0, n=0))),
])
def test_attention_checks(lib, want, kw):
    need = sdi.dlrm_kv_attn_workspace_size(2, 8, 8, 4, 64, 4, 60)
    assert need > 0
    a = dict(q=heads(n=8), b=batch(), c=cache(), d=64, dtype=2, scale=0.1, causal=1, window=0, max_new=4, max_len=60,
             out=heads(n=8), lse=FAKE, ws=FAKE, short=0) | kw
    assert lib.dlrm_kv_attn_fwd(ref(a["q"]), ref(a["b"]), ref(a["c"]), a["d"], a["dtype"], a["scale"], a["causal"],
                                a["window"], a["max_new"], a["max_len"], ref(a["out"]), a["lse"], a["ws"],
                                need - a["short"], None, None) == want


def test_packed_structs_match_the_header():
    for pack, struct, values in ((_history._HEADS, Heads, (5, 6, 7, 8)), (_history._ROPE, Rope, (5, 6, 7, 8, 1)),
                                 (_history._CACHE, Cache, (5, 6, 7, 8, 9, 10, 11, 12)),
                                 (_history._BATCH, Batch, (5, 6, 7, 8, 9, 10, 11))):
        packed = struct.from_buffer_copy(pack(*values))
        assert len(pack(*values)) == ctypes.sizeof(struct)
        assert tuple(getattr(packed, name) for name, _ in struct._fields_) == values


def test_workspace_sizes_of_invalid_sizes(lib):
    assert sdi.dlrm_qk_norm_rope_bwd_workspace_size(-1, 1, 1, 64) == 0
    assert sdi.dlrm_qk_norm_rope_bwd_workspace_size(1, 0, 1, 64) == 0
    assert sdi.dlrm_qk_norm_rope_bwd_workspace_size(1, 1, 1, 257) == 0
    good = (2, 8, 8, 4, 64, 4, 60)
    for i, x in ((0, -1), (1, -1), (2, 6), (2, 0), (3, 0), (4, 0), (4, 257), (5, -1), (6, -1), (6, 1 << 31)):
        bad = list(good)
        bad[i] = x
        assert sdi.dlrm_kv_attn_workspace_size(*bad) == 0, bad
    # a split history keeps partial rows, more with more heads
    one = sdi.dlrm_kv_attn_workspace_size(1, 1, 8, 2, 128, 1, 100000)
    assert 8 * 128 * 4 < one < sdi.dlrm_kv_attn_workspace_size(1, 1, 16, 2, 128, 1, 100000)


def test_binding_refuses_tensors_that_do_not_fit(lib):
    x = torch.zeros(4, 2, 8)
    at = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):  # not on the GPU
        sdi.dlrm_qk_norm_rope_fwd(x, None, None, None, 1e-6, None, at, x.clone(), None)
    with pytest.raises(ValueError):
        sdi.dlrm_kv_append(x, x, at, at[:3], torch.zeros(3, 2, dtype=torch.int32), x[None], x[None])
    ws = torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        sdi.dlrm_kv_attn_fwd(x, at, at[:3], torch.zeros(3, 2, dtype=torch.int32), x[None], x[None], x, 1.0, ws, 1, 1)
