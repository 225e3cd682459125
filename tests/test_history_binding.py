"""What the event-history binding refuses before the C call, with stand-ins for
CUDA tensors (no GPU needed)."""
import pytest
import torch

from sparse_dense_interaction_gb300 import _history, _native


class OnGpu:
    """A tensor that says it is on the GPU; nothing reads its memory."""
    is_cuda = True

    def __init__(self, tensor):
        self._tensor = tensor

    def __getattr__(self, name):
        return getattr(self._tensor, name)


class Library:
    """Takes every call and remembers its name."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append(name) or 0


@pytest.fixture
def lib(monkeypatch):
    stub = Library()
    monkeypatch.setattr(_history, "load", lambda: stub)
    return stub


def heads(n=4, h=2, d=8):
    return OnGpu(torch.zeros(n, h, d))


def gradient(workspace=None, err_flag=None):
    x = heads()
    workspace = OnGpu(torch.zeros(64, dtype=torch.uint8)) if workspace is None else workspace
    _history.dlrm_qk_norm_rope_bwd(x, None, x, None, OnGpu(torch.ones(8)), None, 1e-6, None, None, x, None, None, None,
                                   workspace, err_flag=err_flag, stream=0)


def batch():
    return (OnGpu(torch.tensor([0, 4])), OnGpu(torch.tensor([4])), OnGpu(torch.zeros(1, 1, dtype=torch.int32)),
            OnGpu(torch.zeros(1, 16, 2, 8)), OnGpu(torch.zeros(1, 16, 2, 8)))


def attention(workspace=None, err_flag=None):
    workspace = OnGpu(torch.zeros(64, dtype=torch.uint8)) if workspace is None else workspace
    _history.dlrm_kv_attn_fwd(heads(), *batch(), heads(), 0.1, workspace, 4, 4, err_flag=err_flag, stream=0)


def append(workspace=None, err_flag=None):
    _history.dlrm_kv_append(heads(), heads(), *batch(), err_flag=err_flag, stream=0)


def norm(workspace=None, err_flag=None):
    _history.dlrm_qk_norm_rope_fwd(heads(), None, None, None, 1e-6, None, None, heads(), None, err_flag=err_flag, stream=0)


@pytest.mark.parametrize("call", [gradient, attention])
def test_workspaces_are_contiguous_and_on_the_gpu(lib, call):
    call()
    assert len(lib.calls) == 1
    for bad in (torch.zeros(64, dtype=torch.uint8), OnGpu(torch.zeros(64, 2, dtype=torch.uint8)[:, 0])):
        with pytest.raises(ValueError):
            call(workspace=bad)
    assert len(lib.calls) == 1


@pytest.mark.parametrize("call", [gradient, attention, append, norm])
def test_flags_are_int32_and_on_the_gpu(lib, call):
    call(err_flag=OnGpu(torch.zeros(1, dtype=torch.int32)))
    assert len(lib.calls) == 1
    for bad in (torch.zeros(1, dtype=torch.int32), OnGpu(torch.zeros(1, dtype=torch.int16)),
                OnGpu(torch.zeros(0, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call(err_flag=bad)
    assert len(lib.calls) == 1


@pytest.mark.parametrize("gone", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_the_current_stream_by_the_public_interface(monkeypatch, gone):
    class Stream:
        cuda_stream = 77

    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.setattr(torch._C, name, lambda *args: 5, raising=False)
    assert _native._stream(None) == 5
    monkeypatch.delattr(torch._C, gone)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream())
    assert _native._stream(None) == 77 and _native._stream(3) == 3 and _native._stream(Stream()) == 77
