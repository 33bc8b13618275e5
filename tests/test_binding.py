"""The Python binding without a GPU: what it needs of torch, and the tensors it takes."""
import subprocess
import sys

import pytest

from oracle_top_kv_b200 import hs


class Tensor:
    """What the binding asks of a CUDA tensor."""

    def __init__(self, at, device=0, contiguous=True):
        self.at, self.device, self.contiguous = at, device, contiguous
        self.is_cuda = True

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return self.at


class Library:
    """Takes every call, and notes its arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return hs.HS_OK
        return call


def test_the_module_needs_no_private_names_of_torch():
    """A torch build without CUDA has neither; with them gone the public calls serve."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from oracle_top_kv_b200 import hs
hs.make_params(1, 1, 1, 64, 1, 1)
class S:
    cuda_stream = 77
torch.cuda.current_device = lambda: 3
torch.cuda.current_stream = lambda device=None: S if device == 3 else None
assert hs._current_device() == 3 and hs._stream(None) == 77 and hs._stream(5) == 5 and hs._stream(S) == 77
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(hs, "load", lambda: lib)
    monkeypatch.setattr(hs, "_current_device", lambda: 0)
    return lib


def test_earlier_entry_points_take_a_peers_tensors(lib):
    """Memory of another GPU, which the current one may reach: the caller's to know."""
    p = hs.make_params(1, 1, 1, 64, 1, 1, mode="token", block_size=1, k=1, window=0)
    t = [Tensor(16 * (i + 1), device=1) for i in range(8)]
    hs.hs_decode_step(p, hs.HS_DECODE_SPARSE, *t, stream=0)
    hs.hs_full_attn_index(p, *t[:7], stream=0)
    hs.hs_sparse_attn_reuse(p, *t[:5], None, None, *t[5:7], stream=0)
    pages = Tensor(48, device=1)
    pages.shape = (1, 1)
    assert hs.make_pages(pages, 1, 1).block_table == 48
    assert [name for name, _ in lib.calls] == ["hs_decode_step", "hs_full_attn_index", "hs_sparse_attn_reuse"]
    for (_, args), n in zip(lib.calls, (8, 7, 7)):
        assert {16 * (i + 1) for i in range(n)} <= {a for a in args if isinstance(a, int)}


def test_quantised_entry_points_refuse_a_peers_tensors(lib):
    p = hs.make_params(1, 1, 1, 64, 1, 1, mode="token", block_size=1, k=1, window=0)
    here, there = Tensor(16), Tensor(32, device=1)
    kv = hs.make_kv_quant("int4", here, here, here, here)
    with pytest.raises(ValueError, match="current CUDA device"):
        hs.make_kv_quant("int4", here, there, here, here)
    with pytest.raises(ValueError, match="current CUDA device"):
        hs.hs_kv_quant_write(p, kv, None, here, there, stream=0)
    with pytest.raises(ValueError, match="current CUDA device"):
        hs.hs_kv_quant_read(p, kv, None, there, here, stream=0)
    with pytest.raises(ValueError, match="current CUDA device"):
        hs.hs_decode_step_quant(p, kv, None, hs.HS_DECODE_SPARSE, here, there, here, here, here, stream=0)
    with pytest.raises(ValueError, match="current CUDA device"):
        hs.hs_sparse_attn_reuse_quant(p, kv, None, there, here, here, here, here, stream=0)
    assert not lib.calls
