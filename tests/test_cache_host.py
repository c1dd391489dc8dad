"""The torch side of the 8-bit cache without a GPU: what it asks of torch, and its own refusals."""
from __future__ import annotations

import importlib.util
from types import SimpleNamespace

import pytest
import torch

from layer_wise_paged_gb300 import cache as C


def test_imports_without_the_private_stream_query(monkeypatch):
    """A torch that lacks it gets the public query."""
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: SimpleNamespace(cuda_stream=77 + device))
    spec = importlib.util.spec_from_file_location("layer_wise_paged_gb300.cache_again", C.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    assert again._stream(None, 1) == 78 and again._stream(5, 1) == 5


def test_calls_on_another_device_are_refused(monkeypatch):
    """The library launches on the current device: tensors of another are refused before anything is
    launched, for the cache's calls and for rotary alike."""
    monkeypatch.setattr(C, "_several", True)
    monkeypatch.setattr(C, "_current_device", lambda: 1)
    monkeypatch.setattr(C, "_raw_stream", lambda device: 40 + device)
    assert C._stream(None, 1) == 41 and C._stream(7, 1) == 7 and C._stream(SimpleNamespace(cuda_stream=9), 1) == 9

    class Called(Exception):
        pass

    def launched(*args):
        raise Called

    held = C.QuantCache.__new__(C.QuantCache)
    held._index, held.pool_blocks = 0, 4
    held._report = held._pages = held._cache = None
    held._p = SimpleNamespace(pairs=None, n_pairs=None)
    held._lib = SimpleNamespace(kvl_pages_compact=launched, kvl_pages_copy=launched, kvl_report_reset=launched)
    for call in (held.compact, held.copy_pages, held.reset_status):
        for stream in (None, 7):
            with pytest.raises(ValueError, match="cuda:0"):
                call(stream=stream)
        held._index = 1
        with pytest.raises(Called):
            call()
        held._index = 0

    class Row(SimpleNamespace):
        shape, dtype, is_cuda = (3, 2, 16), torch.float32, True
        dim, stride = (lambda self: 3), (lambda self: (32, 16, 1))
        element_size, data_ptr, get_device = (lambda self: 4), (lambda self: 1 << 20), (lambda self: 0)

    positions = SimpleNamespace(dtype=torch.int32, is_cuda=True, shape=(3,), dim=lambda: 1, is_contiguous=lambda: True,
                                data_ptr=lambda: 1 << 20)
    monkeypatch.setattr(C, "_lib", lambda: SimpleNamespace(kvl_rotary=launched))
    with pytest.raises(ValueError, match="cuda:0"):
        C.rotary(SimpleNamespace(_ref=None), positions, [(Row(), Row())])
