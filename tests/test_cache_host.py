"""The torch side of the 8-bit cache without a GPU: what it asks of torch, and its own refusals."""
from __future__ import annotations

import importlib.util
from types import SimpleNamespace

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
