"""Calls of several host threads on one stream, without a GPU: the launches of a call that pass data through memory of
the stream are not mixed with another's."""
from __future__ import annotations

import threading
import time
from types import SimpleNamespace

import pytest
import torch

from layer_wise_paged_gb300 import cache as C


class Launches:
    """Stands for the library: a call takes a while, in which other threads run, and notes who came between."""

    def __init__(self):
        self.inside, self.mixed, self.memory = 0, 0, []

    def __call__(self, *args):
        self.inside += 1
        self.mixed += self.inside > 1
        time.sleep(0.005)
        self.mixed += self.inside > 1
        self.inside -= 1
        return 0


class Memory(C.QuantCache):
    """A cache without tensors: what a call needs of one before it reaches the library."""

    def __init__(self, lib):
        self._lib, self._index, self._cache, self._report, self._scale = lib, 0, None, None, 0.125
        self._order = threading.Lock()
        self._sizes, self._ws_bytes, self.n_kv_heads, self.head_dim, self.n_slots = {}, 0, 2, 64, 4
        self._args = SimpleNamespace(attn=None, shared=SimpleNamespace(), weighing=SimpleNamespace(), weighing_q=None)

    def _seqs(self, c, starts, slots, n_rows):
        return SimpleNamespace(n_seq=2)

    def _attention(self, *args):
        return "out", None

    def _mass(self, t, name):
        return 0, 8

    def _scratch(self, n, st):
        return 0, None


@pytest.mark.parametrize("name", ["attend_shared", "weigh"])
def test_calls_of_two_threads_are_made_one_after_the_other(monkeypatch, name):
    monkeypatch.setattr(C, "_stream", lambda stream, device: 7)
    for f in ("_rows", "_flat", "_ints"):
        monkeypatch.setattr(C, f, lambda *args: 0)
    launches = Launches()
    cache = Memory(SimpleNamespace(kvl_attend_shared=launches, kvl_attend_shared_parts_bytes=lambda *a: 64,
                                   kvl_weigh=launches, kvl_weigh_workspace_bytes=lambda *a: 64))
    q = SimpleNamespace(shape=(3, 8, 64), dtype=torch.bfloat16)
    t = SimpleNamespace(shape=(4, 8), data_ptr=lambda: 0)
    errors = []

    def calls():
        try:
            for _ in range(10):
                if name == "weigh":
                    cache.weigh(0, q, t, t, t)
                else:
                    cache.attend_shared(0, q, t, t, t, max_new=1)
        except Exception as e:  # noqa: BLE001 (a thread's own would be lost)
            errors.append(e)

    threads = [threading.Thread(target=calls) for _ in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not errors and launches.mixed == 0


def test_two_first_calls_on_a_stream_share_one_workspace(monkeypatch):
    """The first thread's would be freed, and given to other tensors, before its launch is made."""
    class Slow:
        def __enter__(self):
            time.sleep(0.02)

        def __exit__(self, *args):
            return False

    cache = Memory(SimpleNamespace())
    cache.device, cache._ws_bytes, cache._ws = "cpu", 1 << 15, {}
    monkeypatch.setattr(cache, "_on", lambda st: Slow(), raising=False)
    got = []
    threads = [threading.Thread(target=lambda: got.append(cache._workspace(cache._ws, 7, 0))) for _ in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert len(got) == 4 and len({ws[1] for ws in got}) == 1 and cache._ws[7] is got[0]
    assert cache._workspace(cache._ws, 7, 5)[0] == 5 and cache._workspace(cache._ws, 8, 0) is not got[0]
