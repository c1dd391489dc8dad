"""Refused evictions of sequences that a cluster of CTAs selects from: reported, and nothing is changed.

A refusal is found by the plan, which runs beside the selection: its CTAs have read each other's histograms by then."""
from __future__ import annotations

import pytest
import torch

import layer_wise_paged_gb300 as kvl
from tests import _kept as K
from tests import _quant as Q
from tests.test_gpu_evict import case, ints, make, same

pytestmark = pytest.mark.gpu

# room for more tokens a sequence than one CTA holds (8,192): clusters of 2 and of 8
SIZES = {"two CTAs": dict(lens=[9000, 8300, 12], keep=[1000, 8000, 20], B=16),
         "eight CTAs": dict(lens=[70001, 12], keep=[20000, 5], B=64)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvl.build()
    kvl.lib()


def sized(name, **k):
    z = dict(SIZES[name], **k)
    return case(z.pop("lens"), z.pop("keep"), first=4, recent=100, H=1, d=16, L=1, **z)


@pytest.mark.parametrize("mass", ["random", "few"])
@pytest.mark.parametrize("name", SIZES)
def test_too_few_free_pages(name, mass):
    c = sized(name, spare=3, mass=mass)
    cache, masses = make(c)
    dev = Q.on_gpu(cache)
    m, n = masses.cuda(), len(c["lens"])
    slots, keep = ints(list(range(n))), ints(c["keep"])
    for _ in range(20):
        dev.evict(slots, keep, m, first=4, recent=100)
    dev.move_tokens()
    assert dev.status() == (kvl.KVL_ERANGE, n)
    same(dev, cache, m, masses)


@pytest.mark.parametrize("slots,keep,code", [([0, 0], [1000, 1000], "EDUP"), ([0, 9], [1000, 5], "EINVAL"),
                                             ([0, 1], [1000, -1], "EINVAL")])
@pytest.mark.parametrize("name", SIZES)
def test_bad_entries(name, slots, keep, code):
    c = sized(name)
    cache, masses = make(c)
    dev = Q.on_gpu(cache)
    m = masses.cuda()
    dev.evict(ints(slots), ints(keep), m, first=4, recent=100)
    dev.move_tokens()
    assert dev.status()[0] == getattr(kvl, "KVL_" + code)
    same(dev, cache, m, masses)


def test_an_eviction_after_a_refused_one():
    """The same call once there are pages for it."""
    c = sized("two CTAs")
    cache, masses = make(c)
    dev = Q.on_gpu(cache)
    m, free = masses.cuda(), dev.refs == 0
    slots, keep = ints([0, 1, 2]), ints(c["keep"])
    dev.refs[free] = 1
    dev.evict(slots, keep, m, first=4, recent=100)
    assert dev.status() == (kvl.KVL_ERANGE, 3)
    dev.refs[free] = 0
    dev.reset_status()
    dev.evict(slots, keep, m, first=4, recent=100)
    dev.move_tokens()
    assert dev.status() == (0, 0)
    K.evict(cache, [0, 1, 2], c["keep"], masses, 4, 100)
    same(dev, cache, m, masses)
