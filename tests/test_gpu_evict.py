"""kvl_pages_evict and kvl_tokens_move against the plain definitions (tests/_kept.py): everything exactly."""
from __future__ import annotations

import math

import pytest
import torch

import layer_wise_paged_gb300 as kvl
from tests import _kept as K
from tests import _quant as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvl.build()
    kvl.lib()


def case(lens, keep, first=0, recent=0, H=2, d=64, B=16, code="e4m3", L=2, mass="random", spare=None):
    return dict(lens=lens, keep=keep, first=first, recent=recent, H=H, d=d, B=B, code=code, L=L, mass=mass, spare=spare)


CASES = {
    "half": case([100], [50]),
    "first and recent": case([100, 60, 33], [40, 30, 20], first=4, recent=8),
    "whole pages stay": case([200], [100], first=40, recent=20),
    "all fits": case([30, 100, 0], [30, 120, 5]),
    "one token stays": case([70, 17], [1, 1]),
    "nothing stays": case([70, 17], [0, 8]),
    "one goes": case([65, 48, 33], [64, 47, 32], first=2, recent=5),
    "fewer than the first": case([100], [10], first=40, recent=20),
    "fewer than first and recent": case([100], [30], first=20, recent=20),
    "first alone": case([100], [48], first=48),
    "recent alone": case([100], [37], recent=37),
    "no masses": case([100, 50], [40, 49], first=4, recent=10, mass=None),
    "equal masses": case([100, 50], [40, 49], first=4, recent=10, mass="equal"),
    "few different masses": case([300], [150], first=4, recent=10, mass="few"),
    "negative, NaN and infinite masses": case([300], [150], first=4, recent=10, mass="odd"),
    "page of 1": case([40, 9], [13, 5], first=3, recent=2, B=1),
    "page of 5": case([43, 11], [20, 6], first=6, recent=2, B=5),
    "page of 64, int8": case([300, 70], [130, 64], first=70, recent=3, B=64, code="int8"),
    "page of 200": case([700], [333], first=5, B=200, H=1, d=16, L=1),
    "narrow rows": case([100], [37], H=1, d=16, first=3),
    "rows of 48 bytes": case([100], [37], H=3, d=16, first=3),
    "wide rows": case([60], [37], H=8, d=256, L=1, code="int8"),
    "rows of 720 bytes": case([60], [37], H=9, d=80, L=1),
    "long": case([5000, 4097], [3000, 17], first=4, recent=64, H=1, d=16, L=1),
    "longer than a cluster's registers": case([140000, 70001], [9000, 40], first=4, recent=1000, H=1, d=16, L=1, B=64),
    "longer than a cluster's registers, few masses": case([70001], [20000], first=4, recent=70, H=1, d=16, L=1, B=40, mass="few"),
    "many sequences": case([20 + 7 * i for i in range(60)], [10 + 5 * (i % 30) for i in range(60)], first=2, recent=3, H=1,
                           d=16, L=1),
    "more sequences than a CTA's threads": case([5 + i % 29 for i in range(1100)], [3 + i % 17 for i in range(1100)], first=1,
                                                recent=1, H=1, d=16, L=1, B=8),
}


def make(c, seed=7):
    need = sum(-(-k // c["B"]) for n, k in zip(c["lens"], c["keep"]) if n > k)
    cache = Q.make_cache(seed, c["L"], c["H"], c["d"], c["B"], c["lens"], spare=need + 2 if c["spare"] is None else c["spare"],
                         code=c["code"], poison=False)
    # pages' scales differ, so that what meets in one is turned to a common one
    g = torch.Generator().manual_seed(seed + 1)
    cache["scales"] *= torch.exp2(torch.randint(-2, 3, cache["scales"].shape, generator=g).float())
    if c["code"] == "e4m3":
        cache["codes"][0, 0, :, :, 0, :3] = torch.tensor([0x7F, 0xFF, 0x80], dtype=torch.uint8)  # NaN, -NaN, -0
    shape = (len(c["lens"]), max(c["lens"]) + 3)
    x = torch.randn(shape, generator=g).exp()
    if c["mass"] is None:
        return cache, None
    if c["mass"] == "equal":
        x[:] = 0.25
    elif c["mass"] == "few":
        x = torch.randint(0, 4, shape, generator=g).float() * 0.5
    elif c["mass"] == "odd":
        x = torch.randn(shape, generator=g)
        kind = torch.randint(0, 12, shape, generator=g)
        for i, v in enumerate((math.nan, -math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-40)):
            x[kind == i] = v
    return cache, x


def same(dev, want, m, mass):
    assert torch.equal(dev.lens.cpu(), want["lens"])
    assert torch.equal(dev.tables.cpu(), want["tables"])
    assert torch.equal(dev.refs.cpu(), want["refs"])
    if mass is not None:
        assert torch.equal(m.cpu().view(torch.int32), mass.view(torch.int32))
    assert torch.equal(dev.scales.cpu(), want["scales"])
    got, codes = dev.codes.cpu(), want["codes"]
    if want["code"] == "e4m3":  # (a NaN that is turned is a NaN, of either sign)
        nan = (codes & 0x7F) == 0x7F
        assert torch.equal((got & 0x7F) == 0x7F, nan)
        got, codes = torch.where(nan, 0, got), torch.where(nan, 0, codes)
    assert torch.equal(got, codes)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(c, slots=None, cache=None, mass=None, stream=None):
    if cache is None:
        cache, mass = make(c)
    dev = Q.on_gpu(cache)
    m = None if mass is None else mass.cuda()
    slots = list(range(len(c["lens"]))) if slots is None else slots
    s, k = ints(slots), ints(c["keep"])
    torch.cuda.synchronize()
    dev.evict(s, k, m, first=c["first"], recent=c["recent"], stream=stream)
    dev.move_tokens(stream=stream)
    if stream is not None:
        stream.synchronize()
    assert dev.status() == (0, 0)
    K.evict(cache, slots, c["keep"], mass, c["first"], c["recent"])
    same(dev, cache, m, mass)
    return dev


@pytest.mark.parametrize("name", CASES)
def test_against_the_definition(name):
    run(CASES[name])


def test_some_slots_in_any_order():
    c = case([100, 60, 33, 80], [40, 30, 20], first=4, recent=8)
    run(c, slots=[3, 0, 2])


def test_shared_pages_are_not_written():
    """Two sequences of one prompt, shortened by different masses: a page the other still names keeps its bytes."""
    c = case([100, 100, 100], [40, 50, 200], first=20, recent=8)
    cache, mass = make(c)
    for s in (1, 2):
        cache["refs"][cache["tables"][s, :7].long()] = 0
        cache["tables"][s, :7] = cache["tables"][0, :7]
    cache["refs"][cache["tables"][0, :7].long()] = 3
    before = cache["codes"].clone()
    dev = run(c, cache=cache, mass=mass)
    pages = dev.tables[2, :7].long().cpu()
    assert torch.equal(dev.codes.cpu()[:, :, pages], before[:, :, pages])
    assert dev.refs.cpu()[pages].tolist() == [3] + [1] * 6


@pytest.mark.parametrize("spare,fits", [(3, True), (2, False)])
def test_too_few_free_pages(spare, fits):
    c = case([100, 33], [40, 33], spare=spare)
    if fits:
        run(c)
        return
    cache, mass = make(c)
    dev = Q.on_gpu(cache)
    m = mass.cuda()
    dev.evict(ints([0, 1]), ints(c["keep"]), m)
    dev.move_tokens()
    assert dev.status() == (kvl.KVL_ERANGE, 2)
    same(dev, cache, m, mass)


@pytest.mark.parametrize("slots,keep,code,detail", [([0, 0], [5, 5], "EDUP", None), ([0, 2], [5, 5], "EINVAL", 1),
                                                    ([-1, 1], [5, 5], "EINVAL", 0), ([0, 1], [5, -1], "EINVAL", 1)])
def test_bad_entries_change_nothing(slots, keep, code, detail):
    c = case([100, 60], keep)
    cache, mass = make(c)
    dev = Q.on_gpu(cache)
    m = mass.cuda()
    dev.evict(ints(slots), ints(keep), m)
    dev.move_tokens()
    got = dev.status()
    assert got[0] == getattr(kvl, "KVL_" + code) and detail in (None, got[1])
    same(dev, cache, m, mass)


def test_a_sequence_longer_than_its_masses():
    c = case([100, 60], [50, 50])
    cache, mass = make(c)
    dev = Q.on_gpu(cache)
    m = mass[:, :80].contiguous()
    held = m.cuda()
    dev.evict(ints([0, 1]), ints([50, 50]), held)
    assert dev.status() == (kvl.KVL_ERANGE, 0)
    same(dev, cache, held, m)


def test_pages_out_of_range_are_reported():
    c = case([100], [90])
    cache, mass = make(c)
    cache["tables"][0, 3] = cache["codes"].shape[2] + 5
    dev = Q.on_gpu(cache)
    dev.evict(ints([0]), ints([90]), mass.cuda())
    dev.move_tokens()
    assert dev.status() == (kvl.KVL_ERANGE, 0)
    assert dev.lens.tolist() == [90]


def test_nothing_to_move_before_an_eviction_and_no_entries():
    cache, mass = make(case([100], [50]))
    dev = Q.on_gpu(cache)
    dev.move_tokens()
    dev.evict(ints([])[:0], ints([])[:0], mass.cuda())
    dev.move_tokens()
    assert dev.status() == (0, 0)
    same(dev, cache, mass.cuda(), mass)


def test_nothing_to_move_before_a_captured_eviction_runs():
    cache, mass = make(case([100], [50]))
    dev = Q.on_gpu(cache)
    m, slots, keep = mass.cuda(), ints([0]), ints([50])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dev.evict(slots, keep, m)
    dev.move_tokens()
    assert dev.status() == (0, 0)
    same(dev, cache, m, mass)


def test_again_and_again():
    """Evictions one after another, beside the pages that the ones before gave up."""
    cache, mass = make(case([200, 150], [120, 100]))
    dev = Q.on_gpu(cache)
    m = mass.cuda()
    for keep in ([120, 100], [90, 100], [33, 32], [5, 6]):
        dev.evict(ints([0, 1]), ints(keep), m, first=2, recent=3)
        dev.move_tokens()
        K.evict(cache, [0, 1], keep, mass, 2, 3)
        same(dev, cache, m, mass)
    assert dev.status() == (0, 0)


def test_on_another_stream_and_in_a_graph():
    run(CASES["first and recent"], stream=torch.cuda.Stream())
    c = CASES["first and recent"]
    cache, mass = make(c)
    dev = Q.on_gpu(cache)
    m, slots, keep = mass.cuda(), ints([0, 1, 2]), ints(c["keep"])
    state = {k: getattr(dev, k).clone() for k in ("tables", "lens", "refs", "codes", "scales")}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dev.evict(slots, keep, m, first=4, recent=8)
        dev.move_tokens()
    K.evict(cache, [0, 1, 2], c["keep"], out := mass.clone(), 4, 8)
    for _ in range(3):
        for k, v in state.items():
            getattr(dev, k).copy_(v)
        m.copy_(mass)
        graph.replay()
        same(dev, cache, m, out)
    assert dev.status() == (0, 0)
