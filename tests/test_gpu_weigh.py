"""kvl_weigh against the plain 64-bit definition (tests/_kept.py)."""
from __future__ import annotations

import math

import pytest
import torch

import layer_wise_paged_gb300 as kvl
from tests import _kept as K
from tests import _quant as Q

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvl.build()
    kvl.lib()


def case(lens, new, heads=8, kv_heads=2, d=128, B=16, code="e4m3", dtype=BF, causal=True, window=0, gain=1.0, q_gain=1.0,
         begin=True, max_new=None):
    return dict(lens=lens, new=new, heads=heads, kv_heads=kv_heads, d=d, B=B, code=code, dtype=dtype, causal=causal,
                window=window, gain=gain, q_gain=q_gain, begin=begin, max_new=max_new)


CASES = {
    "one token, one held": case([1], [1]),
    "one token": case([777], [1], heads=32, kv_heads=8),
    "adding up": case([130, 20], [1, 2], begin=False),
    "one head each": case([130], [1], heads=4, kv_heads=4),
    "sixteen heads on one": case([95, 33], [1, 1], heads=16, kv_heads=1),
    "odd group": case([61, 200], [1, 2], heads=6, kv_heads=2),
    "more KV heads than are held": case([50], [1], heads=40, kv_heads=40),
    "ragged, empty ones among them": case([0, 1, 15, 16, 17, 300, 0, 64], [0, 1, 1, 1, 1, 1, 0, 0]),
    "rows of an empty sequence": case([0, 20], [3, 2]),
    "more rows than tokens": case([2, 40], [5, 3]),
    "more rows than tokens, all visible": case([2, 40], [5, 3], causal=False),
    "drafted": case([100, 9, 257, 64], [8, 3, 1, 5], kv_heads=4, heads=16, d=64, code="int8", dtype=HF),
    "page of 1": case([19, 5], [2, 1], B=1),
    "page of 5": case([43, 11], [4, 1], B=5),
    "page of 24": case([100, 49], [1, 30], B=24),
    "page of 64": case([100, 300], [5, 1], B=64, heads=32, kv_heads=4),
    "page of 256": case([700, 256], [1, 2], B=256, code="int8"),
    "head of 16": case([90], [2], d=16),
    "head of 80": case([90, 33], [2, 33], d=80, dtype=HF),
    "head of 256": case([90, 150], [1, 40], d=256),
    "window": case([300, 40], [1, 6], window=33),
    "window of 1": case([50], [7], window=1),
    "last rows": case([400], [32]),
    "chunk": case([200], [130]),
    "chunk, f16 int8": case([190], [150], code="int8", dtype=HF, heads=4),
    "chunk on a long prefix": case([1100], [70], heads=8, kv_heads=1),
    "chunks, ragged": case([70, 1, 0, 333, 129], [70, 1, 0, 100, 129], d=64),
    "chunk, all visible": case([150, 260], [150, 40], causal=False),
    "chunk, window": case([400], [180], window=100),
    "chunk, page of 64": case([321], [321], B=64, heads=4, kv_heads=4, d=64, code="int8"),
    "chunk, page of 40": case([321], [121], B=40, heads=4, kv_heads=2),
    "chunk, many heads": case([140], [40], heads=24, kv_heads=12),
    "chunk and tokens": case([500, 90, 31], [1, 90, 1]),
    "peaked": case([500], [3], gain=6.0, q_gain=6.0),
    "peaked chunk": case([300], [140], gain=6.0, q_gain=6.0, heads=4),
    "bound on rows known": case([100, 40], [2, 1], max_new=2),
}


def make(c, seed=5):
    cache = Q.make_cache(seed, 2, c["kv_heads"], c["d"], c["B"], c["lens"], code=c["code"], gain=c["gain"])
    g = torch.Generator().manual_seed(seed + 1)
    starts = torch.tensor([0] + c["new"]).cumsum(0).int()
    wide = (torch.randn((int(starts[-1]), c["heads"] + 3, c["d"]), generator=g) * c["q_gain"]).to(c["dtype"])
    q = wide[:, 1:1 + c["heads"]]
    lse = Q.attend(cache, 1, q, starts, range(len(c["lens"])), 1 / math.sqrt(c["d"]), c["causal"], c["window"])[1].float()
    mass = torch.rand((len(c["lens"]), max(c["lens"]) + 5), generator=g)
    return cache, wide, starts, lse, mass


def held_to(got, want, tol, c, mass):
    """Tokens within their tolerance; what lies past them, and sequences without rows, as they were."""
    got = got.cpu()
    for s, n in enumerate(c["lens"]):
        assert torch.equal(got[s, n:], mass[s, n:]), "wrote past a sequence"
        if c["new"][s] == 0:
            assert torch.equal(got[s], mass[s]), "wrote a sequence without rows"
            continue
        over = (got[s, :n].double() - want[s, :n]).abs() - tol[s, :n]
        assert over.numel() == 0 or float(over.max()) <= 0, f"sequence {s}: {float(over.max())} over"


def run(c, seed=5):
    cache, wide, starts, lse, mass = make(c, seed)
    want, tol = K.weigh(cache, 1, wide[:, 1:1 + c["heads"]], starts, range(len(c["lens"])), lse, mass, c["begin"],
                        1 / math.sqrt(c["d"]), c["causal"], c["window"])
    dev = Q.on_gpu(cache)
    args = dict(begin=c["begin"], causal=c["causal"], window=c["window"],
                max_new=max(c["new"]) if c["max_new"] is None else c["max_new"])
    q, st, z = wide.cuda()[:, 1:1 + c["heads"]], starts.cuda(), lse.cuda()
    # in place
    m = mass.cuda()
    assert dev.weigh(1, q, st, z, m, **args) is m
    held_to(m, want, tol, c, mass)
    # into another tensor, both of them parts of wider ones, without a bound on the rows
    base, into = torch.full((len(mass), mass.shape[1] + 3), 9.0, device="cuda"), torch.full((len(mass), mass.shape[1] + 7), 9.0, device="cuda")
    base[:, :-3], into[:, :-7] = mass.cuda(), mass.cuda()
    dev.weigh(1, q, st, z, base[:, :-3], out=into[:, :-7], **dict(args, max_new=0))
    held_to(into[:, :-7], want, tol, c, mass)
    assert torch.equal(base[:, :-3].cpu(), mass) and (into[:, -7:] == 9).all()
    assert dev.status() == (0, 0)


@pytest.mark.parametrize("name", CASES)
def test_against_the_definition(name):
    run(CASES[name])


def test_the_rows_give_one_each():
    """With attention's own lse every row and head gives its tokens 1 in all: a term is off by what its score and
    its lse are, 2 (d + 8) 2^-23 of scores below 16 in sum, and 300 terms are added up."""
    c = CASES["chunks, ragged"]
    cache, wide, starts, _, mass = make(c)
    dev = Q.on_gpu(cache)
    q, st = wide.cuda()[:, 1:1 + c["heads"]], starts.cuda()
    lse = torch.empty((wide.shape[0], c["heads"]), device="cuda")
    dev.attend(1, q, st, lse=lse)
    m = torch.zeros_like(mass).cuda()
    dev.weigh(1, q, st, lse, m, begin=True)
    got = m.double().sum(dim=1).cpu()
    want = torch.tensor([float(n * c["heads"]) for n in c["new"]], dtype=torch.float64)
    assert float(((got - want).abs() - 1e-3 * want).max()) <= 0


@pytest.mark.parametrize("name", ["one token", "drafted", "chunks, ragged", "chunk on a long prefix"])
def test_the_same_bits_every_time(name):
    c = CASES[name]
    cache, wide, starts, lse, mass = make(c)
    dev = Q.on_gpu(cache)
    q, st, z = wide.cuda()[:, 1:1 + c["heads"]], starts.cuda(), lse.cuda()
    first = dev.weigh(1, q, st, z, mass.cuda(), max_new=max(c["new"]))
    for _ in range(4):
        assert torch.equal(first, dev.weigh(1, q, st, z, mass.cuda(), max_new=max(c["new"])))


@pytest.mark.parametrize("new", [3, 60])
def test_infinite_and_nan_lse(new):
    """A row of an infinite lse gives nothing, one whose lse is NaN makes what it sees NaN, and what no row sees
    keeps its bits whatever the cache holds there."""
    c = case([100], [new], heads=4, kv_heads=1)
    cache, wide, starts, lse, mass = make(c)
    q, st = wide.cuda()[:, 1:5], starts.cuda()
    dev = Q.on_gpu(cache)
    some = lse.clone()
    some[0] = -math.inf
    some[1] = math.inf
    want, tol = K.weigh(cache, 1, wide[:, 1:5], starts, [0], some, mass, False, 1 / math.sqrt(128), True, 0)
    held_to(dev.weigh(1, q, st, some.cuda(), mass.cuda()), want, tol, c, mass)
    some[0, 1] = math.nan
    got = dev.weigh(1, q, st, some.cuda(), mass.cuda()).cpu()[0]
    past = 100 - new + 1  # row 0 sees tokens up to itself
    assert torch.isnan(got[:past]).all() and torch.isfinite(got[past:]).all()


@pytest.mark.parametrize("garbage", [math.inf, -math.inf, math.nan, 3e38])
@pytest.mark.parametrize("new", [3, 60])
def test_rows_of_an_infinite_lse_may_hold_anything(new, garbage):
    """What pads a batch: rows that give nothing, and that the rows beside them do not feel."""
    c = case([100], [new], heads=4, kv_heads=1)
    cache, wide, starts, lse, mass = make(c)
    lse[1, 1:3], lse[2] = -math.inf, math.inf
    want, tol = K.weigh(cache, 1, wide[:, 1:5], starts, [0], lse, mass, False, 1 / math.sqrt(128), True, 0)
    wide[1, 2:4], wide[2] = garbage, garbage
    dev = Q.on_gpu(cache)
    held_to(dev.weigh(1, wide.cuda()[:, 1:5], starts.cuda(), lse.cuda(), mass.cuda()), want, tol, c, mass)


@pytest.mark.parametrize("new", [3, 60])
def test_nan_codes_stay_with_their_token(new):
    """A NaN in a token that rows 0 and 1 do not see: with finite lse it reaches that token's mass alone."""
    c = case([100], [new], heads=4, kv_heads=1)
    cache, wide, starts, lse, mass = make(c)
    cache["codes"][1, 0, int(cache["tables"][0, 99 // 16]), 99 % 16, 0, 5] = 0x7F
    got = Q.on_gpu(cache).weigh(1, wide.cuda()[:, 1:5], starts.cuda(), lse.cuda(), mass.cuda()).cpu()[0]
    assert torch.isnan(got[99]) and torch.isfinite(got[:99]).all()


def test_sequences_longer_than_the_masses_and_bad_pages():
    c = case([100, 40], [1, 1])
    cache, wide, starts, lse, mass = make(c)
    dev = Q.on_gpu(cache)
    m = mass.cuda()[:, 3:63]  # (a part of rows with room for more)
    dev.weigh(1, wide.cuda()[:, 1:9], starts.cuda(), lse.cuda(), m)
    assert dev.status() == (kvl.KVL_ERANGE, 0)
    assert torch.equal(m[0].cpu(), mass[0, 3:63]) and not torch.equal(m[1, :40].cpu(), mass[1, 3:43])
    cache["tables"][1, 1] = -3
    dev = Q.on_gpu(cache)
    got = dev.weigh(1, wide.cuda()[:, 1:9], starts.cuda(), lse.cuda(), mass.cuda()).cpu()
    assert dev.status() == (kvl.KVL_ERANGE, 1)
    assert torch.equal(got[1, 16:32], mass[1, 16:32])  # the tokens of the page that is not there


def test_on_another_stream_and_in_a_graph():
    c = CASES["chunks, ragged"]
    cache, wide, starts, lse, mass = make(c)
    dev = Q.on_gpu(cache)
    q, st, z = wide.cuda()[:, 1:1 + c["heads"]], starts.cuda(), lse.cuda()
    want = dev.weigh(1, q, st, z, mass.cuda(), begin=True)
    m, into = mass.cuda(), mass.cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    dev.weigh(1, q, st, z, m, begin=True, stream=side)
    side.synchronize()
    assert torch.equal(m, want)
    m = mass.cuda()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dev.weigh(1, q, st, z, m, out=into, begin=True)
    for _ in range(3):
        into.copy_(mass)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(into, want)
