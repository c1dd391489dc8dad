"""kvl_attend_shared against the plain 64-bit definition, which knows of no sharing, at the sizes, groups and contents
where attention over a shared prefix can go wrong."""
from __future__ import annotations

import math

import pytest
import torch

import layer_wise_paged_gb300 as kvl
from tests import _kept as K
from tests import _quant as Q
from tests.test_gpu_attend import near

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvl.build()
    kvl.lib()


def case(groups, shared, lens, new, heads=8, kv_heads=2, d=128, B=16, code="e4m3", dtype=BF, causal=True, window=0,
         gain=1.0, q_gain=1.0, max_new=None):
    return dict(groups=groups, shared=shared, lens=lens, new=new, heads=heads, kv_heads=kv_heads, d=d, B=B, code=code,
                dtype=dtype, causal=causal, window=window, gain=gain, q_gain=q_gain, max_new=max_new)


CASES = {
    "two of one prompt": case([0, 2], [32], [40, 35], [1, 1]),
    "shared tokens and the fresh one": case([0, 3], [48], [49, 49, 49], [1, 1, 1]),
    "one shared page": case([0, 2], [16], [17, 30], [1, 2]),
    "nothing shared": case([0, 2], [0], [40, 35], [1, 1]),
    "no groups": case([0], [], [40, 35], [1, 1]),
    "a group of one": case([0, 1], [32], [40], [1]),
    "outside all groups": case([1, 3], [32], [60, 40, 50, 33], [1, 1, 2, 1]),
    "groups, an empty one among them": case([0, 2, 2, 5], [32, 48, 64], [40, 41, 70, 80, 65], [1, 1, 1, 1, 1]),
    "sequences without fresh rows": case([0, 3], [32], [40, 40, 45], [1, 0, 1]),
    "odd group of heads": case([0, 4], [96], [100, 97, 130, 111], [1, 1, 1, 1], heads=6),
    "sixteen heads on one": case([0, 3], [80], [81, 95, 90], [1, 1, 1], heads=16, kv_heads=1),
    "one head each": case([0, 5], [64], [70, 66, 65, 80, 90], [1] * 5, heads=4, kv_heads=4),
    "drafted": case([0, 3, 5], [96, 32], [110, 100, 108, 40, 50], [4, 3, 1, 5, 2], heads=16, kv_heads=4, d=64, code="int8",
                    dtype=HF),
    "inside a page": case([0, 2], [37], [48, 48], [1, 3]),
    "inside a group of slots": case([0, 2], [70], [128, 128], [2, 1], B=64),
    "page of 1": case([0, 3], [19], [22, 21, 20], [1, 1, 1], B=1),
    "page of 5": case([0, 2], [40], [43, 51], [1, 2], B=5),
    "page of 24": case([0, 2], [72], [100, 80], [1, 2], B=24),
    "page of 64": case([0, 3], [320], [330, 400, 321], [1, 1, 1], B=64, heads=32, kv_heads=4),
    "head of 16": case([0, 2], [32], [40, 35], [1, 1], d=16),
    "head of 80": case([0, 2], [32], [40, 35], [1, 3], d=80, dtype=HF),
    "head of 144": case([0, 2], [32], [40, 35], [1, 1], d=144),
    "head of 256": case([0, 2], [32], [40, 35], [1, 2], d=256),
    "many sequences": case([0, 40], [256], [257 + 3 * i for i in range(40)], [1] * 40),
    "seventy sequences, int8": case([0, 70], [512], [513 + i % 40 for i in range(70)], [1] * 70, heads=4, kv_heads=1, d=64,
                                    code="int8", dtype=HF),
    "long prefix": case([0, 3], [2480], [2500, 2490, 2481], [1, 1, 1], heads=4, kv_heads=1),
    "long prefix, many rows": case([0, 9], [1600], [1601 + 5 * i for i in range(9)], [1 + i % 3 for i in range(9)], heads=8,
                                   kv_heads=1),
    "all visible": case([0, 2], [32], [40, 45], [3, 2], causal=False),
    "peaked": case([0, 3], [400], [420, 410, 401], [1, 2, 1], gain=6.0, q_gain=6.0),
    "tiny values": case([0, 2], [96], [100, 99], [2, 1], gain=1e-6),
    "a window": case([0, 2], [32], [80, 50], [1, 2], window=20),
    "prompts behind a prefix": case([0, 2], [64], [140, 160], [70, 90]),
    "no bound on rows": case([0, 2], [64], [70, 80], [1, 2], max_new=0),
}


def make(c, seed=5, spread=False):
    cache = Q.make_cache(seed, 2, c["kv_heads"], c["d"], c["B"], c["lens"], code=c["code"], gain=c["gain"])
    if spread:  # scales of the pages far apart
        f = torch.exp2(torch.linspace(-12, 9, cache["scales"].shape[2])).float()
        cache["scales"] *= f[None, None, torch.randperm(len(f), generator=torch.Generator().manual_seed(2)), None]
    K.fork(cache, c["groups"], c["shared"])
    g = torch.Generator().manual_seed(seed + 1)
    starts = torch.tensor([0] + c["new"]).cumsum(0).int()
    # q and out are parts of wider rows
    wide = (torch.randn((int(starts[-1]), c["heads"] + 3, c["d"]), generator=g) * c["q_gain"]).to(c["dtype"])
    return cache, wide, starts


def call(dev, c, wide, starts, groups=None, shared=None, **more):
    T = wide.shape[0]
    wout = torch.full((T, c["heads"] + 2, c["d"]), 77.0, dtype=c["dtype"], device="cuda")
    lse = torch.full((T, c["heads"]), 77.0, device="cuda")
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (groups or c["groups"], shared or c["shared"])]
    args = dict(out=wout[:, 2:], lse=lse, causal=c["causal"], window=c["window"],
                max_new=max(c["new"]) if c["max_new"] is None else c["max_new"])
    args.update(more)
    dev.attend_shared(1, wide[:, 1:1 + c["heads"]], starts, *ints, **args)
    return wout, lse


def check(c, seed=5, spread=False):
    cache, wide, starts = make(c, seed, spread)
    dev = Q.on_gpu(cache)
    wout, lse = call(dev, c, wide.cuda(), starts.cuda())
    assert dev.status() == (0, 0)
    assert (wout[:, :2] == 77.0).all(), "wrote outside its rows"
    o, z, to, tz = Q.attend(cache, 1, wide[:, 1:1 + c["heads"]], starts, range(len(c["lens"])), 1 / math.sqrt(c["d"]),
                            c["causal"], c["window"])
    near(wout[:, 2:].cpu().double(), o, to, "out")
    near(lse.cpu().double(), z, tz, "lse")


@pytest.mark.parametrize("name", CASES)
def test_against_the_definition(name):
    check(CASES[name])


@pytest.mark.parametrize("name", ["drafted", "many sequences", "long prefix", "page of 5"])
def test_scales_far_apart(name):
    check(CASES[name], spread=True)


@pytest.mark.parametrize("name", ["many sequences", "long prefix, many rows", "drafted"])
def test_the_same_bits_every_time(name):
    c = CASES[name]
    cache, wide, starts = make(c)
    dev = Q.on_gpu(cache)
    first = call(dev, c, wide.cuda(), starts.cuda())
    for _ in range(4):
        again = call(dev, c, wide.cuda(), starts.cuda())
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_what_rows_do_not_see_is_no_part_of_them():
    """NaN codes and infinities past each sequence's end and in pages nobody holds are everywhere already (make_cache);
    NaN in one sequence's own tokens reaches its rows alone."""
    c = CASES["two of one prompt"]
    cache, wide, starts = make(c)
    cache["codes"][1, 1, int(cache["tables"][1, 2]), 1, :, 3] = 0x7F  # token 33 of sequence 1
    dev = Q.on_gpu(cache)
    wout, _ = call(dev, c, wide.cuda(), starts.cuda())
    out = wout[:, 2:].cpu()
    assert torch.isfinite(out[0]).all()
    assert torch.isnan(out[1, :, 3]).all() and torch.isfinite(out[1, :, :3]).all() and torch.isfinite(out[1, :, 4:]).all()


def test_slots_in_any_order():
    c = CASES["groups, an empty one among them"]
    cache, wide, starts = make(c)
    order = [3, 4, 2, 1, 0]  # batch entries: group 0 is slots 3, 4, 2 (of 64 tokens), group 1 slots 1, 0
    dev = Q.on_gpu(cache)
    slots = torch.tensor(order, dtype=torch.int32, device="cuda")
    wout, lse = call(dev, c, wide.cuda(), starts.cuda(), groups=[0, 3, 5], shared=[64, 32], slots=slots)
    assert dev.status() == (0, 0)
    o, z, to, tz = Q.attend(cache, 1, wide[:, 1:1 + c["heads"]], starts, order, 1 / math.sqrt(c["d"]), True, 0)
    near(wout[:, 2:].cpu().double(), o, to, "out")
    near(lse.cpu().double(), z, tz, "lse")


def test_entries_that_do_not_see_all_shared_tokens_are_left_out():
    c = CASES["two of one prompt"]
    cache, wide, starts = make(c)
    dev = Q.on_gpu(cache)
    wout, lse = call(dev, c, wide.cuda(), starts.cuda(), shared=[35])  # of 35 tokens sequence 1's fresh one is the last
    code, detail = dev.status()
    assert (code, detail) == (kvl.KVL_ERANGE, 1)
    assert (wout[1] == 77).all() and (lse[1] == 77).all()
    o, z, to, tz = Q.attend(cache, 1, wide[:, 1:9], starts, range(2), 1 / math.sqrt(128), True, 0)
    near(wout[:1, 2:].cpu().double(), o[:1], to[:1], "out")


@pytest.mark.parametrize("groups,shared,code", [([0, 3], [32], "EINVAL"), ([-1, 2], [32], "EINVAL"), ([2, 0], [32], "EINVAL"),
                                                ([0, 2], [-5], "EINVAL"), ([0, 2], [41], "ERANGE")])
def test_bad_groups(groups, shared, code):
    """They are reported, nothing outside the rows is written, and the call ends."""
    c = CASES["two of one prompt"]
    cache, wide, starts = make(c)
    dev = Q.on_gpu(cache)
    wout, _ = call(dev, c, wide.cuda(), starts.cuda(), groups=groups, shared=shared)
    assert dev.status()[0] == getattr(kvl, "KVL_" + code)
    assert (wout[:, :2] == 77.0).all()


def test_groups_out_of_order_stay_within_their_memory():
    """The same sequences named by two groups: more work than there is room for; it is reported and the call ends."""
    c = CASES["seventy sequences, int8"]
    cache, wide, starts = make(c)
    dev = Q.on_gpu(cache)
    wout, _ = call(dev, c, wide.cuda(), starts.cuda(), groups=[0, 70, 0, 70, 0, 70], shared=[512] * 5)
    assert dev.status()[0] == kvl.KVL_EINVAL
    assert (wout[:, :2] == 77.0).all()


def test_pages_out_of_range_are_reported():
    c = CASES["two of one prompt"]
    cache, wide, starts = make(c)
    cache["tables"][:, 1] = cache["codes"].shape[2]
    dev = Q.on_gpu(cache)
    call(dev, c, wide.cuda(), starts.cuda())
    assert dev.status()[0] == kvl.KVL_ERANGE


def test_on_another_stream_and_in_a_graph():
    c = CASES["long prefix, many rows"]
    cache, wide, starts = make(c)
    dev = Q.on_gpu(cache)
    wide, starts = wide.cuda(), starts.cuda()
    want = call(dev, c, wide, starts)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    groups, shared = (torch.tensor(c[k], dtype=torch.int32, device="cuda") for k in ("groups", "shared"))
    lse = torch.zeros_like(want[1])
    torch.cuda.synchronize()
    q = wide[:, 1:1 + c["heads"]]
    out = dev.attend_shared(1, q, starts, groups, shared, lse=lse, max_new=3, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0][:, 2:]) and torch.equal(lse, want[1])
    graph = torch.cuda.CUDAGraph()
    held = torch.zeros_like(out)
    with torch.cuda.graph(graph, stream=side):
        dev.attend_shared(1, q, starts, groups, shared, out=held, lse=lse, max_new=3)
    for _ in range(3):
        held.zero_()
        lse.zero_()
        torch.cuda.synchronize()
        graph.replay()
        dev.attend_shared(1, q, starts, groups, shared, max_new=3)  # beside it, on the current stream
        torch.cuda.synchronize()
        assert torch.equal(held, out) and torch.equal(lse, want[1])
    assert dev.status() == (0, 0)


def test_no_work():
    c = CASES["two of one prompt"]
    cache, wide, _ = make(c)
    dev = Q.on_gpu(cache)
    none = torch.zeros((0, 8, 128), dtype=BF, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = dev.attend_shared(0, none, zero, zero, zero[:0])
    assert out.shape == (0, 8, 128) and dev.status() == (0, 0)
