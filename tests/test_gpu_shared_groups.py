"""kvl_attend_shared over several groups: of many rows (the tensor-memory kernel), of few, of very unequal sizes, more of
them and of their sequences than the kernels hold at a time."""
from __future__ import annotations

import math

import pytest
import torch

import layer_wise_paged_gb300 as kvl
from tests import _quant as Q
from tests.test_gpu_attend import near
from tests.test_gpu_shared import HF, call, case, check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvl.build()
    kvl.lib()


def groups_of(sizes):
    return [sum(sizes[:g]) for g in range(len(sizes) + 1)]


def of_groups(sizes, shared, own=3, new=1, **k):
    """Group g: sizes[g] sequences that share shared[g] tokens and hold new + 0 .. own more."""
    lens = [P + new + (7 * i) % (own + 1) for n, P in zip(sizes, shared) for i in range(n)]
    return case(groups_of(sizes), list(shared), lens, [new] * len(lens), **k)


# rows of a KV head (sequences x new x heads / kv_heads) are more than 40 a group on average: the tensor-memory kernel
MANY = {
    "two groups, one of two tiles": of_groups([70, 15], [48, 64]),
    "an empty group and one that shares nothing between": of_groups([70, 0, 5, 30], [48, 32, 0, 64]),
    "three tiles, one, two": of_groups([140, 9, 70], [32, 96, 16], heads=4, kv_heads=1),
    "exactly a tile, and one row more": of_groups([64, 65], [48, 16], heads=4, kv_heads=1),
    "inside a page": of_groups([13, 20], [37, 75], own=8),
    "inside a group of slots": of_groups([13, 20], [70, 131], own=50, B=64),
    "page of 1": of_groups([12, 12], [19, 7], B=1),
    "page of 5": of_groups([12, 13], [43, 40], B=5),
    "page of 24": of_groups([12, 13], [72, 50], B=24, heads=16, kv_heads=4),
    "page of 256, int8": of_groups([12, 13], [300, 256], B=256, code="int8", heads=4, kv_heads=1),
    "head of 16": of_groups([12, 13], [50, 64], d=16),
    "head of 80": of_groups([12, 13], [50, 64], d=80, dtype=HF),
    "head of 64, int8": of_groups([12, 13], [50, 64], d=64, code="int8", dtype=HF),
    "drafted": of_groups([5, 9], [96, 61], own=6, new=4, heads=16, kv_heads=2),
    "all visible": of_groups([5, 9], [96, 61], own=6, new=4, heads=16, kv_heads=2, causal=False),
    "peaked": of_groups([20, 15], [400, 90], gain=6.0, q_gain=6.0),
    "one head each": of_groups([45, 50], [64, 30], heads=2, kv_heads=2),
    "odd group of heads": of_groups([20, 31], [64, 30], heads=6),
}
# fewer
FEW = {
    "one large group among single sequences": of_groups([96] + [1] * 60, [160] + [16 + i for i in range(60)], heads=4, kv_heads=1),
    "a group of one, and of forty": of_groups([1, 40, 1, 1, 1], [300, 64, 20, 33, 16], heads=4, kv_heads=1, d=64),
    "more groups than a CTA holds": of_groups([2] * 130, [16 + i % 20 for i in range(130)], heads=2, kv_heads=1, d=64),
    "as many groups as a CTA holds": of_groups([2] * 128, [16 + i % 20 for i in range(128)], heads=2, kv_heads=1, d=64),
    "several sequences a thread": of_groups([3] * 150, [9 + i % 13 for i in range(150)], heads=2, kv_heads=1, d=16, B=8),
    "heads of 256, several groups": of_groups([12, 0, 30], [50, 16, 64], d=256, heads=4, kv_heads=1),
}


@pytest.mark.parametrize("name", MANY)
def test_groups_of_many_rows(name):
    c = MANY[name]
    rows = sum(c["new"]) * (c["heads"] // c["kv_heads"])
    assert rows > 40 * len(c["shared"]) and max(c["new"]) * (c["heads"] // c["kv_heads"]) <= 40
    check(c)


@pytest.mark.parametrize("name", ["inside a page", "page of 5", "two groups, one of two tiles"])
def test_groups_of_many_rows_with_scales_far_apart(name):
    check(MANY[name], spread=True)


@pytest.mark.parametrize("name", FEW)
def test_groups_of_few_rows(name):
    check(FEW[name])


@pytest.mark.parametrize("new", [kvl.KVL_SHARED_ROWS, kvl.KVL_SHARED_ROWS + 1])
def test_as_many_rows_as_share_and_one_more(new):
    """The binding brings memory for parts exactly where the library wants it."""
    check(of_groups([3, 2], [64, 37], own=4, new=new, heads=2, kv_heads=2, d=64))


@pytest.mark.parametrize("groups", [130, 520])
def test_more_groups_of_many_rows_than_are_held(groups):
    """Past 128 groups an entry's group is looked for in memory, past 512 jobs are numbered over several batches."""
    check(of_groups([3] * groups, [5 + i % 23 for i in range(groups)], own=2, heads=16, kv_heads=1, d=16, B=8))


def test_slots_in_any_order_and_padding_rows():
    """Entries of both groups in mixed slots, rows behind the last entry left as they were."""
    c = of_groups([20, 15], [48, 64])
    cache, wide, starts = make(c)
    order = torch.randperm(20, generator=torch.Generator().manual_seed(1)).tolist() + [20 + int(x) for x in torch.randperm(15)]
    wide = torch.cat([wide, wide[:5]])
    dev = Q.on_gpu(cache)
    wout, lse = call(dev, c, wide.cuda(), starts.cuda(), slots=torch.tensor(order, dtype=torch.int32, device="cuda"))
    assert dev.status() == (0, 0)
    o, z, to, tz = Q.attend(cache, 1, wide[:35, 1:9], starts, order, 1 / math.sqrt(128), True, 0)
    near(wout[:35, 2:].cpu().double(), o, to, "out")
    near(lse[:35].cpu().double(), z, tz, "lse")
    assert (wout[35:] == 77.0).all() and (lse[35:] == 77.0).all()


@pytest.mark.parametrize("name", ["two groups, one of two tiles", "page of 1", "exactly a tile, and one row more"])
def test_sharing_changes_no_more_than_roundings(name):
    """attend and attend_shared of the same rows: each within its tolerance of the definition, so within twice that of
    each other."""
    c = MANY[name]
    cache, wide, starts = make(c)
    dev = Q.on_gpu(cache)
    q, st = wide.cuda(), starts.cuda()
    wout, lse = call(dev, c, q, st)
    plain_lse = torch.empty_like(lse)
    plain = dev.attend(1, q[:, 1:1 + c["heads"]], st, lse=plain_lse, max_new=max(c["new"]))
    assert dev.status() == (0, 0)
    _, _, to, tz = Q.attend(cache, 1, wide[:, 1:1 + c["heads"]], starts, range(len(c["lens"])), 1 / math.sqrt(c["d"]), True, 0)
    assert float(((wout[:, 2:].double() - plain.double()).abs().cpu() - 2 * to).max()) <= 0
    assert float(((lse.double() - plain_lse.double()).abs().cpu() - 2 * tz).max()) <= 0


@pytest.mark.parametrize("name", ["two groups, one of two tiles", "three tiles, one, two"])
def test_the_same_bits_every_time(name):
    c = MANY[name]
    cache, wide, starts = make(c)
    dev = Q.on_gpu(cache)
    first = call(dev, c, wide.cuda(), starts.cuda())
    for _ in range(4):
        again = call(dev, c, wide.cuda(), starts.cuda())
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_nan_in_tokens_behind_the_shared_ones():
    """Where the shared tokens end inside a page: its later slots, one sequence's own, hold NaN for that sequence alone."""
    c = of_groups([20], [37], own=8, heads=4, kv_heads=1)  # (sequence 0 holds 38 tokens)
    cache, wide, starts = make(c)
    # each sequence its own copy of the page that holds token 37, all of whose slots hold numbers
    page, other = int(cache["tables"][0, 2]), int(cache["tables"][0, 0])
    cache["codes"][:, :, page, 5:] = cache["codes"][:, :, other, 5:]
    used = set(cache["tables"][cache["tables"] >= 0].tolist())
    for s, b in zip(range(1, 20), [b for b in range(len(cache["refs"])) if b not in used], strict=False):
        cache["tables"][s, 2] = b
        cache["codes"][:, :, b], cache["scales"][:, :, b] = cache["codes"][:, :, page], cache["scales"][:, :, page]
    cache["codes"][1, :, page, 37 % 16, :, 3] = 0x7F
    dev = Q.on_gpu(cache)
    wout, lse = call(dev, c, wide.cuda(), starts.cuda())
    assert dev.status() == (0, 0)
    assert torch.isnan(lse[0]).all() and torch.isfinite(lse[1:]).all() and torch.isfinite(wout[1:, 2:].float()).all()


# ---- what is left out ----------------------------------------------------------------------------------------------

def left_or_right(c, cache, wide, starts, entries, wout, lse):
    """Every row of `entries` was written as the definition has it or not at all; all others not at all."""
    zero = torch.zeros(2, dtype=torch.int32)
    rows = torch.zeros(wide.shape[0], dtype=torch.bool)
    out, z = wout.cpu(), lse.cpu()
    for i in entries:
        a, b = int(starts[i]), int(starts[i + 1])
        rows[a:b] = True
        if (out[a:b, 2:] == 77.0).all() and (z[a:b] == 77.0).all():
            continue
        zero[1] = b - a
        o, y, to, ty = Q.attend(cache, 1, wide[a:b, 1:1 + c["heads"]], zero, [i], 1 / math.sqrt(c["d"]), c["causal"], 0)
        near(out[a:b, 2:].double(), o, to, f"out of entry {i}")
        near(z[a:b].double(), y, ty, f"lse of entry {i}")
    assert (out[~rows] == 77.0).all() and (z[~rows] == 77.0).all() and (out[:, :2] == 77.0).all()


def test_more_jobs_than_there_is_room_for_give_nothing_stale():
    """The same sequences named by several groups are more jobs than parts have room for: no row gets what a call before
    left there."""
    n, times = 1200, 20
    c = of_groups([n], [48], heads=4, kv_heads=1, d=16)
    cache, wide, starts = make(c)
    dev = Q.on_gpu(cache)
    for k in range(2):
        call(dev, c, wide.roll(k + 1, 0).cuda(), starts.cuda(), groups=[0] + [n] * (2 * times - 1), shared=[48] * (2 * times - 1))
        assert dev.status() == (0, 0)
        wout, lse = call(dev, c, wide.cuda(), starts.cuda(), groups=[0, n] * times, shared=[48] * (2 * times - 1))
        assert dev.status() == (kvl.KVL_EINVAL, 1)
        assert (wout == 77.0).all() and (lse == 77.0).all()
        dev.reset_status()


@pytest.mark.parametrize("n,times", [(130, 2), (200, 3), (8, 2)])
def test_groups_out_of_order_give_nothing_wrong(n, times):
    """The same sequences named by several groups: a descending range is reported, and no row gets another's result, nor
    one of a call before."""
    c = of_groups([n], [48], heads=4, kv_heads=1)
    cache, wide, starts = make(c)
    dev = Q.on_gpu(cache)
    groups, shared = [0, n] * times, [48] * (2 * times - 1)
    for k in range(3):  # (the calls before leave their parts in the scratch memory)
        call(dev, c, wide.roll(k + 1, 0).cuda(), starts.cuda(), groups=groups_of([n] + [0] * (2 * times - 2)), shared=shared)
        assert dev.status() == (0, 0)
        wout, lse = call(dev, c, wide.cuda(), starts.cuda(), groups=groups, shared=shared)
        code, detail = dev.status()
        assert code == kvl.KVL_EINVAL and detail == 1
        left_or_right(c, cache, wide, starts, range(n), wout, lse)
        dev.reset_status()


@pytest.mark.parametrize("heads", [4, 1])
def test_rows_out_of_order_give_nothing_wrong(heads):
    """Two groups whose rows lie the other way round, with a bad entry between: it is reported, and no row gets another's
    result."""
    new, a, b = 10, 12, 13
    c = of_groups([a, 1, b], [48, 16, 64], own=5, new=new, heads=heads, kv_heads=1)
    cache, wide, _ = make(c)
    wide = wide[:(a + b) * new]
    starts = torch.tensor([b * new + new * i for i in range(a + 1)] + [new * i for i in range(b + 1)], dtype=torch.int32)
    dev = Q.on_gpu(cache)
    for _ in range(3):
        wout, lse = call(dev, c, wide.cuda(), starts.cuda())
        code, detail = dev.status()
        assert code == kvl.KVL_EINVAL
        left_or_right(c, cache, wide, starts, [i for i in range(a + 1 + b) if i != a], wout, lse)
