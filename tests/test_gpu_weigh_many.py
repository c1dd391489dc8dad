"""kvl_weigh over many entries, and what gives nothing: rows of an infinite lse beside NaN codes, entries out of order."""
from __future__ import annotations

import math

import pytest
import torch

import layer_wise_paged_gb300 as kvl
from tests import _kept as K
from tests import _quant as Q
from tests.test_gpu_weigh import case, held_to, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvl.build()
    kvl.lib()


CASES = {
    "more entries than a CTA's threads": case([3 + i % 29 for i in range(600)], [1] * 600, heads=2, kv_heads=1, d=16, B=8),
    "more entries of many rows than are held": case([6 + i % 29 for i in range(600)], [5] * 600, heads=4, kv_heads=1, d=16, B=8),
    "a prompt's chunk among single tokens": case([500] + [40 + i for i in range(30)], [260] + [1] * 30, heads=4, kv_heads=1),
}


@pytest.mark.parametrize("name", CASES)
def test_many_entries(name):
    run(CASES[name])


@pytest.mark.parametrize("new,dead", [(3, [2]), (60, [59]), (60, [57, 58, 59]), (64, [63]), (200, [199])])
def test_a_nan_key_that_only_rows_of_an_infinite_lse_see(new, dead):
    """It gives nothing, as such rows do: the token's mass stays, and so does everyone else's."""
    c = case([300], [new], heads=4, kv_heads=1)
    cache, wide, starts, lse, mass = make(c)
    for i, r in enumerate(dead):
        lse[r] = (math.inf, -math.inf)[i % 2]
    want, tol = K.weigh(cache, 1, wide[:, 1:5], starts, [0], lse, mass, False, 1 / math.sqrt(128), True, 0)
    first = 300 - new + min(dead)  # the first token that only they see
    for j in range(first, 300):
        cache["codes"][1, 0, int(cache["tables"][0, j // 16]), j % 16, 0, 5] = 0x7F
    got = Q.on_gpu(cache).weigh(1, wide.cuda()[:, 1:5], starts.cuda(), lse.cuda(), mass.cuda())
    held_to(got, want, tol, c, mass)
    assert torch.equal(got[0, first:].cpu(), mass[0, first:])


@pytest.mark.parametrize("new", [3, 60, 64, 200])
@pytest.mark.parametrize("causal", [True, False])
def test_nan_keys_and_no_row_that_counts(new, causal):
    c = case([300], [new], heads=4, kv_heads=1)
    cache, wide, starts, lse, mass = make(c)
    for j in (0, 17, 250, 299):
        cache["codes"][1, 0, int(cache["tables"][0, j // 16]), j % 16, 0, 5] = 0xFF
    lse[:] = math.inf
    got = Q.on_gpu(cache).weigh(1, wide.cuda()[:, 1:5], starts.cuda(), lse.cuda(), mass.cuda(), causal=causal)
    assert torch.equal(got.cpu(), mass)


@pytest.mark.parametrize("new", [10, 60])
def test_entries_out_of_order_give_nothing_wrong(new):
    """Entries whose rows lie the other way round, with a bad one between: it is reported, and every other's masses are as
    the definition has them or as they were."""
    c = case([200, 50, 180], [new, 1, new + 40], heads=8, kv_heads=2)
    cache, wide, _, _, mass = make(c)
    wide = wide[:2 * new + 40]
    starts = torch.tensor([new + 40, 2 * new + 40, 0, new + 40], dtype=torch.int32)
    lse = torch.zeros((2 * new + 40, 8))
    for a, b, s in ((0, new + 40, 2), (new + 40, 2 * new + 40, 0)):
        lse[a:b] = Q.attend(cache, 1, wide[a:b, 1:9], torch.tensor([0, b - a]), [s], 1 / math.sqrt(128), True, 0)[1].float()
    dev = Q.on_gpu(cache)
    got = dev.weigh(1, wide.cuda()[:, 1:9], starts.cuda(), lse.cuda(), mass.cuda(), begin=True).cpu()
    assert dev.status() == (kvl.KVL_EINVAL, 1)
    assert torch.equal(got[1], mass[1])
    for a, b, s, n in ((0, new + 40, 2, 180), (new + 40, 2 * new + 40, 0, 200)):
        if torch.equal(got[s], mass[s]):
            continue
        want, tol = K.weigh(cache, 1, wide[a:b, 1:9], torch.tensor([0, b - a]), [s], lse[a:b], mass, True, 1 / math.sqrt(128), True, 0)
        assert float(((got[s].double() - want[s]).abs() - tol[s]).max()) <= 0
