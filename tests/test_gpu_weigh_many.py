"""kvl_weigh over many entries."""
from __future__ import annotations

import pytest
import torch

import layer_wise_paged_gb300 as kvl
from tests.test_gpu_weigh import case, run

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
