"""The 8-bit cache's operators at the edges of what they take: head sizes, weights, streams and
captures that tests/test_gpu_attend.py and tests/test_gpu_append.py leave out."""
from __future__ import annotations

import math

import pytest
import torch

import layer_wise_paged_gb300 as kvl
from tests import _quant as Q
from tests import test_gpu_append as A
from tests import test_gpu_attend as T

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvl.build()
    kvl.lib()


# ---- head sizes between the kernels' own ----------------------------------------------------------

HEADS = {
    "one token": T.case([90, 33, 16], [1, 1, 1], heads=8, kv_heads=2),
    "many rows": T.case([70, 19], [40, 3], heads=4, kv_heads=2, dtype=HF),
    "page of 5": T.case([43, 11], [4, 1], B=5, heads=6, kv_heads=3),
}


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [144, 192, 240])
@pytest.mark.parametrize("name", HEADS)
def test_heads_between_128_and_256(name, d, code):
    """A row's elements end at head_dim: what lies past it (another head's codes, a slot nobody wrote)
    is NaN here and reaches no result.  Sequences end inside a page."""
    out, lse, (o, z, to, tz) = T.run(dict(HEADS[name], d=d, code=code))
    T.near(out, o, to, "out")
    T.near(lse, z, tz, "lse")


@pytest.mark.parametrize("code,B", [("e4m3", 16), ("int8", 5)])
@pytest.mark.parametrize("d", [48, 144, 192])
def test_another_heads_nan_stays_there(d, code, B):
    """NaN codes (the extreme ones of int8) in every other KV head: the rows of head 1 see none of them."""
    cache = Q.make_cache(11, 1, 3, d, B, [45], spare=0, code=code)
    cache["codes"][:, :, :, :, 0::2] = 0x7F
    dev = Q.on_gpu(cache)
    q = torch.randn((3, 3, d), generator=torch.Generator().manual_seed(4)).to(BF)
    starts = torch.tensor([0, 3]).int()
    out = dev.attend(0, q.cuda(), starts.cuda())
    o, _, to, _ = Q.attend(cache, 0, q, starts, [0], 1 / math.sqrt(d), True, 0)
    T.near(out.cpu().double()[:, 1], o[:, 1], to[:, 1], "out")


@pytest.mark.parametrize("d,B", [(144, 16), (192, 5), (240, 16)])
def test_append_to_heads_between_128_and_256(d, B):
    dev, want = A.run([43, 11, 90], [11, 1, 60], 2, d, B, "e4m3", BF)
    assert torch.equal(dev.scales.cpu(), want["scales"]) and torch.equal(dev.codes.cpu(), want["codes"])
