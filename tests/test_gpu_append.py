"""kvl_cache_append and kvl_rotary against their plain definitions (tests/_quant.py)."""
from __future__ import annotations

import math

import pytest
import torch

import layer_wise_paged_gb300 as kvl
from tests import _quant as Q

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvl.build()
    kvl.lib()


SHAPES = {  # lens after, fresh, H, d, B
    "one token each": ([1, 16, 17, 33, 100], [1, 1, 1, 1, 1], 2, 128, 16),
    "a few tokens": ([5, 18, 40, 64, 0, 31], [5, 3, 30, 17, 0, 2], 3, 64, 16),
    "prompt": ([301], [301], 8, 128, 16),
    "prompt after a part of a page": ([301], [290], 9, 128, 16),
    "page of 1": ([7, 3], [4, 3], 2, 64, 1),
    "page of 5": ([43, 11], [11, 1], 2, 48, 5),
    "page of 32": ([100, 49], [70, 49], 5, 64, 32),
    "page of 64": ([200, 65, 64], [150, 1, 64], 3, 128, 64),
    "page of 128": ([300], [250], 2, 128, 128),
    "page of 200, read twice": ([470, 30], [450, 3], 2, 64, 200),
    "head of 16": ([40], [25], 2, 16, 16),
    "head of 80": ([40], [25], 2, 80, 16),
    "head of 256": ([40, 90], [25, 1], 2, 256, 16),
    "forty sequences": (list(range(1, 41)), [1 + i % 3 if i else 1 for i in range(40)], 1, 64, 16),
}


def run(lens, new, H, d, B, code, dtype, gain=1.0, edit=None, slots=None):
    g = torch.Generator().manual_seed(len(lens) + d)
    cache = Q.make_cache(8, 2, H, d, B, lens, code=code, poison=False)
    cache["scales"] *= 0.5  # some pages' scales grow, some stay
    starts = torch.tensor([0] + list(new)).cumsum(0).int()
    T = int(starts[-1])
    wide = (torch.randn((T, 2 * H + 1, d), generator=g) * gain * torch.exp(torch.randn((T, 1, 1), generator=g))).to(dtype)
    if edit:
        edit(wide)
    dev = Q.on_gpu(cache)
    w = wide.cuda()
    sl = None if slots is None else torch.tensor(slots).int().cuda()
    dev.append(1, w[:, :H], w[:, H + 1:], starts.cuda(), slots=sl)
    assert dev.status() == (0, 0)
    Q.append(cache, 1, wide[:, :H], wide[:, H + 1:], starts, range(len(new)) if slots is None else slots)
    return dev, cache


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("name", SHAPES)
def test_codes_and_scales_are_the_documented_ones(name, dtype, code):
    dev, want = run(*SHAPES[name], code, dtype)
    assert torch.equal(dev.scales.cpu(), want["scales"])
    assert torch.equal(dev.codes.cpu(), want["codes"])  # every byte, the untouched ones too


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_zeros_infinities_and_nan(code):
    def edit(w):
        w[0:3] = 0.0
        w[5, :, 3] = math.inf
        w[6, :, 4] = -math.inf
        w[7, :, 5] = math.nan
        w[30] = 1e-36   # below the smallest scale
        w[20:40, 0] = 0.0  # a page of nothing
    dev, want = run([60], [60], 2, 64, 16, code, BF, edit=edit)
    assert torch.equal(dev.scales.cpu(), want["scales"])
    got, exp = Q.of_codes(dev.codes.cpu(), code), Q.of_codes(want["codes"], code)
    assert torch.equal(torch.isnan(got), torch.isnan(exp)) and torch.equal(got.nan_to_num(), exp.nan_to_num())
    assert torch.isfinite(dev.scales[1]).all()


def test_slots():
    dev, want = run([20, 30, 40], [4, 7], 2, 64, 16, "e4m3", BF, slots=[2, 0])
    assert torch.equal(dev.codes.cpu(), want["codes"]) and torch.equal(dev.scales.cpu(), want["scales"])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,d,B", [(128, 128, 16), (64, 128, 16), (48, 80, 24), (64, 64, 200)])
def test_keys_turned_on_their_way(rot, d, B, interleaved):
    """Codes with rope: the turned key is right to 32 bits, so a code may differ from the exact one
    only where the quotient lies within 2^-20 of a rounding boundary; values differ by less
    than half a step plus that."""
    from layer_wise_paged_gb300.cache import Rope
    lens, new, H = [300, 131], [290, 3], 2
    g = torch.Generator().manual_seed(rot)
    cache = Q.make_cache(8, 1, H, d, B, lens, poison=False)
    starts = torch.tensor([0] + new).cumsum(0).int()
    k, v = (torch.randn((293, H, d), generator=g).to(BF) for _ in range(2))
    rope = Rope.make(rot, base=500000.0, kind="wavelength", factor=8.0, interleaved=interleaved)
    dev = Q.on_gpu(cache)
    dev.append(0, k.cuda(), v.cuda(), starts.cuda(), rope=rope)
    assert dev.status() == (0, 0)
    pos = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)])
    turned = Q.turn(k, pos, rope.inv_freq.cpu(), interleaved)
    for i in range(2):
        n, m = lens[i], new[i]
        for t in range(m):
            p = n - m + t
            page, slot = int(cache["tables"][i, p // B]), p % B
            s = dev.scales[0, 0, page].cpu().double()
            got = Q.of_codes(dev.codes[0, 0, page, slot].cpu(), "e4m3") * s[:, None]
            x = turned[int(starts[i]) + t]
            # half a step of a 4-bit significand, or of the smallest step (2^-9) of the scale
            tol = torch.maximum(x.abs() * 2.0 ** -4, s[:, None] * 2.0 ** -10) * (1 + 2.0 ** -10) + s[:, None] * 2.0 ** -10
            assert ((got - x).abs() <= tol).all()
    Q.append(cache, 0, turned, v, starts, range(2))
    assert torch.allclose(dev.scales.cpu(), cache["scales"], rtol=2.0 ** -20)
    assert float((dev.codes.cpu() != cache["codes"]).double().mean()) < 1e-3


def test_problems_are_reported_and_left_out():
    cache = Q.make_cache(4, 1, 2, 64, 16, [40, 50, 60], poison=False)
    cache["tables"][1, 3] = 9999
    dev = Q.on_gpu(cache)
    k = torch.randn((6, 2, 64)).to(BF)
    starts = torch.tensor([0, 2, 4, 6]).int()
    dev.append(0, k.cuda(), k.cuda(), starts.cuda())
    assert dev.status() == (kvl.KVL_ERANGE, 1)
    Q.append(cache, 0, k[[0, 1, 4, 5]], k[[0, 1, 4, 5]], torch.tensor([0, 2, 4]), [0, 2])
    assert torch.equal(dev.codes.cpu(), cache["codes"]) and torch.equal(dev.scales.cpu(), cache["scales"])
    dev.reset_status()
    dev.lens[0] = 1  # two fresh tokens, one held
    dev.append(0, k.cuda(), k.cuda(), starts.cuda(), slots=torch.tensor([0, 2, 2]).int().cuda()[:3])
    assert dev.status()[0] == kvl.KVL_EINVAL


# ---- rotary -----------------------------------------------------------------------------------

@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("rows,heads,d,rot", [(1, (8, 2), 128, 128), (7, (4,), 64, 32), (130, (3, 1, 2), 80, 72),
                                              (33, (2, 2), 256, 256), (5, (1,), 96, 40)])
def test_rotary(rows, heads, d, rot, dtype, interleaved, inverse):
    """|error| <= the output's rounding + 2^-21 of the pair's magnitude (32-bit products)."""
    from layer_wise_paged_gb300.cache import Rope, rotary
    g = torch.Generator().manual_seed(rows + d)
    f = torch.rand(rot // 2, generator=g)
    f[0] = 1.0
    pos = torch.randint(-5, 2 ** 17, (rows,), generator=g).int()
    pos[0] = 2 ** 31 - 1 if rows > 5 else 3
    wide = torch.randn((rows, sum(heads) + 1, d), generator=g).to(dtype)
    rope = Rope(f.cuda(), interleaved=interleaved, gain=1.25)
    src, at = wide.cuda(), 0
    parts = []
    for n in heads:
        parts.append((at, n))
        at += n
    dst = torch.full((rows, sum(heads), d), 9.0, dtype=dtype, device="cuda")
    p = pos.cuda()
    rotary(rope, p, [(src[:, a:a + n], dst[:, a:a + n]) for a, n in parts], inverse=inverse)
    want = Q.turn(wide[:, :sum(heads)], pos, f, interleaved, 1.25, inverse)
    mag = wide[:, :sum(heads)].double().abs().amax(-1, keepdim=True)
    err = (dst.cpu().double() - want).abs()
    assert (err <= Q.UNIT[dtype] * want.abs() + 2.0 ** -21 * 2.5 * mag + 1e-12).all()
    # in place gives the same
    rotary(rope, p, [(src[:, a:a + n], src[:, a:a + n]) for a, n in parts], inverse=inverse)
    assert torch.equal(src[:, :sum(heads)], dst) and torch.equal(src[:, sum(heads):].cpu(), wide[:, sum(heads):])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_inverse_is_the_gradient(interleaved):
    """<g, R x> = <R' g, x>, and differences of the forward map along each element (the map is
    linear, so a difference of any size is the derivative)."""
    from layer_wise_paged_gb300.cache import Rope, rotary
    rows, d = 3, 16
    g = torch.Generator().manual_seed(3)
    rope = Rope.make(12 - 4, interleaved=interleaved, kind="linear", factor=2.0, scale_gain=True)
    pos = torch.tensor([0, 5, 70000]).int().cuda()
    x, grad = (torch.randn((rows, 1, d), generator=g).cuda() for _ in range(2))
    y, back = torch.empty_like(x), torch.empty_like(x)
    rotary(rope, pos, [(x, y)])
    rotary(rope, pos, [(grad, back)], inverse=True)
    assert abs(float((grad.double() * y.double()).sum() - (back.double() * x.double()).sum())) < 1e-4
    for e in range(d):
        x2, y2 = x.clone(), torch.empty_like(x)
        x2[:, :, e] += 1.0
        rotary(rope, pos, [(x2, y2)])
        diff = ((y2.double() - y.double()) * grad.double()).sum(-1)
        assert torch.allclose(diff, back[:, :, e].double(), atol=1e-5)


def test_rotary_far_positions_keep_their_angle():
    """At position 10^6 a 32-bit product position * frequency has lost the angle; this has not."""
    from layer_wise_paged_gb300.cache import Rope, rotary
    f = torch.tensor([0.7, 0.31, 0.11, 0.043]).cuda()
    pos = torch.tensor([10 ** 6 + 1, 2 ** 24 + 1, 2 ** 31 - 1, -(2 ** 31)]).int().cuda()
    x = torch.zeros((4, 1, 8), device="cuda")
    x[..., :4] = 1.0
    y = torch.empty_like(x)
    rotary(Rope(f), pos, [(x, y)])
    a = pos.cpu().double()[:, None] * f.cpu().double()[None]
    assert torch.allclose(y[:, 0, :4].cpu().double(), torch.cos(a), atol=2e-6)
    assert torch.allclose(y[:, 0, 4:].cpu().double(), torch.sin(a), atol=2e-6)
