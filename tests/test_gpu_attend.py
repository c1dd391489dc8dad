"""kvl_attend against the plain 64-bit definition (tests/_quant.py), at the sizes, masks and
contents where attention over a paged 8-bit cache can go wrong."""
from __future__ import annotations

import math

import pytest
import torch

import layer_wise_paged_gb300 as kvl
from tests import _quant as Q

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvl.build()
    kvl.lib()


def case(lens, new, heads=8, kv_heads=2, d=128, B=16, code="e4m3", dtype=BF, causal=True, window=0, gain=1.0,
         q_gain=1.0, max_new=None):
    return dict(lens=lens, new=new, heads=heads, kv_heads=kv_heads, d=d, B=B, code=code, dtype=dtype, causal=causal,
                window=window, gain=gain, q_gain=q_gain, max_new=max_new)


CASES = {
    "one token, one held": case([1], [1]),
    "one token": case([777], [1], heads=32, kv_heads=8),
    "one head each": case([130], [1], heads=4, kv_heads=4),
    "sixteen heads on one": case([95, 33], [1, 1], heads=16, kv_heads=1),
    "odd group": case([61, 200], [1, 2], heads=6, kv_heads=2),
    "ragged, empty ones among them": case([0, 1, 15, 16, 17, 300, 0, 64], [0, 1, 1, 1, 1, 1, 0, 0]),
    "rows of an empty sequence": case([0, 20], [3, 2]),
    "more rows than tokens": case([2, 40], [5, 3]),
    "more rows than tokens, all visible": case([2, 40], [5, 3], causal=False),
    "drafted": case([100, 9, 257, 64], [8, 3, 1, 5], kv_heads=4, heads=16, d=64, code="int8", dtype=HF),
    "drafted, page of 64": case([100, 9, 257, 64], [8, 3, 1, 5], B=64, heads=32, kv_heads=4),
    "page of 1": case([19, 5], [2, 1], B=1),
    "page of 5": case([43, 11], [4, 1], B=5),
    "page of 24": case([100, 49], [1, 30], B=24),
    "page of 48": case([100, 49, 96], [1, 2, 1], B=48, d=64),
    "page of 256": case([700, 256], [1, 2], B=256, code="int8"),
    "head of 16": case([90], [2], d=16),
    "head of 80": case([90, 33], [2, 33], d=80, dtype=HF),
    "head of 256": case([90, 150], [1, 40], d=256),
    "window": case([300, 40], [1, 6], window=33),
    "window of 1": case([50], [7], window=1),
    "chunk": case([200], [130]),
    "chunk, f16 int8": case([190], [150], code="int8", dtype=HF, heads=4),
    "chunk on a long prefix": case([1100], [70], heads=8, kv_heads=1),
    "chunks, ragged": case([70, 1, 0, 333, 129], [70, 1, 0, 100, 129], d=64),
    "chunk, all visible": case([150, 260], [150, 40], causal=False),
    "chunk, window": case([400], [180], window=100),
    "chunk, window inside a page": case([300], [300], window=7, heads=4, kv_heads=2),
    "chunk, page of 64": case([321], [321], B=64, heads=4, kv_heads=4, d=64, code="int8"),
    "chunk and tokens": case([500, 90, 31], [1, 90, 1]),
    "peaked": case([500], [3], gain=6.0, q_gain=6.0),
    "peaked chunk": case([400], [140], gain=6.0, q_gain=6.0, heads=4),
    "tiny values": case([100], [2], gain=1e-6),
    "bound on rows known": case([100, 40], [2, 1], max_new=2),
}


def run(c, seed=5, spread=False, stream=None):
    cache = Q.make_cache(seed, 2, c["kv_heads"], c["d"], c["B"], c["lens"], code=c["code"], gain=c["gain"])
    if spread:  # scales of the pages far apart
        f = torch.exp2(torch.linspace(-12, 9, cache["scales"].shape[2])).float()
        cache["scales"] *= f[None, None, :, None]
    g = torch.Generator().manual_seed(seed + 1)
    starts = torch.tensor([0] + c["new"]).cumsum(0).int()
    T = int(starts[-1])
    # q and out are parts of wider rows
    wide = (torch.randn((T, c["heads"] + 3, c["d"]), generator=g) * c["q_gain"]).to(c["dtype"])
    q = wide[:, 1:1 + c["heads"]]
    dev = Q.on_gpu(cache)
    wq = wide.cuda()
    wout = torch.full((T, c["heads"] + 2, c["d"]), 77.0, dtype=c["dtype"], device="cuda")
    lse = torch.full((T, c["heads"]), 77.0, device="cuda")
    out = wout[:, 2:]
    args = dict(out=out, lse=lse, causal=c["causal"], window=c["window"],
                max_new=max(c["new"] + [0]) if c["max_new"] is None else c["max_new"])
    if stream is None:
        dev.attend(1, wq[:, 1:1 + c["heads"]], starts.cuda(), **args)
    else:
        s0 = starts.cuda()
        torch.cuda.synchronize()
        dev.attend(1, wq[:, 1:1 + c["heads"]], s0, stream=stream, **args)
        stream.synchronize()
    assert dev.status() == (0, 0)
    assert (wout[:, :2] == 77.0).all(), "wrote outside its rows"
    want = Q.attend(cache, 1, q, starts, range(len(c["lens"])), 1 / math.sqrt(c["d"]), c["causal"], c["window"])
    return out.cpu().double(), lse.cpu().double(), want


def near(got, want, tol, what):
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), what
    ok = torch.isfinite(want)
    over = ((got - want).abs() - tol)[ok]
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: {float(over.max())} over its tolerance"


@pytest.mark.parametrize("name", CASES)
def test_against_the_definition(name):
    out, lse, (o, z, to, tz) = run(CASES[name])
    near(out, o, to, "out")
    near(lse, z, tz, "lse")


@pytest.mark.parametrize("name", ["one token", "drafted", "chunk", "page of 5"])
def test_scales_far_apart(name):
    out, lse, (o, z, to, tz) = run(CASES[name], spread=True)
    near(out, o, to, "out")
    near(lse, z, tz, "lse")


@pytest.mark.parametrize("name", ["one token", "chunk", "chunk and tokens"])
def test_on_another_stream(name):
    out, lse, (o, z, to, tz) = run(CASES[name], stream=torch.cuda.Stream())
    near(out, o, to, "out")
    near(lse, z, tz, "lse")


@pytest.mark.parametrize("bound", [0, 1, 3, 200])
def test_the_bound_on_rows_changes_nothing(bound):
    """max_new chooses kernels; a wrong or missing bound still gives every row."""
    c = dict(CASES["chunk and tokens"], max_new=bound)
    out, lse, (o, z, to, tz) = run(c)
    near(out, o, to, "out")
    near(lse, z, tz, "lse")


@pytest.mark.parametrize("new", [1, 6, 150])
@pytest.mark.parametrize("seqs", [1, 70, 300])
def test_many_sequences_and_splits(seqs, new):
    """Every row of a large batch equals the row computed alone, bit for bit where the split
    is the same and within the rounding of the parts' sums otherwise."""
    if seqs * new > 20000:
        pytest.skip("the pair above covers it")
    g = torch.Generator().manual_seed(seqs + new)
    lens = [max(new, int(x)) for x in torch.randint(1, 900 if seqs > 1 else 5000, (seqs,), generator=g)]
    cache = Q.make_cache(3, 1, 2, 64, 16, lens)
    dev = Q.on_gpu(cache)
    q = torch.randn((seqs * new, 4, 64), generator=g).to(BF).cuda()
    starts = (torch.arange(seqs + 1) * new).int().cuda()
    whole = dev.attend(0, q, starts, max_new=new)
    again = dev.attend(0, q, starts, max_new=new)
    assert torch.equal(whole, again), "two calls differ"
    for i in sorted({0, seqs // 3, seqs - 1}):
        K, V = (Q.tokens(cache, 0, p, i, lens[i]).cuda() for p in (0, 1))
        rows = q[i * new:(i + 1) * new].double()
        s = torch.einsum("thd,khd->thk", rows, K.repeat_interleave(2, 1)) / 8.0
        pos = torch.arange(lens[i] - new, lens[i], device="cuda")
        s.masked_fill_((torch.arange(lens[i], device="cuda")[None] > pos[:, None])[:, None], -math.inf)
        p = torch.softmax(s, -1)
        want = torch.einsum("thk,khd->thd", p, V.repeat_interleave(2, 1))
        mag = torch.einsum("thk,khd->thd", p, V.abs().repeat_interleave(2, 1))
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -9 * mag + 1e-4
        assert float(((whole[i * new:(i + 1) * new].double() - want).abs() - tol).max()) <= 0


@pytest.mark.parametrize("new,lens", [(6, 90), (140, 200)])
def test_nan_in_a_token_reaches_only_the_rows_that_see_it(new, lens):
    """A NaN value of a later token does not reach the rows before it."""
    cache = Q.make_cache(9, 1, 2, 64, 16, [lens])
    at = lens - 3
    page, slot = int(cache["tables"][0, at // 16]), at % 16
    cache["codes"][0, 1, page, slot, 0, 5] = 0x7F  # V, head 0, element 5
    cache["codes"][0, 0, page, slot, 1, 7] = 0xFF  # K, head 1
    dev = Q.on_gpu(cache)
    q = torch.randn((new, 4, 64), generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    out = dev.attend(0, q, torch.tensor([0, new], dtype=torch.int32).cuda(), max_new=new)
    sees = torch.arange(lens - new, lens) >= at
    bad = torch.isnan(out).cpu()
    want = torch.zeros_like(bad)
    want[sees, 0:2, 5] = True   # the query heads of KV head 0
    want[sees, 2:4, :] = True   # a NaN score: the whole row
    assert torch.equal(bad, want)


def test_slots_and_packed_tables():
    """Entries of the batch that name their slots, and tables packed back to back with offsets
    (as a plan's block tables are)."""
    lens = [40, 7, 130]
    cache = Q.make_cache(4, 1, 2, 64, 16, lens)
    dev = Q.on_gpu(cache)
    g = torch.Generator().manual_seed(2)
    q = torch.randn((4, 4, 64), generator=g).to(BF)
    starts, slots = torch.tensor([0, 2, 4]).int(), torch.tensor([2, 0]).int()
    out = dev.attend(0, q.cuda(), starts.cuda(), slots=slots.cuda())
    o, _, to, _ = Q.attend(cache, 0, q, starts, [2, 0], 0.125, True, 0)
    near(out.cpu().double(), o, to, "slots")
    n = [-(-x // 16) for x in lens]
    packed = torch.cat([cache["tables"][i, :k] for i, k in enumerate(n)]).cuda()
    offs = torch.tensor([0] + n).cumsum(0).cuda()
    out2, qd, sd = torch.zeros_like(out), q.cuda(), starts.cuda()
    sl = slots.cuda()
    seqs = kvl.kvl_sequences(2, 3, 4, 0, packed.data_ptr(), offs.data_ptr(), dev.lens.data_ptr(), sl.data_ptr(),
                             sd.data_ptr())
    rows = [kvl.kvl_rows(t.data_ptr(), 4 * 64 * 2, 64 * 2) for t in (qd, out2)]
    a = kvl.kvl_attention(rows[0], rows[1], None, 4, kvl.KVL_TYPE_BFLOAT, 0.125, 1, 0, 0)
    ws = torch.zeros(kvl.lib().kvl_attend_workspace_bytes(dev._c), dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert kvl.lib().kvl_attend(dev._c, 0, seqs, a, ws.data_ptr(), ws.numel(), None, st) == kvl.KVL_OK
    assert torch.equal(out, out2)


def test_pool_beyond_32_bit_offsets():
    """A pool of more than 2^32 codes a plane, the sequence's pages at its far end."""
    N, B, H, d = 262144 + 64, 16, 8, 128   # 16 KiB pages: 4.3 GB a plane
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough free device memory")
    from layer_wise_paged_gb300.cache import QuantCache
    small = Q.make_cache(6, 1, H, d, B, [150], spare=0)
    k = small["codes"].shape[2]
    codes = torch.empty((1, 2, N, B, H, d), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((1, 2, N, H), device="cuda")
    codes[:, :, N - k:], scales[:, :, N - k:] = small["codes"].cuda(), small["scales"].cuda()
    tables = torch.where(small["tables"] >= 0, small["tables"] + N - k, small["tables"]).cuda()
    dev = QuantCache(codes, scales, tables, small["lens"].cuda(), torch.zeros(N, dtype=torch.int32, device="cuda"))
    for new in (1, 60):
        q = torch.randn((new, 8, d), generator=torch.Generator().manual_seed(1)).to(BF)
        starts = torch.tensor([0, new]).int()
        out = dev.attend(0, q.cuda(), starts.cuda(), max_new=new)
        o, _, to, _ = Q.attend(small, 0, q, starts, [0], 1 / math.sqrt(d), True, 0)
        near(out.cpu().double(), o, to, "out")


def test_device_side_problems_are_reported_and_left_out():
    cache = Q.make_cache(4, 1, 2, 64, 16, [40, 50, 60])
    cache["tables"][1, 2] = cache["codes"].shape[2]  # a page number past the pool
    dev = Q.on_gpu(cache)
    q = torch.randn((3, 4, 64)).to(BF).cuda()
    starts = torch.tensor([0, 1, 2, 3]).int().cuda()
    good = dev.attend(0, q, starts)
    assert dev.status() == (kvl.KVL_ERANGE, 1)
    dev.reset_status()
    assert dev.status() == (0, 0)
    dev.lens[1] = 16 * dev.tables.shape[1] + 1  # more tokens than its table row holds
    out = torch.zeros_like(good)
    dev.attend(0, q, starts, out=out)
    assert dev.status() == (kvl.KVL_ERANGE, 1)
    assert torch.equal(out[[0, 2]], good[[0, 2]]) and (out[1] == 0).all()
    dev.reset_status()
    dev.lens[1] = 50
    dev.attend(0, q, torch.tensor([0, 1, 5, 3]).int().cuda(), out=out)  # rows past the array
    assert dev.status()[0] == kvl.KVL_EINVAL
    dev.reset_status()
    dev.attend(0, q, starts, out=out, slots=torch.tensor([0, 3, 2]).int().cuda())
    assert dev.status() == (kvl.KVL_EINVAL, 1)
    assert torch.equal(out[[0, 2]], good[[0, 2]])
