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


# ---- small weights beside a large one -----------------------------------------------------------------

@pytest.mark.parametrize("share", [0.5, 0.8, 0.95])
@pytest.mark.parametrize("tokens,new,seqs", [(131072, 64, 320), (131072, 2, 320), (131072, 64, 1), (20000, 130, 3)])
def test_long_tail_beside_a_peak(tokens, new, seqs, share):
    """The first token holds `share` of the softmax and has no V; a long tail whose V is about 1 holds the
    rest, each token far below 2^-14 of the largest weight.  Many sequences (that share their pages) keep a
    row in one CTA, so that all of its tail stands beside the peak.

    A weight enters its product as a half with 2^4 or more for the largest of the row, so it is off by
    2^-11 of itself, or by 2^-25 (2^-29 of the largest) where it is a subnormal half; out is rounded
    to 2^-8 of itself, and a score is a sum of two products in 32 bits (72 roundings of 2^-23 bound it)."""
    d, B = 64, 16
    g = torch.Generator().manual_seed(tokens + new)
    cache = Q.make_cache(12, 1, 1, d, B, [1], spare=0)  # (its tensors are replaced)
    N = tokens // B
    codes = torch.zeros((1, 2, N, B, 1, d), dtype=torch.uint8)
    k = torch.zeros((N * B, d))
    k[1:, 1] = torch.rand(tokens - 1, generator=g) * 2 - 1
    k[0, 0] = 440.0 / 16
    v = torch.zeros((N * B, d))
    v[1:] = 1.0 + 0.25 * torch.rand((tokens - 1, 1), generator=g)
    codes[0, 0, :, :, 0] = Q.to_codes(k * 16, "e4m3").view(N, B, d)
    codes[0, 1, :, :, 0] = Q.to_codes(v * 16, "e4m3").view(N, B, d)
    kd, vd = (Q.of_codes(codes[0, p], "e4m3").view(N * B, d) / 16 for p in (0, 1))
    top = math.log(share / (1 - share) * tokens * math.sinh(1.0))  # the tail's mean of exp is sinh(1)
    q = torch.zeros((new, 1, d))
    q[:, 0, 0] = top * 8 / float(kd[0, 0])
    q[:, 0, 1] = 8.0
    q = q.to(BF)
    perm = torch.randperm(N, generator=g)
    pool = torch.empty_like(codes)
    pool[:, :, perm] = codes
    from layer_wise_paged_gb300.cache import QuantCache
    dev = QuantCache(pool.cuda(), torch.full((1, 2, N, 1), 1 / 16).cuda(), perm.int().expand(seqs, N).contiguous().cuda(),
                     torch.full((seqs,), tokens).int().cuda(), torch.full((N,), seqs, dtype=torch.int32, device="cuda"))
    starts = (torch.arange(seqs + 1) * new).int().cuda()
    out = dev.attend(0, q.repeat(seqs, 1, 1).cuda(), starts, max_new=new).view(seqs, new, d).cpu().double()
    s = (q[:, 0].double() @ kd.T) / 8.0
    s.masked_fill_(torch.arange(tokens)[None] > torch.arange(tokens - new, tokens)[:, None], -math.inf)
    p = torch.softmax(s, -1)
    want = p @ vd
    assert 0.5 * (1 - share) < float(want.min()) and float(want.max()) < 2.5 * (1 - share)
    ds = 72 * 2.0 ** -23 * float(q.double().abs().max() * kd.abs().max() / 8)
    tol = (2.0 ** -8 + 2.0 ** -11 + 2 * ds) * want + tokens * 2.0 ** -29 * p.amax(-1, keepdim=True) * 1.25
    assert float(((out - want).abs() - tol).max()) <= 0, float(((out - want).abs() / want).max())


# ---- captures -------------------------------------------------------------------------------------

def _long_cache(seed=21):
    """Sequences that are cut over several CTAs, queries of one and of 70 tokens, and their results."""
    cache = Q.make_cache(seed, 1, 2, 64, 16, [6000, 9000])
    dev = Q.on_gpu(cache)
    g = torch.Generator().manual_seed(seed)
    calls = []
    for new in (1, 70):
        q = torch.randn((2 * new, 4, 64), generator=g).to(BF).cuda()
        starts = torch.tensor([0, new, 2 * new]).int().cuda()
        calls.append((q, starts, new, dev.attend(0, q, starts, max_new=new)))
    torch.cuda.synchronize()
    return dev, calls


def _attend_all(dev, calls, outs):
    for (q, starts, new, _), out in zip(calls, outs):
        dev.attend(0, q, starts, out=out, max_new=new)


def _outs(calls):
    return [torch.zeros_like(want) for _, _, _, want in calls]


def _dirty_pool():
    """A graph whose memory pool holds free memory full of ones."""
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
        big.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    del big
    return graph


def test_second_capture_runs_without_the_first():
    """Two captures in a row on the same stream, without a call there before; only the second is run."""
    dev, calls = _long_cache()
    dirty = _dirty_pool()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], [_outs(calls) for _ in range(2)]
    for graph, out in zip(graphs, outs):
        with torch.cuda.graph(graph, pool=dirty.pool()):
            _attend_all(dev, calls, out)
    for _ in range(3):
        graphs[1].replay()
    torch.cuda.synchronize()
    for (_, _, _, want), first, second in zip(calls, *outs):
        assert not bool(first.any())
        assert torch.equal(second, want)
    graphs[0].replay()
    torch.cuda.synchronize()
    for (_, _, _, want), first in zip(calls, outs[0]):
        assert torch.equal(first, want)
    assert dev.status() == (0, 0)


def test_calls_on_a_stream_after_a_capture_that_never_ran():
    dev, calls = _long_cache()
    dirty = _dirty_pool()
    graph, stream, never, outs = torch.cuda.CUDAGraph(), torch.cuda.Stream(), _outs(calls), _outs(calls)
    with torch.cuda.graph(graph, pool=dirty.pool(), stream=stream):
        _attend_all(dev, calls, never)
    with torch.cuda.stream(stream):
        _attend_all(dev, calls, outs)
    torch.cuda.synchronize()
    for (_, _, _, want), out, no in zip(calls, outs, never):
        assert torch.equal(out, want) and not bool(no.any())


def test_two_graphs_and_calls_at_the_same_time():
    """Graphs captured on one stream, run on two others beside calls on the capture's stream."""
    dev, calls = _long_cache()
    side = torch.cuda.Stream()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], [_outs(calls) for _ in range(3)]
    for graph, out in zip(graphs, outs):
        with torch.cuda.graph(graph, stream=side):
            _attend_all(dev, calls, out)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(30):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        with torch.cuda.stream(side):
            _attend_all(dev, calls, outs[2])
    torch.cuda.synchronize()
    for out in outs:
        for (_, _, _, want), x in zip(calls, out):
            assert torch.equal(x, want)
    assert dev.status() == (0, 0)


# ---- streams ----------------------------------------------------------------------------------------

def test_result_made_for_another_stream():
    """The result of a call on a given stream is that stream's memory: not a block that was just freed on the
    current one, where work on it is still to come."""
    dev, calls = _long_cache()
    side = torch.cuda.Stream()
    q, starts, new, want = calls[1]
    for cycles in (1000, 200_000_000):  # (the first time its kernels are loaded, which waits for the GPU)
        dev.attend(0, q, starts, out=torch.empty_like(want), max_new=new, stream=side)
        torch.cuda.synchronize()
        freed = torch.empty_like(want)
        torch.cuda._sleep(cycles)  # 0.1 s of the current stream, behind which it still writes `freed`
        freed.fill_(7.0)
        del freed
        out = dev.attend(0, q, starts, max_new=new, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        del out
    out = dev.attend(0, q, starts, max_new=new, stream=torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ---- windows ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("window", [1, 19, 2 ** 30, 2 ** 31 - 1])
@pytest.mark.parametrize("lens,new", [([2, 40], [5, 3]), ([20, 33], [60, 33])])
def test_windows_up_to_the_largest(lens, new, window):
    """Also where an entry has more rows than tokens, so that its first rows stand before token 0."""
    out, lse, (o, z, to, tz) = T.run(T.case(lens, new, window=window))
    T.near(out, o, to, "out")
    T.near(lse, z, tz, "lse")


@pytest.mark.parametrize("name", ["window", "max_new"])
@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 5, -2 ** 32 + 5])
def test_numbers_past_32_bits_are_refused(name, n):
    """They do not wrap round to another window."""
    dev = Q.on_gpu(Q.make_cache(1, 1, 2, 64, 16, [40]))
    q, starts = torch.zeros((1, 4, 64), dtype=BF, device="cuda"), torch.tensor([0, 1]).int().cuda()
    with pytest.raises(ValueError, match="32-bit"):
        dev.attend(0, q, starts, **{name: n})


# ---- V scales far apart ---------------------------------------------------------------------------------

@pytest.mark.parametrize("zero_scale", [1e-30, 0.0])
@pytest.mark.parametrize("new", [1, 64])
def test_pages_of_zeros_beside_large_values(new, zero_scale):
    """Pages whose V is zero (append gives them the smallest scale, an empty cache holds 0) count in the
    softmax however large the other pages' V scales are."""
    tokens, d = 4000 + new, 64
    cache = Q.make_cache(13, 1, 1, d, 16, [tokens], spare=0)
    k = torch.zeros((tokens + 16, d))
    k[16:, 0] = -15 * math.log(2.0)
    pages = cache["tables"][0, :-(-tokens // 16)].long()
    n = len(pages)
    cache["codes"][:] = 0
    cache["codes"][0, 0, pages, :, 0] = Q.to_codes(k[:n * 16] * 16, "e4m3").view(n, 16, d)
    cache["scales"][0, 0] = 1 / 16
    cache["scales"][0, 1] = zero_scale
    cache["codes"][0, 1, pages[0]] = Q.to_codes(1 + torch.rand((16, 1, d), generator=torch.Generator().manual_seed(1)), "e4m3")
    cache["scales"][0, 1, pages[0]] = 2.0 ** 20
    q = torch.zeros((new, 1, d))
    q[:, 0, 0] = 8.0
    q, starts = q.to(BF), torch.tensor([0, new]).int()
    dev = Q.on_gpu(cache)
    lse = torch.zeros((new, 1), device="cuda")
    out = dev.attend(0, q.cuda(), starts.cuda(), lse=lse, max_new=new)
    o, z, to, tz = Q.attend(cache, 0, q, starts, [0], 1 / 8.0, True, 0)
    T.near(out.cpu().double(), o, to, "out")
    T.near(lse.cpu().double(), z, tz, "lse")


@pytest.mark.parametrize("new", [1, 64])
def test_softmax_sums_of_a_cache_of_zeros(new):
    """V zero everywhere, and scores that grow along the sequence: the sums stay finite."""
    tokens, d = 40000, 64
    cache = Q.make_cache(14, 1, 1, d, 16, [tokens], spare=0)
    pages = cache["tables"][0, :tokens // 16].long()
    k = torch.zeros((tokens, d))
    k[1024:, 0] = 7.0
    cache["codes"][:] = 0
    cache["codes"][0, 0, pages, :, 0] = Q.to_codes(k * 16, "e4m3").view(-1, 16, d)
    cache["scales"][0, 0], cache["scales"][0, 1] = 1 / 16, 1e-30
    q = torch.zeros((new, 1, d))
    q[:, 0, 0] = 8.0
    q = q.to(BF)
    # one sequence would be cut over all CTAs: 320 that share their pages are not
    from layer_wise_paged_gb300.cache import QuantCache
    dev = QuantCache(cache["codes"].cuda(), cache["scales"].cuda(), cache["tables"].expand(320, -1).contiguous().cuda(),
                     torch.full((320,), tokens).int().cuda(), cache["refs"].cuda() * 320)
    lse = torch.zeros((320 * new, 1), device="cuda")
    out = dev.attend(0, q.repeat(320, 1, 1).cuda(), (torch.arange(321) * new).int().cuda(), lse=lse, max_new=new)
    kd = Q.of_codes(Q.to_codes(k[:, 0] * 16, "e4m3"), "e4m3") / 16
    seen = torch.arange(tokens)[None] <= torch.arange(tokens - new, tokens)[:, None]
    want = torch.logsumexp(torch.where(seen, kd[None], torch.full_like(kd, -math.inf)[None]), -1)
    assert not bool(out.any())
    assert float((lse.view(320, new).cpu().double() - want).abs().max()) < 1e-4


# ---- sizes where the choice of kernel changes -----------------------------------------------------------

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [31, 32, 33, 40, 41, 64])
def test_rows_around_the_choice_of_kernel(rows, d):
    """In a batch whose entries lie on both sides, and as the only entry."""
    for new in ([rows, 1, 70], [rows]):
        c = T.case([100, 40, 90][:len(new)], new, heads=2, kv_heads=2, d=d)
        out, lse, (o, z, to, tz) = T.run(c)
        T.near(out, o, to, "out")
        T.near(lse, z, tz, "lse")


# ---- append with the turn -------------------------------------------------------------------------------

def _turned(lens, new, H, d, B, rot, interleaved, code, dtype=BF):
    g = torch.Generator().manual_seed(rot + d)
    cache = Q.make_cache(8, 1, H, d, B, lens, code=code, poison=False)
    starts = torch.tensor([0] + new).cumsum(0).int()
    k, v = (torch.randn((sum(new), H, d), generator=g).to(dtype) for _ in range(2))
    from layer_wise_paged_gb300.cache import Rope
    rope = Rope.make(rot, base=500000.0, interleaved=interleaved)
    pos = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)])
    return cache, starts, k, v, rope, pos


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,d,B", [(128, 128, 16), (48, 80, 24), (64, 64, 200), (192, 192, 16)])
def test_int8_keys_turned_on_their_way(rot, d, B, interleaved):
    """The turned key is right to 2^-20 of its pair, so its code is the nearest integer of the exact key over the
    scale, or one beside it where the quotient lies within 127 * 2^-18 of a half; values differ
    by half a step and that much."""
    lens, new, H = [300, 131], [290, 3], 2
    cache, starts, k, v, rope, pos = _turned(lens, new, H, d, B, rot, interleaved, "int8")
    dev = Q.on_gpu(cache)
    dev.append(0, k.cuda(), v.cuda(), starts.cuda(), rope=rope)
    assert dev.status() == (0, 0)
    turned = Q.turn(k, pos, rope.inv_freq.cpu(), interleaved)
    for i, (n, m) in enumerate(zip(lens, new)):
        for t in range(m):
            page, slot = int(cache["tables"][i, (n - m + t) // B]), (n - m + t) % B
            s = dev.scales[0, 0, page].cpu().double()[:, None]
            got = Q.of_codes(dev.codes[0, 0, page, slot].cpu(), "int8") * s
            assert ((got - turned[int(starts[i]) + t]).abs() <= s * (0.5 + 127 * 2.0 ** -18)).all()
    Q.append(cache, 0, turned, v, starts, range(2))
    assert torch.allclose(dev.scales.cpu(), cache["scales"], rtol=2.0 ** -20)
    step = (Q.of_codes(dev.codes.cpu(), "int8") - Q.of_codes(cache["codes"], "int8")).abs()
    assert float(step.max()) <= 1 and float((step > 0).double().mean()) < 1e-3
    assert torch.equal(dev.codes[0, 1].cpu(), cache["codes"][0, 1])  # V is not turned


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_pairs_that_append_does_not_take(code):
    """24 turned elements of 96: append refuses 12 pairs (not a multiple of 8); rotary takes them, in place, and
    append the turned keys."""
    from layer_wise_paged_gb300.cache import rotary
    cache, starts, k, v, rope, pos = _turned([40, 9], [30, 9], 2, 96, 16, 24, False, code, dtype=F32)
    dev = Q.on_gpu(cache)
    kd, vd, sd = k.cuda(), v.cuda(), starts.cuda()
    with pytest.raises(kvl.KvlError):
        dev.append(0, kd, vd, sd, rope=rope)
    rotary(rope, pos.int().cuda(), [(kd, kd)])
    dev.append(0, kd, vd, sd)
    assert dev.status() == (0, 0)
    Q.append(cache, 0, kd.cpu(), v, starts, range(2))
    assert torch.equal(dev.codes.cpu(), cache["codes"]) and torch.equal(dev.scales.cpu(), cache["scales"])


# ---- large batches of many rows ---------------------------------------------------------------------------

@pytest.mark.parametrize("code,window", [("e4m3", 0), ("int8", 200)])
def test_many_sequences_of_many_rows(code, window):
    """300 entries of 150 rows: each CTA has several jobs, whole and in parts.  Tolerance as in
    tests/test_gpu_attend.py's batches: the output's rounding and 2^-9 of the magnitudes it sums."""
    seqs, new = 300, 150
    g = torch.Generator().manual_seed(9)
    lens = [max(new, int(x)) for x in torch.randint(1, 900, (seqs,), generator=g)]
    cache = Q.make_cache(3, 1, 2, 64, 16, lens, code=code)
    dev = Q.on_gpu(cache)
    q = torch.randn((seqs * new, 4, 64), generator=g).to(BF).cuda()
    starts = (torch.arange(seqs + 1) * new).int().cuda()
    out = dev.attend(0, q, starts, max_new=new, window=window)
    assert torch.equal(out, dev.attend(0, q, starts, max_new=new, window=window)), "two calls differ"
    assert dev.status() == (0, 0)
    for i in sorted({0, 1, 100, 151, 222, seqs - 1}):
        K, V = (Q.tokens(cache, 0, p, i, lens[i]).cuda() for p in (0, 1))
        s = torch.einsum("thd,khd->thk", q[i * new:(i + 1) * new].double(), K.repeat_interleave(2, 1)) / 8.0
        pos = torch.arange(lens[i] - new, lens[i], device="cuda")[:, None]
        at = torch.arange(lens[i], device="cuda")[None]
        hidden = at > pos if not window else (at > pos) | (at <= pos - window)
        p = torch.softmax(s.masked_fill(hidden[:, None], -math.inf), -1)
        want = torch.einsum("thk,khd->thd", p, V.repeat_interleave(2, 1))
        mag = torch.einsum("thk,khd->thd", p, V.abs().repeat_interleave(2, 1))
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -9 * mag + 1e-4
        assert float(((out[i * new:(i + 1) * new].double() - want).abs() - tol).max()) <= 0
