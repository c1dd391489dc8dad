"""The operators together, as examples/branches.py uses them."""
from __future__ import annotations

import pytest
import torch

import layer_wise_paged_gb300 as kvl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvl.build()
    kvl.lib()


def _check_attention(cache, layer, slots, starts, q, out):
    """out against float64 attention over the dequantised cache.  The weights are rounded to 11 bits (relative
    2^-12 each, of numerator and none of the denominator: at most 2^-11 of the largest |V|) and out to 8
    bits (relative 2^-9 of |out| <= max |V|); float32 sums and exponentials add less than 2^-11."""
    B, H, d = cache.block_tokens, cache.n_kv_heads, cache.head_dim
    group = q.shape[1] // H
    for i, slot in enumerate(slots.tolist()):
        n, r0, r1 = int(cache.lens[slot]), int(starts[i]), int(starts[i + 1])
        pages = cache.tables[slot, :-(-n // B)].long()
        if cache.code == "e4m3":
            codes = cache.codes[layer][:, pages].view(torch.float8_e4m3fn).double()
        else:
            codes = cache.codes[layer][:, pages].view(torch.int8).double()
        kv = (codes * cache.scales[layer][:, pages, None, :, None].double()).view(2, -1, H, d)[:, :n]
        k, v = kv[0].repeat_interleave(group, 1), kv[1].repeat_interleave(group, 1)
        s = torch.einsum("rhd,thd->hrt", q[r0:r1].double(), k) / d ** 0.5
        p = torch.arange(n - (r1 - r0), n, device="cuda")
        s = s.masked_fill(torch.arange(n, device="cuda")[None, :] > p[:, None], -torch.inf)
        want = torch.einsum("hrt,thd->rhd", s.softmax(-1), v)
        top = v.abs().amax((0, 2))  # per query head
        err = (out[r0:r1].double() - want).abs().amax((0, 2))
        assert bool((err <= 2 ** -8 * top).all()), (slot, float((err / top).max()))


def _check_pages(cache):
    want = torch.zeros_like(cache.refs)
    for slot in range(cache.n_slots):
        n = -(-int(cache.lens[slot]) // cache.block_tokens)
        want.index_add_(0, cache.tables[slot, :n].long(), torch.ones(n, dtype=torch.int32, device="cuda"))
    assert torch.equal(want, cache.refs)


@pytest.mark.parametrize("code,block", [("e4m3", 16), ("int8", 24), ("e4m3", 64)])
def test_branches(code, block):
    from examples import branches

    def watch(cache, layer, slots, starts, q, out):
        _check_attention(cache, layer, slots, starts, q, out)
        _check_pages(cache)

    said, cache = branches.run(block_tokens=block, code=code, watch=watch)
    # two prompts' worth of branches spoke all the way, one of each stopped half-way
    assert sorted(len(s) for s in said) == [6, 6, 6, 12, 12, 12, 12, 12, 12]
    # compacted half-way, then grown by 6 tokens a branch, lowest numbers first: no holes
    live = torch.nonzero(cache.refs).flatten()
    assert int(live.max()) + 1 == len(live)


def test_page_numbers_do_not_matter():
    """Renumbering the pages changes no bit of what follows."""
    from examples import branches
    a, ca = branches.run(compact=True)
    b, cb = branches.run(compact=False)
    assert a == b
    assert int(torch.nonzero(ca.refs).max()) < int(torch.nonzero(cb.refs).max())


def test_runs_twice_alike():
    from examples import branches
    assert branches.run()[0] == branches.run()[0]


def test_step_in_a_graph():
    """A decode step captured once and replayed leaves what the same steps leave call by call."""
    from layer_wise_paged_gb300.cache import QuantCache, Rope, rotary

    def make():
        cache = QuantCache.empty(2, 2, 64, 16, 40, 4, 10)
        rope = Rope.make(64)
        slots = torch.arange(4, dtype=torch.int32, device="cuda")
        ones = torch.ones_like(slots)
        starts = torch.arange(5, dtype=torch.int32, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(3)
        x = torch.randn(4, 8 + 2 + 2, 64, generator=g, device="cuda").to(torch.bfloat16)
        q, out = torch.empty(4, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16,
                                                                                      device="cuda")

        def step():
            rotary(rope, cache.lens, [(x[:, :8], q)])  # a token's position is the length before it
            cache.extend(slots, ones)
            cache.copy_pages()
            for layer in range(2):
                cache.append(layer, x[:, 8:10], x[:, 10:], starts, rope=rope)
                cache.attend(layer, q, starts, out=out[layer], max_new=1)

        return cache, out, step

    side = torch.cuda.Stream()
    a, out_a, step_a = make()
    b, out_b, step_b = make()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step_a()  # the workspace of this stream is made before the capture
        step_b()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step_a()
    for _ in range(20):
        graph.replay()
    with torch.cuda.stream(side):
        for _ in range(20):
            step_b()
    torch.cuda.synchronize()
    assert a.status() == b.status() == (0, 0)
    assert torch.equal(a.lens, b.lens) and int(a.lens[0]) == 21
    assert torch.equal(a.tables, b.tables) and torch.equal(a.refs, b.refs)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    assert torch.equal(out_a, out_b) and bool(out_a.any())
