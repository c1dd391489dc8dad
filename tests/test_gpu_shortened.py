"""Shared prefixes, weights and eviction together, as examples/branches.py uses them."""
from __future__ import annotations

import pytest
import torch

import layer_wise_paged_gb300 as kvl
from tests.test_gpu_branches import _check_attention, _check_pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvl.build()
    kvl.lib()


@pytest.mark.parametrize("code,block,budget", [("e4m3", 16, 0), ("int8", 24, 100), ("e4m3", 64, 130), ("e4m3", 16, 40)])
def test_branches_of_shortened_prompts(code, block, budget):
    from examples import branches
    lengths = []

    def watch(cache, layer, slots, starts, q, out):
        _check_attention(cache, layer, slots, starts, q, out)
        _check_pages(cache)
        lengths.append(cache.lens[slots.long()].tolist())

    said, cache = branches.run(block_tokens=block, code=code, watch=watch, share=True, budget=budget)
    assert sorted(len(s) for s in said) == [6, 6, 6, 12, 12, 12, 12, 12, 12]
    kept = [min(n, budget or n) for n in (37, 300, 1)]
    assert lengths[0] == [37, 300, 1]
    assert lengths[1] == [n + 1 for n in kept for _ in range(3)]
    live = torch.nonzero(cache.refs).flatten()
    assert int(live.max()) + 1 == len(live)


def test_sharing_changes_no_more_than_roundings():
    """A step's attention with and without it: of the same cache both are within their tolerance of the definition
    (above); here their answers' first tokens, chosen before any rounding differs, are the same."""
    from examples import branches
    a, _ = branches.run(steps=2)
    b, _ = branches.run(steps=2, share=True)
    assert [s[0] for s in a] == [s[0] for s in b]


def test_a_prompt_within_the_budget_keeps_everything():
    """A budget that every prompt fits evicts nothing: the caches hold the same tokens."""
    from examples import branches
    _, a = branches.run(budget=300, steps=2)
    _, b = branches.run(budget=400, steps=2)
    assert torch.equal(a.lens, b.lens) and torch.equal(a.tables, b.tables) and torch.equal(a.codes, b.codes)


def test_a_step_in_a_graph():
    """A decode step (extend, copies, append, shared attention, weights) captured once and replayed leaves what the
    same steps leave call by call; so does an eviction after them."""
    from layer_wise_paged_gb300.cache import QuantCache, Rope, rotary

    def make():
        cache = QuantCache.empty(2, 2, 64, 16, 120, 6, 12)
        rope = Rope.make(64)
        slots = torch.arange(6, dtype=torch.int32, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(3)
        # a prompt of 70 tokens, forked
        cache.extend(slots[:1], torch.full((1,), 70, dtype=torch.int32, device="cuda"))
        x = torch.randn(70, 4, 64, generator=g, device="cuda").to(torch.bfloat16)
        for layer in range(2):
            cache.append(layer, x[:, :2], x[:, 2:], torch.tensor([0, 70], dtype=torch.int32, device="cuda"), slots=slots[:1])
        cache.fork(torch.zeros(5, dtype=torch.int32, device="cuda"), slots[1:])
        ones, starts = torch.ones_like(slots), torch.arange(7, dtype=torch.int32, device="cuda")
        groups, shared = torch.tensor([0, 6], dtype=torch.int32, device="cuda"), torch.tensor([64], dtype=torch.int32, device="cuda")
        x = torch.randn(6, 8 + 2 + 2, 64, generator=g, device="cuda").to(torch.bfloat16)
        q = torch.empty(6, 8, 64, dtype=torch.bfloat16, device="cuda")
        out, lse = torch.zeros(2, 6, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(6, 8, device="cuda")
        mass = torch.zeros(6, 12 * 16, device="cuda")

        def step():
            rotary(rope, cache.lens, [(x[:, :8], q)])
            cache.extend(slots, ones)
            cache.copy_pages()
            for layer in range(2):
                cache.append(layer, x[:, 8:10], x[:, 10:], starts, rope=rope)
                cache.attend_shared(layer, q, starts, groups, shared, out=out[layer], lse=lse, max_new=1)
                cache.weigh(layer, q, starts, lse, mass, begin=layer == 0, max_new=1)

        def shorten():
            cache.evict(slots, torch.full_like(slots, 75), mass, first=4, recent=8)
            cache.move_tokens()

        return cache, (out, mass), step, shorten

    a, got, step_a, shorten_a = make()
    b, want, step_b, shorten_b = make()
    for _ in range(20):
        step_b()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step_a()
    for _ in range(20):
        graph.replay()
    shorten_a()
    shorten_b()
    torch.cuda.synchronize()
    assert a.status() == b.status() == (0, 0)
    assert a.lens.tolist() == [75] * 6
    for x, y in [(a.lens, b.lens), (a.tables, b.tables), (a.refs, b.refs), (a.codes, b.codes), (a.scales, b.scales), *zip(got, want)]:
        assert torch.equal(x, y)
    assert bool(got[0].any()) and bool(got[1].any())
