"""kvl_pages_* against a sequential restatement of their documentation."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import layer_wise_paged_gb300 as kvl
from tests import _quant as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvl.build()
    kvl.lib()


class Plain:
    """The bookkeeping, one entry after another."""

    def __init__(self, tables, lens, refs, B):
        self.t, self.n, self.r, self.B = tables.copy(), lens.copy(), refs.copy(), B
        self.pairs = []

    def pages(self, s):
        return -(-int(self.n[s]) // self.B)

    def extend(self, slots, counts):
        shared, free = self.r > 1, [int(i) for i in np.flatnonzero(self.r == 0)]
        plan, need = [], 0
        for s, c in zip(slots, counts):
            first = self.pages(s)
            cow = c > 0 and self.n[s] % self.B and shared[self.t[s, first - 1]]
            first -= bool(cow)
            last = -(-(int(self.n[s]) + c) // self.B)
            if last > self.t.shape[1]:
                return False
            plan.append((s, first, last, cow))
            need += last - first
        self.pairs = []
        if need > len(free):
            return False
        for (s, first, last, cow), c in zip(plan, counts):
            for k in range(first, last):
                p = free.pop(0)
                if cow and k == first:
                    self.pairs.append((int(self.t[s, k]), p))
                    self.r[self.t[s, k]] -= 1
                self.t[s, k] = p
                self.r[p] = 1
            self.n[s] += c
        return True

    def fork(self, parents, children):
        for a, c in zip(parents, children):
            k = self.pages(a)
            self.t[c, :k] = self.t[a, :k]
            self.n[c] = self.n[a]
            for p in self.t[a, :k]:
                self.r[p] += 1

    def free(self, slots):
        for s in slots:
            for p in self.t[s, :self.pages(s)]:
                self.r[p] -= 1
            self.n[s] = 0

    def compact(self):
        live = [int(i) for i in np.flatnonzero(self.r > 0)]
        holes = [int(i) for i in np.flatnonzero(self.r <= 0) if i < len(live)]
        move = dict(zip([i for i in live if i >= len(live)], holes))
        self.pairs = list(move.items())
        for s in range(len(self.n)):
            for k in range(self.pages(s)):
                self.t[s, k] = move.get(int(self.t[s, k]), self.t[s, k])
        for a, b in self.pairs:
            self.r[b], self.r[a] = self.r[a], 0


def make(seed, slots, N, B, W, L=2, H=2, d=16):
    from layer_wise_paged_gb300.cache import QuantCache
    c = QuantCache.empty(L, H, d, B, N, slots, W)
    g = torch.Generator(device="cuda").manual_seed(seed)
    c.codes.copy_(torch.randint(0, 256, c.codes.shape, generator=g, device="cuda", dtype=torch.uint8))
    c.scales.copy_(torch.rand(c.scales.shape, generator=g, device="cuda"))
    return c, Plain(c.tables.cpu().numpy(), c.lens.cpu().numpy(), c.refs.cpu().numpy(), B)


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def same(c, p, what):
    assert np.array_equal(c.tables.cpu().numpy(), p.t), what
    assert np.array_equal(c.lens.cpu().numpy(), p.n), what
    assert np.array_equal(c.refs.cpu().numpy(), p.r), what
    n = int(c.n_pairs)
    assert [tuple(x) for x in c.pairs[:n].tolist()] == [(int(a), int(b)) for a, b in p.pairs], what


@pytest.mark.parametrize("seed,slots,N,B", [(1, 6, 40, 4), (2, 50, 900, 16), (3, 3, 9000, 1), (4, 2100, 20000, 16),
                                             (5, 1500, 8192, 2), (6, 40, 257, 64)])
def test_random_lives(seed, slots, N, B):
    """Random steps of extend, fork, free, compact; tables, lengths, references, pairs and the
    copied bytes follow the restatement."""
    rng = np.random.default_rng(seed)
    W = max(4, 2 * N // slots)
    c, p = make(seed, slots, N, B, W)
    for step in range(30):
        empty, full = np.flatnonzero(p.n == 0), np.flatnonzero(p.n > 0)
        what = ["extend", "extend", "fork", "free", "compact"][rng.integers(5)]
        name = f"step {step}: {what}"
        if what == "extend":
            s = rng.permutation(slots)[:rng.integers(1, slots + 1)]
            n = [int(x) for x in rng.integers(0, max(2, N * B // (2 * slots)), len(s))]
            c.extend(ints(s), ints(n))
            fits = p.extend([int(x) for x in s], n)
            if not fits:
                p.pairs = []
            assert c.status()[0] == (kvl.KVL_OK if fits else kvl.KVL_ERANGE), name
            c.reset_status()
        elif what == "fork" and len(empty) and len(full):
            k = min(len(empty), int(rng.integers(1, 2 * len(full) + 1)))
            kids, dads = rng.permutation(empty)[:k], full[rng.integers(0, len(full), k)]
            c.fork(ints(dads), ints(kids))
            p.fork([int(x) for x in dads], [int(x) for x in kids])
        elif what == "free" and len(full):
            s = rng.permutation(full)[:rng.integers(1, len(full) + 1)]
            c.free(ints(s))
            p.free([int(x) for x in s])
        elif what == "compact":
            c.compact()
            p.compact()
        same(c, p, name)
        if what in ("extend", "compact"):
            codes, scales = c.codes.clone(), c.scales.clone()
            for a, b in p.pairs:
                codes[:, :, b], scales[:, :, b] = c.codes[:, :, a], c.scales[:, :, a]
            c.copy_pages()
            assert torch.equal(c.codes, codes) and torch.equal(c.scales, scales), name
        assert c.status() == (0, 0), name


@pytest.mark.parametrize("L,H,d,B", [(1, 1, 16, 1), (3, 5, 80, 24), (2, 8, 128, 64), (1, 2, 256, 200)])
def test_copies_of_every_page_size(L, H, d, B):
    c, _ = make(3, 4, 60, B, 8, L, H, d)
    g = torch.Generator().manual_seed(1)
    ids = torch.randperm(60, generator=g)
    src, dst = ids[:25].cuda(), ids[25:50].cuda()
    c.pairs[:25, 0], c.pairs[:25, 1] = src.int(), dst.int()
    c.n_pairs.fill_(25)
    codes, scales = c.codes.clone(), c.scales.clone()
    codes[:, :, dst], scales[:, :, dst] = codes[:, :, src], scales[:, :, src]
    c.copy_pages()
    assert torch.equal(c.codes, codes) and torch.equal(c.scales, scales)
    assert c.status() == (0, 0)


def test_shared_last_page_copied_for_each():
    """Parent and children extend in one call: the page was shared by all when it began, so each
    gets its own copy and the page falls free."""
    c, p = make(1, 8, 32, 4, 6)
    c.extend(ints([0]), ints([6]))
    p.extend([0], [6])
    c.fork(ints([0, 0]), ints([1, 2]))
    p.fork([0, 0], [1, 2])
    same(c, p, "fork")
    c.extend(ints([2, 0, 1]), ints([1, 3, 0]))
    p.extend([2, 0, 1], [1, 3, 0])
    same(c, p, "extend")
    assert int(c.n_pairs) == 2 and c.status() == (0, 0)


def test_problems_leave_the_state_alone():
    c, p = make(1, 8, 32, 4, 6)
    c.extend(ints([0, 1]), ints([6, 9]))
    p.extend([0, 1], [6, 9])
    for slots, counts, code in [([2, 3], [24, 300], kvl.KVL_ERANGE),     # a table row is too short
                                ([2, 3, 4, 5, 6], [24] * 5, kvl.KVL_ERANGE),  # 30 pages, 27 free
                                ([2, 2], [1, 1], kvl.KVL_EDUP),
                                ([9], [1], kvl.KVL_EINVAL), ([-1], [1], kvl.KVL_EINVAL), ([2], [-1], kvl.KVL_EINVAL)]:
        c.extend(ints(slots), ints(counts))
        p.pairs = []
        same(c, p, (slots, counts))
        assert c.status()[0] == code, (slots, counts)
        c.reset_status()
    c.fork(ints([0, 0, 77]), ints([1, 0, 3]))  # a child that holds tokens, itself, no such parent
    same(c, p, "fork")
    assert c.status() == (kvl.KVL_EINVAL, 0)
    c.reset_status()
    c.free(ints([0, 0, 5]))  # twice, and an empty one: the first counts
    p.free([0])
    same(c, p, "free")
    c.pairs[0] = ints([3, 32])
    c.n_pairs.fill_(1)
    before = c.codes.clone()
    c.copy_pages()
    assert c.status() == (kvl.KVL_ERANGE, 0) and torch.equal(before, c.codes)


def test_empty_calls():
    c, p = make(1, 4, 16, 4, 4)
    c.extend(ints([]), ints([]))
    c.free(ints([]))
    c.fork(ints([]), ints([]))
    c.compact()
    c.copy_pages()
    same(c, p, "nothing")
    assert c.status() == (0, 0)


def test_cache_blocks_move_through_the_copy_calls():
    """Codes and scales are pools of the layer-wise copy calls: gathered into objects and scattered
    back into another pool, a sequence attends to the same result."""
    from layer_wise_paged_gb300.batch import Batch
    from types import SimpleNamespace
    L, H, d, B, n = 2, 4, 64, 16, 75
    cache = Q.make_cache(2, L, H, d, B, [n], poison=False)
    dev = Q.on_gpu(cache)
    N, nblk = cache["codes"].shape[2], -(-n // B)
    other = Q.on_gpu({**cache, "codes": torch.zeros_like(cache["codes"]), "scales": torch.zeros_like(cache["scales"])})
    for t, rows, to, tok in ((dev.codes, H * d, other.codes, n), (dev.scales, 4 * H, other.scales, nblk)):
        blk = B if tok == n else 1
        obj = torch.zeros(L * 2 * nblk * blk * rows, dtype=torch.uint8, device="cuda")
        # the sequence as a request whose tokens all come from (unused) miss rows
        miss = torch.zeros(L * tok * 2 * rows, dtype=torch.uint8, device="cuda")
        req = SimpleNamespace(t_hit=0, t_miss=tok, hit_off=0, hit_src_blocks=0, hit_block_stride=0, hit_token_stride=0,
                              hit_layer_stride=0, src_table_off=-1, miss_off=0, miss_token_stride=2 * rows,
                              miss_layer_stride=tok * 2 * rows, obj_off=0, obj_layer_stride=2 * nblk * blk * rows,
                              obj_plane_stride=nblk * blk * rows, obj_block_stride=blk * rows)
        b = Batch((L, 2, blk, rows, N), [req], None, miss, obj, dev.tables[0, :nblk].contiguous())
        b.plan()
        for l in range(L):
            b.gather(l, t.view(torch.uint8).view(-1))
            b.scatter_back(l, to.view(torch.uint8).view(-1))
        assert b.status() == (0, 0)
    q = torch.randn((1, 8, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    starts = ints([0, 1])
    for l in range(L):
        assert torch.equal(dev.attend(l, q, starts), other.attend(l, q, starts))
