"""Shared prefixes, weights of cached tokens and eviction without a GPU: struct layouts, and refusals on the host
before any device work."""
from __future__ import annotations

import ctypes
import math
import subprocess

import pytest

import layer_wise_paged_gb300 as kvl
from tests.test_quant_host import FAKE, ROOT, attention, cache, seqs

STRUCTS = [kvl.kvl_shared, kvl.kvl_weighing, kvl.kvl_eviction, kvl.kvl_moves]


@pytest.fixture(scope="module")
def lib():
    kvl.build()
    return kvl.lib()


def test_struct_layouts_match_the_header(tmp_path):
    lines = []
    for t in STRUCTS:
        lines.append(f'printf("{t.__name__} %zu\\n", sizeof({t.__name__}));')
        lines += [f'printf("{t.__name__}.{f[0]} %zu\\n", offsetof({t.__name__}, {f[0].rstrip("_")}));' for f in t._fields_]
    (tmp_path / "l.c").write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kvl.h"\nint main(void) {' +
                                  "\n".join(lines) + "return 0; }")
    subprocess.run(["gcc", "-std=c99", "-I", str(ROOT / "include"), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")],
                   check=True)
    got = dict(x.split() for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    for t in STRUCTS:
        assert int(got[t.__name__]) == ctypes.sizeof(t)
        for f in t._fields_:
            assert int(got[f"{t.__name__}.{f[0]}"]) == getattr(t, f[0]).offset, (t, f)


def changed(x, k):
    for n, v in k.items():
        setattr(x, n, v)
    return x


def shared(**k):
    return changed(kvl.kvl_shared(1, 0, FAKE, FAKE), k)


def weighing(**k):
    return changed(kvl.kvl_weighing(kvl.kvl_rows(FAKE, 8 * 256, 256), FAKE, FAKE, FAKE, 100, 100, 100, 8, kvl.KVL_TYPE_BFLOAT, 0.1,
                                    1, 0, 0, 0, 0), k)


def eviction(**k):
    return changed(kvl.kvl_eviction(FAKE, FAKE, 100, 100, 4, 8), k)


def moves(**k):
    return changed(kvl.kvl_moves(FAKE, FAKE, FAKE, FAKE), k)


def pages(**k):
    return changed(kvl.kvl_pages(64, 16, 4, 8, FAKE, FAKE, FAKE, FAKE, FAKE), k)


LOTS = 1 << 40


def attend_shared(lib, c=None, layer=0, s=None, sh=None, a=None, ws=FAKE, ws_bytes=LOTS, parts=FAKE, parts_bytes=LOTS, rep=FAKE):
    return lib.kvl_attend_shared(c or cache(), layer, s or seqs(), sh or shared(), a or attention(max_new=1), ws, ws_bytes,
                                 parts, parts_bytes, rep, None)


def test_attend_shared_refusals(lib):
    for bad in (dict(n_groups=-1), dict(n_groups=(1 << 20) + 1), dict(reserved=1), dict(groups=None), dict(tokens=None)):
        assert attend_shared(lib, sh=shared(**bad)) == kvl.KVL_EINVAL, bad
    for bad in (dict(groups=FAKE + 2), dict(tokens=FAKE + 1)):
        assert attend_shared(lib, sh=shared(**bad)) == kvl.KVL_EALIGN, bad
    assert lib.kvl_attend_shared(cache(), 0, seqs(), None, attention(), FAKE, LOTS, FAKE, LOTS, FAKE, None) == kvl.KVL_EINVAL
    for bad in (dict(n_heads=6), dict(type=kvl.KVL_TYPE_FLOAT), dict(sm_scale=math.nan), dict(window=-1), dict(max_new=-1)):
        assert attend_shared(lib, a=attention(**bad)) == kvl.KVL_EINVAL, bad
    assert attend_shared(lib, c=cache(head_dim=24)) == kvl.KVL_EINVAL
    assert attend_shared(lib, s=seqs(lens=None)) == kvl.KVL_EINVAL
    assert attend_shared(lib, layer=2) == kvl.KVL_EINVAL
    assert attend_shared(lib, ws=None) == kvl.KVL_EINVAL and attend_shared(lib, ws_bytes=100) == kvl.KVL_EINVAL
    assert attend_shared(lib, parts=None) == kvl.KVL_EINVAL and attend_shared(lib, parts=FAKE + 8) == kvl.KVL_EALIGN
    assert attend_shared(lib, rep=FAKE + 8) == kvl.KVL_EALIGN
    n = lib.kvl_attend_shared_parts_bytes(cache(), 2, 1, 5, 8)
    assert n >= 5 * 8 * 130 * 4
    assert attend_shared(lib, parts_bytes=n - 1) == kvl.KVL_EINVAL
    for bad in ((cache(head_dim=0), 2, 1, 5, 8), (cache(), 2, 1, -1, 8), (cache(), 2, 1, 5, 0), (cache(), 2, 1, 1 << 31, 8),
                (cache(), 2, -1, 5, 8), (cache(), -1, 1, 5, 8), (cache(), 2, 1, 5, 6)):
        assert lib.kvl_attend_shared_parts_bytes(*bad) == 0
    for nothing in (dict(n_rows=0), dict(n_seq=0)):
        assert attend_shared(lib, s=seqs(**nothing), parts=None, ws=None) == kvl.KVL_OK


def test_weigh_refusals(lib):
    def call(w=None, c=None, layer=0, s=None, ws=FAKE, n=LOTS, rep=FAKE):
        return lib.kvl_weigh(c or cache(), layer, s or seqs(), w or weighing(), ws, n, rep, None)
    for bad in (dict(n_heads=6), dict(n_heads=0), dict(type=kvl.KVL_TYPE_FLOAT), dict(sm_scale=0.0), dict(sm_scale=math.inf),
                dict(causal=2), dict(window=-1), dict(window=5, causal=0), dict(max_new=-1), dict(begin=2), dict(reserved=1),
                dict(lse=None), dict(mass_in=None), dict(mass_out=None), dict(in_stride=99), dict(out_stride=-5), dict(tokens=0),
                dict(q=kvl.kvl_rows(None, 256, 256))):
        assert call(weighing(**bad)) == kvl.KVL_EINVAL, bad
    for bad in (dict(lse=FAKE + 2), dict(mass_in=FAKE + 1), dict(mass_out=FAKE + 3), dict(q=kvl.kvl_rows(FAKE + 8, 256, 256))):
        assert call(weighing(**bad)) == kvl.KVL_EALIGN, bad
    assert lib.kvl_weigh(cache(), 0, seqs(), None, FAKE, LOTS, FAKE, None) == kvl.KVL_EINVAL
    assert call(c=cache(codes=None)) == kvl.KVL_EINVAL and call(s=seqs(tables=None)) == kvl.KVL_EINVAL
    assert call(layer=-1) == kvl.KVL_EINVAL and call(rep=FAKE + 4) == kvl.KVL_EALIGN
    assert call(ws=None) == kvl.KVL_EINVAL and call(ws=FAKE + 8) == kvl.KVL_EALIGN
    n = lib.kvl_weigh_workspace_bytes(cache(), 2, 5, 8, 0)
    assert n > 0 and call(n=n - 1) == kvl.KVL_EINVAL
    for bad in ((cache(head_dim=0), 2, 5, 8, 0), (cache(), -1, 5, 8, 0), (cache(), 2, -1, 8, 0), (cache(), 2, 5, 0, 0),
                (cache(), 2, 5, 8, -1)):
        assert lib.kvl_weigh_workspace_bytes(*bad) == 0
    group = 64  # rows of a KV head are counted in 32 bits
    rows = (2**31 - 256) // group
    assert call(weighing(n_heads=4 * group), s=seqs(n_rows=rows)) == kvl.KVL_EINVAL
    for nothing in (dict(n_rows=0), dict(n_seq=0)):
        assert call(s=seqs(**nothing), ws=None) == kvl.KVL_OK


def test_evict_refusals(lib):
    def call(p=None, n=1, slots=FAKE, e=None, m=None, rep=FAKE):
        return lib.kvl_pages_evict(p or pages(), n, slots, e or eviction(), m or moves(), rep, None)
    for bad in (dict(pool_blocks=0), dict(block_tokens=0), dict(n_slots=0), dict(table_stride=0), dict(tables=None),
                dict(lens=None), dict(refs=None)):
        assert call(pages(**bad)) == kvl.KVL_EINVAL, bad
    for bad in (dict(keep=None), dict(first=-1), dict(recent=-1), dict(mass_stride=99), dict(tokens=0)):
        assert call(e=eviction(**bad)) == kvl.KVL_EINVAL, bad
    for bad in (dict(from_=None), dict(to=None), dict(at=None), dict(n=None)):
        assert call(m=moves(**bad)) == kvl.KVL_EINVAL, bad
    for bad in (dict(from_=FAKE + 4), dict(to=FAKE + 2), dict(at=FAKE + 1), dict(n=FAKE + 3)):
        assert call(m=moves(**bad)) == kvl.KVL_EALIGN, bad
    assert call(n=5) == kvl.KVL_EINVAL and call(n=-1) == kvl.KVL_EINVAL and call(slots=None) == kvl.KVL_EINVAL
    assert lib.kvl_pages_evict(pages(), 1, FAKE, None, moves(), FAKE, None) == kvl.KVL_EINVAL
    assert lib.kvl_pages_evict(pages(), 1, FAKE, eviction(), None, FAKE, None) == kvl.KVL_EINVAL
    assert call(slots=FAKE + 2) == kvl.KVL_EALIGN and call(e=eviction(mass=FAKE + 2)) == kvl.KVL_EALIGN
    assert call(rep=FAKE + 8) == kvl.KVL_EALIGN


def test_move_refusals(lib):
    def call(c=None, m=None, most=5, rep=FAKE):
        return lib.kvl_tokens_move(c or cache(), m or moves(), most, rep, None)
    assert call(cache(head_dim=8)) == kvl.KVL_EINVAL
    assert call(most=-1) == kvl.KVL_EINVAL and call(most=1 << 31) == kvl.KVL_EINVAL
    assert call(m=moves(from_=None)) == kvl.KVL_EINVAL and call(m=moves(to=FAKE + 2)) == kvl.KVL_EALIGN
    assert call(rep=FAKE + 4) == kvl.KVL_EALIGN
    assert call(most=0) == kvl.KVL_OK


def test_launch_counts(lib):
    assert [kvl.kvl_launches_per_call(w) for w in (12, 13, 14, 15, 16)] == [3, 2, 2, 1, 0]
