"""The 8-bit cache's entry points without a GPU: struct layouts, host-side refusals before any
device work, and the rotary frequencies (host work)."""
from __future__ import annotations

import ctypes
import math
import subprocess
from pathlib import Path

import numpy as np
import pytest

import layer_wise_paged_gb300 as kvl

ROOT = Path(__file__).resolve().parent.parent
FAKE = 1 << 20  # never dereferenced: every call below is refused on the host


@pytest.fixture(scope="module")
def lib():
    kvl.build()
    return kvl.lib()


STRUCTS = [kvl.kvl_cache, kvl.kvl_sequences, kvl.kvl_rows, kvl.kvl_rope, kvl.kvl_attention, kvl.kvl_pages]


def test_struct_layouts_match_the_header(tmp_path):
    lines = []
    for t in STRUCTS:
        lines.append(f'printf("{t.__name__} %zu\\n", sizeof({t.__name__}));')
        lines += [f'printf("{t.__name__}.{f[0]} %zu\\n", offsetof({t.__name__}, {f[0]}));' for f in t._fields_]
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


def cache(**k):
    c = kvl.kvl_cache(2, 4, 128, 16, 64, kvl.KVL_CODE_FLOAT, 0, FAKE, FAKE)
    for n, v in k.items():
        setattr(c, n, v)
    return c


def seqs(**k):
    s = kvl.kvl_sequences(2, 2, 5, 8, FAKE, None, FAKE, None, FAKE)
    for n, v in k.items():
        setattr(s, n, v)
    return s


def attention(**k):
    r = kvl.kvl_rows(FAKE, 8 * 256, 256)
    a = kvl.kvl_attention(r, r, None, 8, kvl.KVL_TYPE_BFLOAT, 0.1, 1, 0, 0)
    for n, v in k.items():
        setattr(a, n, v)
    return a


BAD_CACHE = [dict(n_layers=0), dict(n_kv_heads=0), dict(head_dim=0), dict(head_dim=24), dict(head_dim=272),
             dict(block_tokens=0), dict(pool_blocks=0), dict(pool_blocks=1 << 31), dict(code_type=2), dict(reserved=1),
             dict(codes=None), dict(scales=None)]
BAD_SEQS = [dict(n_seq=-1), dict(n_slots=-1), dict(n_rows=-1), dict(n_rows=1 << 31), dict(tables=None), dict(lens=None),
            dict(starts=None), dict(table_stride=0), dict(n_seq=3)]


@pytest.mark.parametrize("bad", BAD_CACHE, ids=str)
def test_bad_caches(lib, bad):
    c = cache(**bad)
    assert lib.kvl_attend_workspace_bytes(c) == 0
    r = kvl.kvl_rows(FAKE, 1024, 256)
    assert lib.kvl_attend(c, 0, seqs(), attention(), FAKE, 1 << 40, FAKE, None) == kvl.KVL_EINVAL
    assert lib.kvl_cache_append(c, 0, seqs(), 0, r, r, None, FAKE, None) == kvl.KVL_EINVAL
    assert lib.kvl_pages_copy(c, FAKE, FAKE, 5, FAKE, None) == kvl.KVL_EINVAL


@pytest.mark.parametrize("bad", BAD_SEQS, ids=str)
def test_bad_sequences(lib, bad):
    r = kvl.kvl_rows(FAKE, 1024, 256)
    assert lib.kvl_attend(cache(), 0, seqs(**bad), attention(), FAKE, 1 << 40, FAKE, None) == kvl.KVL_EINVAL
    assert lib.kvl_cache_append(cache(), 0, seqs(**bad), 0, r, r, None, FAKE, None) == kvl.KVL_EINVAL


@pytest.mark.parametrize("bad,code", [
    (dict(n_heads=6), kvl.KVL_EINVAL), (dict(n_heads=0), kvl.KVL_EINVAL), (dict(type=kvl.KVL_TYPE_FLOAT), kvl.KVL_EINVAL),
    (dict(sm_scale=0.0), kvl.KVL_EINVAL), (dict(sm_scale=math.nan), kvl.KVL_EINVAL), (dict(sm_scale=math.inf), kvl.KVL_EINVAL),
    (dict(causal=2), kvl.KVL_EINVAL),
    (dict(window=-1), kvl.KVL_EINVAL), (dict(window=5, causal=0), kvl.KVL_EINVAL), (dict(max_new=-1), kvl.KVL_EINVAL),
    (dict(q=kvl.kvl_rows(None, 256, 256)), kvl.KVL_EINVAL), (dict(q=kvl.kvl_rows(FAKE + 8, 256, 256)), kvl.KVL_EALIGN),
    (dict(out=kvl.kvl_rows(FAKE, 256, 8)), kvl.KVL_EALIGN), (dict(out=kvl.kvl_rows(FAKE, 264, 256)), kvl.KVL_EALIGN),
    (dict(lse=FAKE + 2), kvl.KVL_EALIGN)], ids=str)
def test_bad_attention(lib, bad, code):
    assert lib.kvl_attend(cache(), 0, seqs(), attention(**bad), FAKE, 1 << 40, FAKE, None) == code


def test_attend_refusals(lib):
    need = lib.kvl_attend_workspace_bytes(cache())
    assert need >= kvl.KVL_ATTEND_ZERO_BYTES
    for layer in (-1, 2):
        assert lib.kvl_attend(cache(), layer, seqs(), attention(), FAKE, need, FAKE, None) == kvl.KVL_EINVAL
    assert lib.kvl_attend(cache(), 0, seqs(), attention(), FAKE, need - 1, FAKE, None) == kvl.KVL_EINVAL
    assert lib.kvl_attend(cache(), 0, seqs(), attention(), None, need, FAKE, None) == kvl.KVL_EINVAL
    assert lib.kvl_attend(cache(), 0, seqs(), attention(), FAKE + 4, need, FAKE, None) == kvl.KVL_EALIGN
    assert lib.kvl_attend(cache(), 0, seqs(), attention(), FAKE, need, FAKE + 8, None) == kvl.KVL_EALIGN
    assert lib.kvl_attend(cache(codes=FAKE + 1), 0, seqs(), attention(), FAKE, need, FAKE, None) == kvl.KVL_EALIGN
    assert lib.kvl_attend(cache(), 0, seqs(lens=FAKE + 1), attention(), FAKE, need, FAKE, None) == kvl.KVL_EALIGN
    assert lib.kvl_attend(cache(), 0, seqs(), None, FAKE, need, FAKE, None) == kvl.KVL_EINVAL
    for nothing in (dict(n_rows=0), dict(n_seq=0)):  # no work: nothing is read, nothing launched
        assert lib.kvl_attend(cache(), 0, seqs(**nothing), attention(), FAKE, need, FAKE, None) == kvl.KVL_OK


def test_append_refusals(lib):
    r = kvl.kvl_rows(FAKE, 1024, 256)

    def call(layer=0, type_=0, k=r, v=r, rope=None, rep=FAKE):
        return lib.kvl_cache_append(cache(), layer, seqs(), type_, k, v, rope, rep, None)
    assert call(layer=2) == kvl.KVL_EINVAL and call(type_=3) == kvl.KVL_EINVAL
    assert call(k=kvl.kvl_rows(None, 0, 0)) == kvl.KVL_EINVAL
    assert call(v=kvl.kvl_rows(FAKE, 1000, 256)) == kvl.KVL_EALIGN
    assert call(rep=FAKE + 4) == kvl.KVL_EALIGN
    for rope in (kvl.kvl_rope(FAKE, 0, 0, 1.0, 0), kvl.kvl_rope(FAKE, 12, 0, 1.0, 0), kvl.kvl_rope(FAKE, 72, 0, 1.0, 0),
                 kvl.kvl_rope(FAKE, 64, 2, 1.0, 0), kvl.kvl_rope(None, 64, 0, 1.0, 0), kvl.kvl_rope(FAKE, 64, 0, 1.0, 1)):
        assert call(rope=rope) == kvl.KVL_EINVAL


def test_rotary_refusals(lib):
    r = (kvl.kvl_rows * 1)(kvl.kvl_rows(FAKE, 1024, 256))
    heads = (ctypes.c_int32 * 1)(4)
    good = kvl.kvl_rope(FAKE, 64, 0, 1.0, 0)

    def call(rope=good, rows=3, dim=128, type_=0, pos=FAKE, n=1, src=r, dst=r, h=heads, inverse=0):
        return lib.kvl_rotary(rope, rows, dim, type_, pos, n, src, dst, h, inverse, None)
    for bad in (dict(rows=-1), dict(dim=132), dict(dim=0), dict(dim=520), dict(type_=3), dict(pos=None), dict(n=0),
                dict(n=5), dict(inverse=2), dict(h=(ctypes.c_int32 * 1)(0)), dict(rope=kvl.kvl_rope(FAKE, 66, 0, 1.0, 0)),
                dict(rope=kvl.kvl_rope(FAKE, 6, 0, 1.0, 0)), dict(rope=kvl.kvl_rope(None, 64, 0, 1.0, 0)), dict(dim=126),
                dict(dst=(kvl.kvl_rows * 1)(kvl.kvl_rows(FAKE, 2048, 256)))):  # the same memory, other strides
        assert call(**bad) == kvl.KVL_EINVAL, bad
    assert call(src=(kvl.kvl_rows * 1)(kvl.kvl_rows(FAKE + 8, 1024, 256))) == kvl.KVL_EALIGN
    assert call(pos=FAKE + 2) == kvl.KVL_EALIGN
    assert call(rows=0) == kvl.KVL_OK


def test_pages_refusals(lib):
    def pages(**k):
        p = kvl.kvl_pages(64, 16, 4, 8, FAKE, FAKE, FAKE, FAKE, FAKE)
        for n, v in k.items():
            setattr(p, n, v)
        return p
    for bad in (dict(pool_blocks=0), dict(pool_blocks=1 << 31), dict(block_tokens=0), dict(n_slots=0),
                dict(n_slots=(1 << 20) + 1), dict(table_stride=0), dict(tables=None), dict(lens=None), dict(refs=None),
                dict(pairs=None), dict(n_pairs=None)):
        p = pages(**bad)
        assert lib.kvl_pages_extend(p, 1, FAKE, FAKE, FAKE, None) == kvl.KVL_EINVAL, bad
        assert lib.kvl_pages_fork(p, 1, FAKE, FAKE, FAKE, None) == kvl.KVL_EINVAL, bad
        assert lib.kvl_pages_free(p, 1, FAKE, FAKE, None) == kvl.KVL_EINVAL, bad
        assert lib.kvl_pages_compact(p, FAKE, None) == kvl.KVL_EINVAL, bad
    p = pages()
    assert lib.kvl_pages_extend(p, 5, FAKE, FAKE, FAKE, None) == kvl.KVL_EINVAL  # more entries than slots
    assert lib.kvl_pages_extend(p, 1, FAKE, None, FAKE, None) == kvl.KVL_EINVAL
    assert lib.kvl_pages_free(p, -1, FAKE, FAKE, None) == kvl.KVL_EINVAL
    assert lib.kvl_pages_extend(p, 1, FAKE + 2, FAKE, FAKE, None) == kvl.KVL_EALIGN
    assert lib.kvl_pages_compact(pages(pairs=FAKE + 4), FAKE, None) == kvl.KVL_EALIGN
    assert lib.kvl_pages_compact(p, FAKE + 8, None) == kvl.KVL_EALIGN
    assert lib.kvl_pages_fork(p, 0, None, None, None, None) == kvl.KVL_OK
    assert lib.kvl_pages_copy(cache(), None, FAKE, 5, FAKE, None) == kvl.KVL_EINVAL
    assert lib.kvl_pages_copy(cache(), FAKE + 4, FAKE, 5, FAKE, None) == kvl.KVL_EALIGN
    assert lib.kvl_pages_copy(cache(), FAKE, FAKE, -1, FAKE, None) == kvl.KVL_EINVAL
    assert lib.kvl_pages_copy(cache(), FAKE, FAKE, 0, FAKE, None) == kvl.KVL_OK
    assert lib.kvl_report_reset(None, None) == kvl.KVL_EINVAL
    assert lib.kvl_report_reset(FAKE + 8, None) == kvl.KVL_EALIGN


def test_rotary_frequencies(lib):
    from layer_wise_paged_gb300.cache import rope_frequencies
    i = np.arange(64)
    plain = 500000.0 ** (-i / 64)
    f, g = rope_frequencies(128, 500000.0)
    assert np.allclose(f, plain, rtol=2.0 ** -23) and g == 1.0
    f, g = rope_frequencies(128, 500000.0, "linear", factor=4.0, scale_gain=True)
    assert np.allclose(f, plain / 4, rtol=2.0 ** -23) and math.isclose(g, 0.1 * math.log(4.0) + 1, rel_tol=1e-6)
    f, _ = rope_frequencies(128, 500000.0, "base", factor=8.0)
    assert f[0] == 1.0 and np.isclose(f[-1], plain[-1] / 8, rtol=1e-6)  # the slowest pair slows by the factor
    f, _ = rope_frequencies(128, 500000.0, "wavelength", factor=8.0, low=1.0, high=4.0, trained_context=8192)
    turns = 8192 * plain / (2 * math.pi)
    assert np.allclose(f[turns >= 4], plain[turns >= 4], rtol=2.0 ** -22)
    assert np.allclose(f[turns <= 1], plain[turns <= 1] / 8, rtol=2.0 ** -22)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and (f[mid] < plain[mid]).all() and (f[mid] > plain[mid] / 8).all()
    out = (ctypes.c_float * 4)()
    call = lib.kvl_rotary_frequencies
    for bad in ((9, 1e4, 4, 1.0, 1.0, 4.0, 8192.0), (0, -1.0, 4, 1.0, 1.0, 4.0, 8192.0), (0, 1e4, 0, 1.0, 1.0, 4.0, 8192.0),
                (1, 1e4, 4, 0.0, 1.0, 4.0, 8192.0), (2, 1e4, 1, 2.0, 1.0, 4.0, 8192.0), (3, 1e4, 4, 2.0, 4.0, 4.0, 8192.0),
                (3, 1e4, 4, 2.0, 1.0, 4.0, 0.0)):
        assert call(*bad, 0, ctypes.addressof(out), None) == kvl.KVL_EINVAL, bad
    assert call(0, 1e4, 4, 1.0, 1.0, 4.0, 8192.0, 0, None, None) == kvl.KVL_EINVAL


def test_attend_refuses_rows_past_32_bits(lib):
    """Rows of a KV head (rows times grouped heads) are counted in 32 bits."""
    c = cache()
    need = lib.kvl_attend_workspace_bytes(c)
    group = 64
    rows = (2**31 - 256) // group
    a = attention(n_heads=c.n_kv_heads * group)
    assert lib.kvl_attend(c, 0, seqs(n_rows=rows), a, FAKE, need, FAKE, None) == kvl.KVL_EINVAL
    # one row fewer gets past this check, to that of the workspace
    assert lib.kvl_attend(c, 0, seqs(n_rows=rows - 1), a, FAKE + 8, need, FAKE, None) == kvl.KVL_EALIGN
