"""The rows up to which attention shares prefixes stand in the header, which the kernels use, and in the binding."""
from __future__ import annotations

import re
from pathlib import Path

import layer_wise_paged_gb300 as kvl
from layer_wise_paged_gb300 import cache

ROOT = Path(__file__).resolve().parent.parent


def test_the_binding_has_the_headers_number():
    found = re.findall(r"#define KVL_SHARED_ROWS (\d+)", (ROOT / "include" / "kvl.h").read_text())
    assert found == [str(kvl.KVL_SHARED_ROWS)] and cache.KVL_SHARED_ROWS == kvl.KVL_SHARED_ROWS


def test_a_call_of_as_many_rows_needs_parts():
    """Refused before any device work (with one row more the library would need no parts, and launch)."""
    from tests.test_more_host import FAKE, LOTS, attend_shared, attention, cache as make_cache, seqs
    kvl.build()
    most = kvl.KVL_SHARED_ROWS // (8 // make_cache().n_kv_heads)
    assert attend_shared(kvl.lib(), s=seqs(n_rows=1000), a=attention(max_new=most), ws=FAKE, ws_bytes=LOTS,
                         parts_bytes=0) == kvl.KVL_EINVAL
