"""An 8-bit paged KV cache bound to torch device tensors: marshalling around the C ABI.

``QuantCache`` holds the codes, scales and page bookkeeping of a cache and forwards each
step (append, attend, extend, fork, free, compact, page copies) to libkvl.so;
``rotary`` turns rows of heads by their positions.  No step runs here, nothing
synchronises, and every call enqueues on the current stream unless it is given one.
Device-side problems (a page number out of range, too few free pages) are read with
``QuantCache.status()``, which synchronises.

Rows of fresh tokens are tensors [rows, heads, head_dim] whose last dimension is contiguous;
rows and heads may be strided (parts of one fused projection).
"""
from __future__ import annotations

import ctypes
import math
import threading

import numpy as np
import torch

from . import lib as _lib
from . import (KVL_ATTEND_ZERO_BYTES, KVL_CODE_FLOAT, KVL_CODE_INT, KVL_REPORT_BYTES, KVL_ROPE_BASE,
               KVL_ROPE_LINEAR, KVL_ROPE_PLAIN, KVL_ROPE_WAVELENGTH, KVL_TYPE_BFLOAT, KVL_TYPE_FLOAT,
               KVL_TYPE_HALF, check, kvl_attention, kvl_cache, kvl_pages, kvl_read_status,
               kvl_rope, kvl_rows, kvl_sequences)

CODES = {"e4m3": KVL_CODE_FLOAT, "int8": KVL_CODE_INT}
TYPES = {torch.bfloat16: KVL_TYPE_BFLOAT, torch.float16: KVL_TYPE_HALF, torch.float32: KVL_TYPE_FLOAT}
ROPE_KINDS = {"plain": KVL_ROPE_PLAIN, "linear": KVL_ROPE_LINEAR, "base": KVL_ROPE_BASE,
              "wavelength": KVL_ROPE_WAVELENGTH}


# torch.cuda.current_stream without its Stream object (5 us), where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_MOST = 2 ** 31 - 1
_several = None  # whether there is another device than the current one (asked at the first call)


def _stream(stream, device):
    """The handle of the stream a call goes to.  The library launches on the current device, whatever
    the tensors' is."""
    global _several
    if _several is None:
        _several = torch.cuda.device_count() > 1
    if _several and _current_device() != device:
        raise ValueError(f"the tensors are on cuda:{device}, which is not the current device: call within "
                         f"torch.cuda.device({device})")
    if stream is None:
        return _raw_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# The checks below run on every call, some of them on the few-microsecond path of a single
# token: they are plain conditions, and a message is put together only when one fails.

def _ints(t, name, n=None):
    """The address of a contiguous int32 device vector (of n entries)."""
    if t.dtype is not torch.int32 or not t.is_cuda or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous int32 vector in device memory")
    if n is not None and t.shape[0] != n:
        raise ValueError(f"{name}: {n} entries, not {t.shape[0]}")
    return t.data_ptr()


def _rows(r, t, name, heads, dim):
    """Fill the kvl_rows `r` with a [rows, heads, dim] tensor."""
    if t.dim() != 3 or not t.is_cuda or t.dtype not in TYPES:
        raise ValueError(f"{name}: a [rows, heads, dim] device tensor of bf16, f16 or f32")
    _, h, d = t.shape
    if h != heads or d != dim:
        raise ValueError(f"{name}: [rows, {heads}, {dim}], not {tuple(t.shape)}")
    s0, s1, s2 = t.stride()
    if s2 != 1:
        raise ValueError(f"{name}: the last dimension is contiguous")
    z = t.element_size()
    r.data, r.row_stride, r.head_stride = t.data_ptr(), s0 * z, s1 * z


class _Args(threading.local):
    """The C structs of a call, each thread's own: filling their fields takes a few hundred nanoseconds
    where making them anew takes microseconds."""

    def __init__(self, cache=None):
        self.a, self.b = kvl_rows(), kvl_rows()
        self.attn = kvl_attention()
        # (views into the struct: q and out are filled in place)
        self.q, self.out = self.attn.q, self.attn.out
        self.seqs = kvl_sequences()
        self.src, self.dst, self.heads = (kvl_rows * 4)(), (kvl_rows * 4)(), (ctypes.c_int32 * 4)()
        self.sets = [(self.src[i], self.dst[i]) for i in range(4)]
        if cache is not None:
            p = cache._p
            self.seqs.n_slots, self.seqs.table_stride = cache.n_slots, cache.tables.shape[1]
            self.seqs.tables, self.seqs.lens = p.tables, p.lens


_args = _Args()


def _flat(t, dtype, shape, name):
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous() or t.shape != shape:
        raise ValueError(f"{name}: contiguous {dtype} {list(shape)} in device memory")


class Rope:
    """Rotary positions: float32 device frequencies of the pairs, pair layout, gain."""

    def __init__(self, inv_freq, interleaved=False, gain=1.0):
        _flat(inv_freq, torch.float32, (inv_freq.numel(),), "inv_freq")
        self.inv_freq = inv_freq
        self.interleaved, self.gain = bool(interleaved), float(gain)
        self._c = kvl_rope(inv_freq.data_ptr(), inv_freq.shape[0], int(self.interleaved), self.gain, 0)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def make(cls, rot_dim, base=10000.0, kind="plain", factor=1.0, low=1.0, high=4.0, trained_context=8192,
             scale_gain=False, interleaved=False, device="cuda"):
        """Frequencies of rot_dim / 2 pairs (kvl_rotary_frequencies)."""
        f, g = rope_frequencies(rot_dim, base, kind, factor, low, high, trained_context, scale_gain)
        return cls(torch.from_numpy(f).to(device), interleaved, g)


def rope_frequencies(rot_dim, base=10000.0, kind="plain", factor=1.0, low=1.0, high=4.0, trained_context=8192,
                     scale_gain=False):
    """(float32 frequencies, gain) on the host; see kvl_rotary_frequencies in kvl.h."""
    if kind not in ROPE_KINDS or rot_dim <= 0 or rot_dim % 2:
        raise ValueError(f"kind: one of {sorted(ROPE_KINDS)}; rot_dim: a positive even number")
    f, g = np.zeros(rot_dim // 2, np.float32), ctypes.c_float(1.0)
    check(_lib().kvl_rotary_frequencies(ROPE_KINDS[kind], base, rot_dim // 2, factor, low, high, trained_context,
                                       int(bool(scale_gain)), f.ctypes.data, ctypes.byref(g)), "kvl_rotary_frequencies")
    return f, g.value


def rotary(rope, positions, pairs, inverse=False, stream=None):
    """Turn each (x, y) of `pairs` (y may be x), [rows, heads, dim] tensors of one type, by
    int32 `positions` [rows], in one launch.  inverse: the gradient of x from that of y."""
    n = len(pairs)
    if not 1 <= n <= 4:
        raise ValueError("pairs: one to four (source, destination)")
    x0 = pairs[0][0]
    rows, _, dim = x0.shape
    c, heads = _args, _args.heads
    for i, (x, y) in enumerate(pairs):
        if x.dtype is not x0.dtype or y.dtype is not x0.dtype or x.shape[0] != rows or y.shape[0] != rows:
            raise ValueError("pairs: tensors of one type, with the same rows")
        h = heads[i] = x.shape[1]
        src, dst = c.sets[i]
        _rows(src, x, "source", h, dim)
        _rows(dst, y, "destination", h, dim)
    check(_lib().kvl_rotary(rope._ref, rows, dim, TYPES[x0.dtype], _ints(positions, "positions", rows), n, c.src, c.dst,
                            heads, 1 if inverse else 0, _stream(stream, x0.get_device())), "kvl_rotary")


class QuantCache:
    """The 8-bit paged cache of one model.

    codes: uint8 [L, 2, N, B, H, d]; scales: float32 [L, 2, N, H]; tables: int32
    [slots, pages per sequence]; lens: int32 [slots] tokens held; refs: int32 [N] references
    of each page (0: free).  pairs / n_pairs (made here when not given) receive the page copies
    that ``extend`` and ``compact`` ask for; ``copy_pages`` makes them.  ``empty`` allocates
    all of it.
    """

    def __init__(self, codes, scales, tables, lens, refs, code="e4m3", pairs=None, n_pairs=None):
        if code not in CODES or codes.dim() != 6 or codes.shape[1] != 2 or tables.dim() != 2:
            raise ValueError(f"code: one of {sorted(CODES)}; codes: [L, 2, N, B, H, d]; tables: [slots, pages]")
        L, _, N, B, H, d = codes.shape
        _flat(codes, torch.uint8, codes.shape, "codes")
        _flat(scales, torch.float32, (L, 2, N, H), "scales")
        _flat(tables, torch.int32, tables.shape, "tables")
        _ints(lens, "lens", tables.shape[0])
        _ints(refs, "refs", N)
        self.codes, self.scales, self.tables, self.lens, self.refs, self.code = codes, scales, tables, lens, refs, code
        self.n_layers, self.pool_blocks, self.block_tokens, self.n_kv_heads, self.head_dim = L, N, B, H, d
        self.device, self._index = codes.device, codes.get_device()
        self.pairs = torch.empty((N, 2), dtype=torch.int32, device=self.device) if pairs is None else pairs
        # the report and, unless given, the number of pairs
        own = torch.zeros(KVL_REPORT_BYTES + 16, dtype=torch.uint8, device=self.device)
        self.report = own[:KVL_REPORT_BYTES]
        self.n_pairs = own[KVL_REPORT_BYTES:KVL_REPORT_BYTES + 4].view(torch.int32) if n_pairs is None else n_pairs
        _flat(self.pairs, torch.int32, (N, 2), "pairs")
        _ints(self.n_pairs, "n_pairs", 1)
        self.n_slots = tables.shape[0]
        self._lib = _lib()
        self._c = kvl_cache(L, H, d, B, N, CODES[code], 0, codes.data_ptr(), scales.data_ptr())
        self._p = kvl_pages(N, B, self.n_slots, tables.shape[1], tables.data_ptr(), lens.data_ptr(), refs.data_ptr(),
                            self.pairs.data_ptr(), self.n_pairs.data_ptr())
        self._cache, self._pages = ctypes.byref(self._c), ctypes.byref(self._p)
        self._ws_bytes = int(self._lib.kvl_attend_workspace_bytes(self._cache))
        if self._ws_bytes == 0:
            raise ValueError(f"no such cache: head_dim {d} (a multiple of 16 up to 256), block_tokens {B}, {H} heads")
        # a workspace for each stream (calls on two streams may run at the same time), and one for the newest
        # capture on it (the graph may run beside them)
        self._ws, self._ws_captured = {}, {}
        self._capture_id = self._lib.kvl_capture_id
        self._scale = 1.0 / math.sqrt(d)
        self._args = _Args(self)
        self._report = self.report.data_ptr()
        self.reset_status()

    @classmethod
    def empty(cls, n_layers, n_kv_heads, head_dim, block_tokens, pool_blocks, max_seqs, max_pages, code="e4m3",
              device="cuda"):
        """A cache of free pages and empty sequences."""
        shape = (n_layers, 2, pool_blocks, block_tokens, n_kv_heads, head_dim)
        codes = torch.zeros(shape, dtype=torch.uint8, device=device)
        scales = torch.zeros((n_layers, 2, pool_blocks, n_kv_heads), dtype=torch.float32, device=device)
        tables = torch.zeros((max_seqs, max_pages), dtype=torch.int32, device=device)
        lens = torch.zeros(max_seqs, dtype=torch.int32, device=device)
        refs = torch.zeros(pool_blocks, dtype=torch.int32, device=device)
        return cls(codes, scales, tables, lens, refs, code=code)

    # -- rows -----------------------------------------------------------------
    def _seqs(self, c, starts, slots, n_rows):
        n = starts.shape[0] - 1
        if n < 0 or (slots is None and n > self.n_slots):
            raise ValueError(f"starts: one more entry than there are sequences, of which there are {self.n_slots}")
        s = c.seqs
        s.n_seq, s.n_rows, s.starts = n, n_rows, _ints(starts, "starts")
        s.slots = None if slots is None else _ints(slots, "slots", n)
        return s

    def append(self, layer, k, v, starts, rope=None, slots=None, stream=None):
        """Quantise fresh k, v [rows, H, d] into the pages of `layer`: rows starts[i] ..
        starts[i + 1] are the last tokens of sequence slots[i] (or i).  rope: turn k by the
        tokens' positions first (a multiple of 8 pairs; ``rotary`` turns keys of other numbers beforehand)."""
        n_rows, dtype, c = k.shape[0], k.dtype, self._args
        if dtype is not v.dtype or n_rows != v.shape[0]:
            raise ValueError("k, v: one type and shape")
        _rows(c.a, k, "k", self.n_kv_heads, self.head_dim)
        _rows(c.b, v, "v", self.n_kv_heads, self.head_dim)
        r = self._lib.kvl_cache_append(self._cache, layer, self._seqs(c, starts, slots, n_rows), TYPES[dtype], c.a, c.b,
                                       None if rope is None else rope._ref, self._report, _stream(stream, self._index))
        if r:
            check(r, "kvl_cache_append")

    def attend(self, layer, q, starts, out=None, lse=None, sm_scale=None, causal=True, window=0, slots=None,
               max_new=0, stream=None):
        """Attention of fresh rows q [rows, n_heads, d] (laid out as append's) over their
        sequences' tokens in `layer`; returns out [rows, n_heads, d], which belongs to the call's
        stream where it is made here.  lse: float32 [rows, n_heads]
        that receives the logarithms of the softmax sums.  max_new: a bound the caller knows on the
        rows of any one sequence.

        Calls of one stream share a workspace, kept here.  Calls captured into a graph (torch.cuda.graph) have one
        of that graph's own memory, which each run of the graph clears first: graphs may run in any
        order, or beside each other and other calls where they have memory pools of their own."""
        n_rows, heads, _ = q.shape
        dtype, c = q.dtype, self._args
        _rows(c.q, q, "q", heads, self.head_dim)
        st = _stream(stream, self._index)
        if out is None:
            shape = n_rows, heads, self.head_dim
            if stream is None:
                out = torch.empty(shape, dtype=dtype, device=q.device)
            else:
                with self._on(st):
                    out = torch.empty(shape, dtype=dtype, device=q.device)
        elif out.dtype is not dtype or out.shape[0] != n_rows:
            raise ValueError("out: the type and shape of q")
        _rows(c.out, out, "out", heads, self.head_dim)
        a = c.attn
        if lse is None:
            a.lse = None
        else:
            _flat(lse, torch.float32, (n_rows, heads), "lse")
            a.lse = lse.data_ptr()
        if not (-_MOST <= window <= _MOST and -_MOST <= max_new <= _MOST):  # (a C int would wrap round)
            raise ValueError("window, max_new: 32-bit numbers")
        capture = self._capture_id(st)
        held = self._ws_captured if capture else self._ws
        ws = held.get(st)
        if ws is None or ws[0] != capture:
            ws = self._workspace(held, st, capture)
        a.n_heads, a.type, a.sm_scale = heads, TYPES[dtype], self._scale if sm_scale is None else sm_scale
        a.causal, a.window, a.max_new = 1 if causal else 0, window, max_new
        r = self._lib.kvl_attend(self._cache, layer, self._seqs(c, starts, slots, n_rows), a, ws[1], self._ws_bytes,
                                 self._report, st)
        if r:
            check(r, "kvl_attend")
        return out

    def _on(self, st):
        """Allocations for calls on stream `st` are made on it: memory just freed on another may still be
        in use there."""
        on = self.device
        return torch.cuda.stream(torch.cuda.ExternalStream(st, device=on) if st else torch.cuda.default_stream(on))

    def _workspace(self, held, st, capture):
        # In a capture the zeroing is a part of the graph, and the memory its pool's, as the graph's
        # temporaries are.
        with self._on(st):
            ws = torch.empty(self._ws_bytes, dtype=torch.uint8, device=self.device)
            ws[:KVL_ATTEND_ZERO_BYTES].zero_()
        held[st] = capture, ws.data_ptr(), ws
        return held[st]

    # -- pages ----------------------------------------------------------------
    def extend(self, slots, counts, stream=None):
        """Sequence slots[i] will hold counts[i] more tokens; make ``copy_pages`` before they are
        appended (a shared last page is replaced by a copy)."""
        n = slots.shape[0]
        check(self._lib.kvl_pages_extend(self._pages, n, _ints(slots, "slots"), _ints(counts, "counts", n),
                                         self._report, _stream(stream, self._index)), "kvl_pages_extend")

    def fork(self, parents, children, stream=None):
        """children[i] (empty) becomes a copy of parents[i] that shares its pages."""
        n = parents.shape[0]
        check(self._lib.kvl_pages_fork(self._pages, n, _ints(parents, "parents"), _ints(children, "children", n),
                                       self._report, _stream(stream, self._index)), "kvl_pages_fork")

    def free(self, slots, stream=None):
        """The sequences of `slots` end; their pages lose a reference."""
        check(self._lib.kvl_pages_free(self._pages, slots.shape[0], _ints(slots, "slots"), self._report,
                                       _stream(stream, self._index)), "kvl_pages_free")

    def compact(self, stream=None):
        """Renumber the live pages into the lowest numbers; ``copy_pages`` moves them."""
        check(self._lib.kvl_pages_compact(self._pages, self._report, _stream(stream, self._index)), "kvl_pages_compact")

    def copy_pages(self, stream=None):
        """Make the copies that the last extend or compact asked for (every layer)."""
        check(self._lib.kvl_pages_copy(self._cache, self._p.pairs, self._p.n_pairs, self.pool_blocks, self._report,
                                       _stream(stream, self._index)), "kvl_pages_copy")

    # -- status ---------------------------------------------------------------
    def status(self, stream=None):
        """(code, detail) of the problems recorded so far (synchronises)."""
        return kvl_read_status(self._report, _stream(stream, self._index))

    def reset_status(self, stream=None):
        check(self._lib.kvl_report_reset(self._report, _stream(stream, self._index)), "kvl_report_reset")
