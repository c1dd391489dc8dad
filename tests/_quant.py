"""Plain 64-bit definitions of the 8-bit cache's operators, for the tests: loops over
sequences, pages and tokens on the CPU, sharing nothing with the CUDA path."""
from __future__ import annotations

import math

import torch

QMAX = {"e4m3": 448.0, "int8": 127.0}
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def of_codes(u8, code):
    return u8.view(torch.float8_e4m3fn).float().double() if code == "e4m3" else u8.view(torch.int8).double()


def to_codes(x, code):
    """Nearest code, ties to even, of float32 values; NaN is NaN (e4m3) or 0 (int8)."""
    q = QMAX[code]
    y = torch.where(torch.isnan(x), x, x.clamp(-q, q))
    if code == "e4m3":
        return y.to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.where(torch.isnan(y), torch.zeros_like(y), torch.round(y)).to(torch.int8).view(torch.uint8)


def tokens(cache, layer, plane, slot, n):
    """The first n tokens of a sequence, dequantised: [n, H, d] in 64 bits."""
    B = cache["codes"].shape[3]
    out = torch.zeros((n, *cache["codes"].shape[4:]), dtype=torch.float64)
    for t in range(n):
        page = int(cache["tables"][slot, t // B])
        out[t] = of_codes(cache["codes"][layer, plane, page, t % B], cache["code"]) * \
            cache["scales"][layer, plane, page].double()[:, None]
    return out


def attend(cache, layer, q, starts, slots, sm_scale, causal, window):
    """(out, lse, tolerance of out, tolerance of lse), each [rows, heads(, d)] in 64 bits.

    Tolerances: probabilities enter the products with 11 significant bits (relative error
    2^-11 each, 2^-25 of the largest where they are below 2^-14), the result is rounded once to
    its type; scores are sums of d products in 32 bits (each addition at most 2^-23 off where
    the unit truncates), which changes a probability by a factor exp(+-error)."""
    T, Hq, d = q.shape
    H = cache["codes"].shape[4]
    G = Hq // H
    out = torch.zeros((T, Hq, d), dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for i, slot in enumerate(slots):
        a, b, n = int(starts[i]), int(starts[i + 1]), int(cache["lens"][slot])
        if b == a:
            continue
        K, V = (tokens(cache, layer, p, slot, n) for p in (0, 1))
        for t in range(a, b):
            p = n - (b - a) + t - a
            hi = min(n, p + 1) if causal else n
            lo = max(0, p - window + 1) if window else 0
            if hi <= lo:
                continue
            for h in range(Hq):
                k, v = K[lo:hi, h // G], V[lo:hi, h // G]
                x = q[t, h].double()
                s = (k @ x) * sm_scale
                z = torch.logsumexp(s, 0)
                w = torch.exp(s - z)
                out[t, h] = w @ v
                lse[t, h] = z
                ds = (d + 8) * 2.0 ** -23 * sm_scale * float((k.abs() @ x.abs()).max())
                top = v.abs().max(dim=0).values
                tol[t, h] = UNIT[q.dtype] * out[t, h].abs() + (2.0 ** -10 + 2 * ds) * (w @ v.abs()) + \
                    (hi - lo) * 2.0 ** -25 * top + 2.0 ** -24
                tol_lse[t, h] = ds + 1e-5 + 2.0 ** -22 * abs(float(z))
    return out, lse, tol, tol_lse


def turn(x, pos, inv_freq, interleaved=False, gain=1.0, inverse=False):
    """Rotary positions of x [rows, heads, dim] in 64 bits."""
    n = inv_freq.shape[0]
    a = pos.double()[:, None] * inv_freq.double()[None]
    c, s = gain * torch.cos(a)[:, None], gain * torch.sin(a)[:, None] * (-1.0 if inverse else 1.0)
    y = x.double().clone()
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    p, q = x[..., i].double(), x[..., j].double()
    y[..., i], y[..., j] = p * c - q * s, q * c + p * s
    return y


def append(cache, layer, k, v, starts, slots):
    """Append rows of 64-bit (or exact) values, page by page; changes `cache`.  The arithmetic is the
    documented one in 32 bits, so codes come out exactly."""
    B, qmax, code = cache["codes"].shape[3], QMAX[cache["code"]], cache["code"]
    for i, slot in enumerate(slots):
        a, b = int(starts[i]), int(starts[i + 1])
        if b == a:
            continue
        n = int(cache["lens"][slot])
        p0 = n - (b - a)
        for blk in range(p0 // B, (n - 1) // B + 1):
            lo, hi = max(p0, blk * B), min(n, (blk + 1) * B)
            page = int(cache["tables"][slot, blk])
            for plane, x in ((0, k), (1, v)):
                rows = x[a + lo - p0:a + hi - p0].float()
                mag = torch.where(torch.isfinite(rows), rows.abs(), torch.zeros_like(rows)).amax(dim=(0, 2))
                s, c = cache["scales"][layer, plane, page], cache["codes"][layer, plane, page]
                was = s.clone() if lo > blk * B else torch.zeros_like(s)
                now = torch.maximum(torch.maximum(was, mag * torch.tensor(1.0 / qmax, dtype=torch.float32)), torch.full_like(s, 1e-30))
                if lo > blk * B:
                    held = c[:lo - blk * B]
                    same = (was == now)[None, :, None]
                    new = to_codes(of_codes(held, code).float() * (was / now)[None, :, None], code)
                    c[:lo - blk * B] = torch.where(same, held, new)
                c[lo - blk * B:hi - blk * B] = to_codes(rows * (1.0 / now)[None, :, None], code)
                s.copy_(now)


def make_cache(seed, L, H, d, B, lens, spare=3, code="e4m3", extra_slots=0, poison=True, gain=1.0):
    """A cache on the CPU whose sequences hold `lens` tokens in shuffled pages.  With poison,
    every slot past a sequence's end, every page nobody holds, their scales and the table entries
    past the end hold NaN codes (or extreme ones), NaN scales and page numbers out of range."""
    g = torch.Generator().manual_seed(seed)
    n = [-(-x // B) for x in lens]
    N = sum(n) + spare
    perm = torch.randperm(N, generator=g).int()
    slots = len(lens) + extra_slots
    W = max([1] + n) + 2
    tables = torch.full((slots, W), -7 if poison else 0, dtype=torch.int32)
    x = torch.randn((L, 2, N, B, H, d), generator=g) * gain
    scales = (x.abs().amax(dim=(3, 5)) / QMAX[code]).contiguous()
    codes = to_codes(x / scales[:, :, :, None, :, None], code)
    if poison:
        held = torch.zeros((N, B), dtype=torch.bool)
    at = 0
    for s, (k, length) in enumerate(zip(n, lens)):
        tables[s, :k] = perm[at:at + k]
        if poison:
            for j in range(k):
                held[int(perm[at + j]), :min(B, length - j * B)] = True
        at += k
    if poison:
        codes[:, :, ~held] = 0x7F
        scales[:, :, ~held.any(dim=1)] = math.nan
    refs = torch.zeros(N, dtype=torch.int32)
    refs[perm[:at].long()] = 1
    full = torch.zeros(slots, dtype=torch.int32)
    full[:len(lens)] = torch.tensor(lens, dtype=torch.int32)
    return dict(codes=codes.contiguous(), scales=scales, tables=tables, lens=full, refs=refs, code=code)


def on_gpu(cache):
    from layer_wise_paged_gb300.cache import QuantCache
    return QuantCache(*(cache[k].cuda() for k in ("codes", "scales", "tables", "lens", "refs")), code=cache["code"])
