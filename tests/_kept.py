"""Plain 64-bit definitions of the weights of cached tokens and of eviction, for the tests: loops on the CPU that
share nothing with the CUDA path."""
from __future__ import annotations

import math

import torch

from tests import _quant as Q


def fork(cache, groups, shared):
    """Let the sequences of each group (ranges of slots) name the first one's pages for their first shared[g] tokens."""
    B = cache["codes"].shape[3]
    for g, P in enumerate(shared):
        n = -(-P // B)
        for s in range(groups[g] + 1, groups[g + 1]):
            cache["tables"][s, :n] = cache["tables"][groups[g], :n]


def weigh(cache, layer, q, starts, slots, lse, mass, begin, sm_scale, causal, window):
    """(mass, tolerance), [slots, tokens] in 64 bits.

    Tolerances: a term is a factor exp(+-error) off, where the error is that of its score (sums of d products in 32
    bits, each addition at most 2^-23 off) and what 32 bits leave of x - lse in units of log 2 (three roundings
    of numbers below 2 |x| + 2 |lse|); the exponential is 2^-22 off, and a sum of n terms n 2^-24."""
    T, Hq, d = q.shape
    G = Hq // cache["codes"].shape[4]
    out, tol = mass.double().clone(), torch.zeros_like(mass, dtype=torch.float64)
    for i, slot in enumerate(slots):
        a, b, n = int(starts[i]), int(starts[i + 1]), int(cache["lens"][slot])
        if b == a:
            continue
        K = Q.tokens(cache, layer, 0, slot, n)
        if begin:
            out[slot, max(0, n - (b - a)):n] = 0
        add, off = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
        terms = 1
        for t in range(a, b):
            p = n - (b - a) + t - a
            hi = min(n, p + 1) if causal else n
            lo = max(0, p - window + 1) if window else 0
            if hi <= lo:
                continue
            for h in range(Hq):
                z = float(lse[t, h])
                if math.isinf(z):
                    continue
                k, x = K[lo:hi, h // G], q[t, h].double()
                s = (k @ x) * sm_scale
                w = torch.exp(s - z)
                ds = (d + 8) * 2.0 ** -23 * sm_scale * (k.abs() @ x.abs()) + 2.0 ** -22 * (s.abs() + abs(z))
                add[lo:hi] += w
                off[lo:hi] += w * (2 * ds + 2.0 ** -22)
                terms += 1
        out[slot, :n] += add
        tol[slot, :n] = off + (terms + 2) * 2.0 ** -24 * out[slot, :n].abs() + 1e-30
    return out, tol


def kept(mass, n, keep, first, recent):
    """The tokens that stay of n, in order; mass: a list of numbers or None."""
    if n <= keep:
        return list(range(n))
    f = min(first, keep)
    r = min(recent, keep - f)
    middle = list(range(f, n - r))
    if mass is not None:
        rank = {j: (1, 0.0) if math.isnan(mass[j]) else (0, -mass[j]) for j in middle}
        middle.sort(key=lambda j: rank[j])  # (stable: of equals the first)
    return list(range(f)) + sorted(middle[:keep - f - r]) + list(range(n - r, n))


def evict(cache, slots, keep, mass, first, recent):
    """Shorten sequences of `cache` (changed in place, mass [slots, tokens] too) by the documented rules; codes in
    32-bit arithmetic, so they come out exactly."""
    codes, scales, tables, refs, code = (cache[k] for k in ("codes", "scales", "tables", "refs", "code"))
    L, _, N, B = codes.shape[:4]
    free = [b for b in range(N) if int(refs[b]) == 0]
    for i, slot in enumerate(slots):
        n, k = int(cache["lens"][slot]), keep[i]
        if n <= k:
            continue
        stay = kept(None if mass is None else mass[slot].tolist(), n, k, first, recent)
        old = tables[slot].clone()
        if mass is not None:
            row = mass[slot, stay].clone()
            mass[slot] = 0
            mass[slot, :k] = row
        u = min(first, k) // B
        for blk in range(u, -(-k // B)):
            page = free.pop(0)
            refs[page] = 1
            tables[slot, blk] = page
            here = stay[blk * B:(blk + 1) * B]
            for layer in range(L):
                for p in range(2):
                    was = torch.stack([scales[layer, p, int(old[j // B])] for j in here])
                    now = was.amax(dim=0)
                    for y, j in enumerate(here):
                        c = codes[layer, p, int(old[j // B]), j % B]
                        new = Q.to_codes(Q.of_codes(c, code).float() * (was[y] / now)[:, None], code)
                        codes[layer, p, page, y] = torch.where((was[y] == now)[:, None], c, new)
                    scales[layer, p, page] = now
        for blk in range(u, -(-n // B)):
            refs[int(old[blk])] -= 1
        cache["lens"][slot] = k
