"""Measured cases of the 8-bit paged cache operators.

Four operators: attention over the 8-bit cache ("attend"), the append that quantises
fresh K/V rows into its pages ("append"), rotary positions ("rotary") and the pages'
bookkeeping and copies ("pages").  ``run`` computes each in its plain form (elementary
torch operations in 32 bits) or, with ``own``, through this repository's package.

A cache holds codes [L, 2, N, B, H, d] of one byte (e4m3 or int8; plane 0 is K, 1 is V) and
float32 scales [L, 2, N, H]: a value is its code times the scale of its page and head.
Sequence r's token t lives in page tables[r, t // B], slot t % B.
"""
import math

import numpy as np
import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
TINY = 1e-30  # smallest scale an append writes
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


def _attend(name, **k):
    c = dict(op="attend", seqs=1, kv=1000, kv_mix="same", new=1, new_mix="same", heads=32,
             kv_heads=8, d=128, block=16, code="e4m3", dtype="bf16", causal=True, window=0, mix=1)
    c.update(k)
    return dict(c, name=name) if name else c


def _append(name, **k):
    c = dict(op="append", seqs=1, old=0, old_mix="same", new=1, new_mix="same", heads=32,
             kv_heads=8, d=128, block=16, code="e4m3", dtype="bf16", rope=True, mix=1)
    c.update(k)
    return dict(c, name=name) if name else c


def _rotary(name, **k):
    c = dict(op="rotary", rows=1, heads=32, kv_heads=8, d=128, rot=128, interleaved=False,
             dtype="bf16", inverse=False, start=0, scaling="none")
    c.update(k)
    return dict(c, name=name) if name else c


def _pages(name, **k):
    c = dict(op="pages", mode="branch", seqs=16, forks=3, tokens=500, new=5, layers=32, kv_heads=8,
             d=128, block=16, code="e4m3", spare=1.3, mix=1)
    c.update(k)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user of an 8B-class model, one layer of one decoded token: latency
        _attend("attend_one_token", kv=777),
        # a decode step of a full server: the 256 small requests of the copy benchmark
        _attend("attend_decode_256", seqs=256, kv=2200, kv_mix="lognormal", mix=5),
        # one token against a 128K context of a 32B-class model (64 query heads)
        _attend("attend_long_token", kv=128000, heads=64, block=64),
        # an agentic turn: 512 fresh tokens on a cached prefix of 30,720
        _attend("attend_turn_512", kv=31232, new=512),
        # verification of drafted tokens, 1 to 8 a sequence, small heads, int8 codes, f16
        _attend("attend_drafted", seqs=48, kv=6000, kv_mix="ragged", new=8, new_mix="ragged",
                heads=16, kv_heads=4, d=64, block=32, code="int8", dtype="f16", mix=7),
        # fresh prompts of several users in one batch, nothing cached, a sliding window
        _attend("attend_prompts", seqs=6, kv=4096, kv_mix="ragged", new=0, new_mix="whole",
                window=2048, mix=3),
        # the decode step's writes: one token for each of 256 sequences
        _append("append_decode_256", seqs=256, old=2200, old_mix="lognormal", mix=5),
        # the writes of a long fresh prompt, whose first page is already partly filled
        _append("append_prompt", old=37, new=31001),
        # positions of a small decode batch, q and k of one layer
        _rotary("rotary_decode", rows=7, start=2048),
        # the gradient of a long prompt's positions: interleaved pairs, half of the head,
        # scaled for a longer context than the model was trained on
        _rotary("rotary_prompt_gradient", rows=32000, heads=64, rot=64, interleaved=True,
                inverse=True, scaling="wavelength"),
        # a step of branched decoding: fork, extend, copy shared last pages, drop the branches
        _pages("pages_branch"),
        # half of the sequences have ended: compaction of what is left
        _pages("pages_compact", mode="compact", seqs=64, forks=0, tokens=400, new=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    largest = max(_cost(c) for c in listed())
    while True:
        c = _draw(rng)
        if _fits(c) and _cost(c) <= largest:
            return c


def _draw(rng):
    mix = rng.randrange(1 << 20)
    code, dtype = rng.choice(["e4m3", "int8"]), rng.choice(["bf16", "f16"])
    heads, kv_heads = rng.choice([(8, 8), (16, 4), (32, 8), (64, 8), (32, 4), (16, 1)])
    d, block = rng.choice([64, 128]), rng.choice([16, 32, 64])
    op = rng.choice(["attend", "attend", "attend", "append", "rotary", "pages"])
    if op == "attend":
        kind = rng.choice(["token", "drafted", "turn", "prompts"])
        c = _attend("", heads=heads, kv_heads=kv_heads, d=d, block=block, code=code, dtype=dtype, mix=mix,
                    window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]))
        if kind == "token":
            c.update(seqs=_log(rng, 1, 256), kv=_log(rng, 1, 131072), kv_mix=rng.choice(["same", "ragged", "lognormal"]))
        elif kind == "drafted":
            c.update(seqs=_log(rng, 1, 128), kv=_log(rng, 8, 32768), kv_mix="ragged", new=rng.randint(2, 9), new_mix="ragged")
        elif kind == "turn":
            c.update(seqs=rng.randint(1, 4), kv=_log(rng, 64, 65536), kv_mix="same", new=_log(rng, 16, 2048))
            c["new"] = min(c["new"], c["kv"])
        else:
            c.update(seqs=rng.randint(1, 8), kv=_log(rng, 16, 4096), kv_mix="ragged", new=0, new_mix="whole",
                     causal=rng.random() < 0.8)
            c["window"] = c["window"] if c["causal"] else 0
        return c
    if op == "append":
        c = _append("", heads=heads, kv_heads=kv_heads, d=d, block=block, code=code, dtype=dtype, mix=mix,
                    rope=code == "e4m3" and rng.random() < 0.7)
        if rng.random() < 0.5:
            c.update(seqs=_log(rng, 1, 256), old=_log(rng, 1, 8192), old_mix="ragged", new=rng.randint(1, 8), new_mix="ragged")
        else:
            c.update(seqs=rng.randint(1, 4), old=rng.randint(0, 200), new=_log(rng, 32, 16384))
        return c
    if op == "rotary":
        rot = rng.choice([d, d, d // 2, d // 4])
        return _rotary("", rows=_log(rng, 1, 32000), heads=heads, kv_heads=kv_heads, d=d, rot=rot, dtype=rng.choice(["bf16", "f16", "f32"]),
                       interleaved=rng.random() < 0.5, inverse=rng.random() < 0.4, start=_log(rng, 1, 100000),
                       scaling=rng.choice(["none", "linear", "wavelength"]))
    if rng.random() < 0.5:
        return _pages("", seqs=_log(rng, 1, 32), forks=rng.randint(1, 4), tokens=_log(rng, 16, 1000), new=rng.randint(1, 40),
                      layers=rng.choice([2, 8, 32]), kv_heads=kv_heads, d=d, block=block, code=code, mix=mix)
    return _pages("", mode="compact", seqs=_log(rng, 4, 128), forks=0, tokens=_log(rng, 32, 1000), new=0,
                  layers=rng.choice([2, 8, 32]), kv_heads=kv_heads, d=d, block=block, code=code, mix=mix)


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def _fits(c):
    """Whether the plain form's temporaries and the state stay within a few GB."""
    if c["op"] == "attend":
        kv, new = _lengths(c)
        s, k, n = len(kv), int(kv.max()), int(new.max())
        return s * k * c["kv_heads"] * c["d"] * 4 <= 9 << 30 and s * c["heads"] * n * k * 4 <= 13 << 30
    if c["op"] == "pages":
        return _pages_n(c) * c["block"] * c["kv_heads"] * c["d"] * 2 * c["layers"] <= 2300 << 20
    return True


# ---- sizes a case stands for (from the case alone) ------------------------------------

def _spread(mix, n, size, how, low=1):
    g = np.random.RandomState(mix)
    if how == "ragged":
        return np.maximum(low, g.randint(1, size + 1, n)).astype(np.int64) if size else np.zeros(n, np.int64)
    if how == "lognormal":
        return np.clip(np.rint(g.lognormal(math.log(size), 0.5, n)), max(1, size // 8), size * 4).astype(np.int64)
    return np.full(n, size, np.int64)


def _lengths(c):
    """(tokens held, fresh tokens) of each sequence: the fresh ones are the last held."""
    n = c["seqs"]
    if c["op"] == "append":
        old = _spread(c["mix"], n, c["old"], c["old_mix"])
        new = _spread(c["mix"] + 1, n, c["new"], c["new_mix"])
        return old + new, new
    kv = _spread(c["mix"], n, c["kv"], c["kv_mix"])
    if c["new_mix"] == "whole":
        return kv, kv.copy()
    new = _spread(c["mix"] + 1, n, c["new"], c["new_mix"])
    return np.maximum(kv, new), new


def _pages_n(c):
    g = np.random.RandomState(c["mix"])
    held = g.randint(max(1, c["tokens"] // 2), c["tokens"] * 3 // 2 + 1, c["seqs"])
    need = int((-(-held // c["block"])).sum()) + c["seqs"] * c["forks"] * (2 + c["new"] // c["block"])
    return max(8, int(need * c["spare"]))


def _visible(c):
    """Visible (query, key) pairs summed over the sequences, and tokens any query sees."""
    kv, new = _lengths(c)
    pairs, seen = 0, 0
    for k, n in zip(kv.tolist(), new.tolist()):
        pos = np.arange(k - n, k, dtype=np.int64)
        hi = pos + 1 if c["causal"] else np.full(n, k)
        lo = np.maximum(0, pos + 1 - c["window"]) if c["window"] else np.zeros(n, np.int64)
        pairs += int((hi - lo).sum())
        seen += int(hi.max() - lo.min()) if n else 0
    return pairs, seen


def _moved(c):
    """Pages a "pages" case copies, from the case alone."""
    t = _page_state(c)
    if c["mode"] == "branch":
        held = t["lens"][: c["seqs"]]
        return int(c["forks"] * (held % c["block"] != 0).sum())
    live = np.flatnonzero(t["refs"])
    return int((live >= live.size).sum())


def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["rows"] * (c["heads"] + c["kv_heads"])
        return {"bytes": 2 * n * c["d"] * SIZES[c["dtype"]], "flops": 3 * n * c["rot"]}
    if c["op"] == "pages":
        page = c["layers"] * 2 * (c["block"] * c["kv_heads"] * c["d"] + 4 * c["kv_heads"])
        return {"bytes": 2 * _moved(c) * page + 4 * _pages_n(c), "flops": 0}
    kv, new = _lengths(c)
    rows, H, d = int(new.sum()), c["kv_heads"], c["d"]
    if c["op"] == "append":
        b = rows * H * d * 2 * (SIZES[c["dtype"]] + 1)
        return {"bytes": b, "flops": 4 * rows * H * d}
    pairs, seen = _visible(c)
    b = seen * H * d * 2 + 8 * H * -(-seen // c["block"]) + 2 * rows * c["heads"] * d * 2
    return {"bytes": b, "flops": 4 * pairs * c["heads"] * d}


# ---- inputs -----------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)


def _inv_freq(rot, scaling):
    """Frequencies of the rotated pairs; "linear" divides positions by 4, "wavelength" slows
    the pairs whose wavelength passes the trained context (8192) by 8, with a smooth join."""
    f = 500000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if scaling == "linear":
        f = f / 4.0
    elif scaling == "wavelength":
        turns = 8192.0 * f / (2 * math.pi)
        mixed = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = f * mixed + f / 8.0 * (1 - mixed)
    return torch.from_numpy(f.astype(np.float32)).cuda()


def _fill_cache(g, L, N, c):
    """Codes and scales of a pool holding normal values, some heads and channels larger."""
    B, H, d = c["block"], c["kv_heads"], c["d"]
    codes = torch.empty((L, 2, N, B, H, d), dtype=torch.uint8, device="cuda")
    scales = torch.empty((L, 2, N, H), dtype=torch.float32, device="cuda")
    gain = torch.exp(0.5 * torch.randn((L, 2, 1, 1, H, 1), generator=g, device="cuda"))
    gain = gain * torch.exp(0.3 * torch.randn((L, 2, 1, 1, H, d), generator=g, device="cuda"))
    step = max(1, (1 << 28) // (B * H * d))
    for l in range(L):
        for p in range(2):
            for a in range(0, N, step):
                x = torch.randn((min(step, N - a), B, H, d), generator=g, device="cuda") * gain[l, p]
                s = x.abs().amax(dim=(1, 3)) / QMAX[c["code"]]
                scales[l, p, a:a + step] = s
                codes[l, p, a:a + step] = _to_codes(x / s[:, None, :, None], c["code"])
    return codes, scales


def _to_codes(x, code):
    x = x.clamp(-QMAX[code], QMAX[code])
    if code == "e4m3":
        return x.to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.round(x).to(torch.int8).view(torch.uint8)


def _of_codes(u8, code):
    return u8.view(torch.float8_e4m3fn if code == "e4m3" else torch.int8).float()


def _tables(g, kv, B, N):
    """Block tables [S, W] of sequences of kv tokens from a shuffled pool of N pages."""
    n = -(-kv // B)
    perm = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
    W = max(1, int(n.max()))
    starts = torch.from_numpy(np.concatenate([[0], np.cumsum(n)[:-1]])).cuda()
    at = starts[:, None] + torch.arange(W, device="cuda")[None, :]
    return torch.where(torch.arange(W, device="cuda")[None, :] < torch.from_numpy(n).cuda()[:, None],
                       perm[at.clamp(max=N - 1)], torch.full((), -1, dtype=torch.int32, device="cuda")).contiguous()


def _refs(tables, N):
    t = tables[tables >= 0].long()
    return torch.zeros(N, dtype=torch.int32, device="cuda").index_add_(0, t, torch.ones_like(t, dtype=torch.int32))


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "rotary":
        dt = DTYPES[c["dtype"]]
        # q and k side by side with v, as a fused projection leaves them
        qkv = torch.randn((c["rows"], c["heads"] + 2 * c["kv_heads"], c["d"]), generator=g, device="cuda").to(dt)
        s["q"], s["k"] = qkv[:, : c["heads"]], qkv[:, c["heads"]: c["heads"] + c["kv_heads"]]
        s["q_out"] = torch.empty((c["rows"], c["heads"], c["d"]), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((c["rows"], c["kv_heads"], c["d"]), dtype=dt, device="cuda")
        s["pos"] = torch.arange(c["start"], c["start"] + c["rows"], dtype=torch.int32, device="cuda")
        s["inv_freq"] = _inv_freq(c["rot"], c["scaling"])
        if own:
            from layer_wise_paged_gb300 import cache
            s["rope"] = cache.Rope(s["inv_freq"], interleaved=c["interleaved"], gain=1.0)
        return s
    if c["op"] == "pages":
        return _prepare_pages(c, s, g)
    kv, new = _lengths(c)
    B, H, d, dt = c["block"], c["kv_heads"], c["d"], DTYPES[c["dtype"]]
    N = int(math.ceil(1.25 * int((-(-kv // B)).sum())))
    s["codes"], s["scales"] = _fill_cache(g, 1, N, c)
    s["tables"] = _tables(g, kv, B, N)
    s["lens"] = torch.from_numpy(kv.astype(np.int32)).cuda()
    s["starts"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
    s["refs"] = _refs(s["tables"], N)
    T = int(new.sum())
    qkv = torch.randn((T, c["heads"] + 2 * H, d), generator=g, device="cuda").to(dt)
    s["q"], s["k"], s["v"] = qkv[:, : c["heads"]], qkv[:, c["heads"]: c["heads"] + H], qkv[:, c["heads"] + H:]
    s["max_new"], s["max_kv"] = int(new.max()), int(kv.max())
    if c["op"] == "attend":
        s["out"] = torch.empty((T, c["heads"], d), dtype=dt, device="cuda")
        s["lse"] = torch.empty((T, c["heads"]), dtype=torch.float32, device="cuda")
    else:
        s["inv_freq"] = _inv_freq(d, "wavelength")
    if own:
        from layer_wise_paged_gb300 import cache
        s["cache"] = cache.QuantCache(s["codes"], s["scales"], s["tables"], s["lens"], s["refs"], code=c["code"])
        if c["op"] == "append" and c["rope"]:
            s["rope"] = cache.Rope(s["inv_freq"], interleaved=False, gain=1.0)
    return s


def _page_state(c):
    """The bookkeeping before a "pages" case, from the case alone (numpy)."""
    g = np.random.RandomState(c["mix"])
    B, S, N = c["block"], c["seqs"], _pages_n(c)
    lens = g.randint(max(1, c["tokens"] // 2), c["tokens"] * 3 // 2 + 1, S).astype(np.int32)
    n = -(-lens // B)
    perm = g.permutation(N).astype(np.int32)
    slots = S * (1 + c["forks"])
    W = int(n.max()) + 2 + c["new"] // B
    tables = np.full((slots, W), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(n)])
    for r in range(S):
        tables[r, : n[r]] = perm[at[r]: at[r + 1]]
    full = np.zeros(slots, np.int32)
    full[:S] = lens
    if c["mode"] == "compact":  # every other sequence has ended
        full[1:S:2] = 0
    refs = np.zeros(N, np.int32)
    for r in range(S):
        refs[tables[r, : -(-int(full[r]) // B)]] += 1
    return {"tables": tables, "lens": full, "refs": refs}


def _prepare_pages(c, s, g):
    t = _page_state(c)
    N = t["refs"].size
    L, H, d, B = c["layers"], c["kv_heads"], c["d"], c["block"]
    # the copies move bytes: any codes but e4m3's NaN do
    s["codes"] = torch.randint(0, 127, (L, 2, N, B, H, d), generator=g, device="cuda", dtype=torch.uint8)
    s["scales"] = torch.rand((L, 2, N, H), generator=g, device="cuda") + 0.5
    for k, v in t.items():
        s[k] = torch.from_numpy(v).cuda()
        s[k + "0"] = s[k].clone()
    S, F = c["seqs"], c["forks"]
    s["parents"] = torch.arange(S, dtype=torch.int32, device="cuda").repeat_interleave(F)
    s["children"] = torch.arange(S, S + S * F, dtype=torch.int32, device="cuda")
    s["counts"] = torch.full((S * F,), c["new"], dtype=torch.int32, device="cuda")
    s["pairs"] = torch.zeros((N, 2), dtype=torch.int32, device="cuda")
    s["n_pairs"] = torch.zeros((1,), dtype=torch.int32, device="cuda")
    if own:
        from layer_wise_paged_gb300 import cache
        s["cache"] = cache.QuantCache(s["codes"], s["scales"], s["tables"], s["lens"], s["refs"], code=c["code"],
                                      pairs=s["pairs"], n_pairs=s["n_pairs"])
    return s


# ---- one pass -----------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if c["op"] == "attend":
        if own:
            s["cache"].attend(0, s["q"], s["starts"], out=s["out"], lse=s["lse"], causal=c["causal"],
                              window=c["window"], max_new=s["max_new"])
            return {"out": s["out"], "lse": s["lse"]}
        return _plain_attend(s, c)
    if c["op"] == "append":
        if own:
            s["cache"].append(0, s["k"], s["v"], s["starts"], rope=s.get("rope"))
        else:
            _plain_append(s, c)
        return {"codes": s["codes"].view(_value_type(c)), "scales": s["scales"]}
    if c["op"] == "rotary":
        if own:
            from layer_wise_paged_gb300 import cache
            cache.rotary(s["rope"], s["pos"], [(s["q"], s["q_out"]), (s["k"], s["k_out"])], inverse=c["inverse"])
            return {"q": s["q_out"], "k": s["k_out"]}
        cos, sin = _cos_sin(s["pos"], s["inv_freq"])
        sin = -sin if c["inverse"] else sin
        return {n: _plain_rotate(s[n].float(), cos, sin, c["interleaved"]).to(s[n].dtype) for n in ("q", "k")}
    (_own_pages if own else _plain_pages)(s, c)
    out = {k: s[k] for k in ("tables", "lens", "refs", "pairs", "n_pairs", "scales")}
    return dict(out, codes=s["codes"].view(_value_type(c)))


def _value_type(c):
    return torch.float8_e4m3fn if c["code"] == "e4m3" else torch.int8


def _own_pages(s, c):
    k = s["cache"]
    if c["mode"] == "branch":
        k.fork(s["parents"], s["children"])
        k.extend(s["children"], s["counts"])
        k.copy_pages()
        k.free(s["children"])
        return
    # the program's snapshot of its bookkeeping, so that there is something to compact
    s["tables"].copy_(s["tables0"])
    s["refs"].copy_(s["refs0"])
    k.compact()
    k.copy_pages()


def _cos_sin(pos, inv_freq):
    # 32 bits hold no fraction of a turn at positions of 10^5: the angle alone is reduced in 64
    a = torch.remainder(pos.double()[:, None] * inv_freq.double()[None, :], 2 * math.pi).float()
    return torch.cos(a)[:, None, :], torch.sin(a)[:, None, :]


def _plain_rotate(x, cos, sin, interleaved):
    n = cos.shape[-1]
    r = x[..., : 2 * n]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = r[..., :n], r[..., n:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., 2 * n:]], dim=-1)


def _plain_attend(s, c):
    B, H, d, G = c["block"], c["kv_heads"], c["d"], c["heads"] // c["kv_heads"]
    lens, starts = s["lens"].long(), s["starts"].long()
    new = starts[1:] - starts[:-1]
    S, W, n = s["tables"].shape[0], s["tables"].shape[1], s["max_new"]
    pages = s["tables"].long().clamp(min=0)
    j = torch.arange(W * B, device="cuda")
    there = (j[None, :] < lens[:, None])[:, :, None, None]

    def plane(p):  # [S, H, W*B, d] in 32 bits, nothing where no token is
        x = _of_codes(s["codes"][0, p][pages], c["code"]) * s["scales"][0, p][pages][:, :, None, :, None]
        return torch.where(there, x.reshape(S, W * B, H, d), 0.0).transpose(1, 2)

    i = torch.arange(n, device="cuda")
    rows = (starts[:-1, None] + i[None, :]).clamp(max=max(0, s["q"].shape[0] - 1))
    q = s["q"][rows].float().reshape(S, n, H, G, d).permute(0, 2, 3, 1, 4).reshape(S, H, G * n, d)
    x = torch.matmul(q, plane(0).transpose(2, 3)).mul_(1.0 / math.sqrt(d)).reshape(S, H, G, n, W * B)
    pos = (lens - new)[:, None] + i[None, :]
    see = (j[None, None, :] < lens[:, None, None]).expand(S, n, W * B)
    if c["causal"]:
        see = see & (j[None, None, :] <= pos[:, :, None])
    if c["window"]:
        see = see & (j[None, None, :] > pos[:, :, None] - c["window"])
    x.masked_fill_(~see[:, None, None], float("-inf"))
    m = x.amax(dim=-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    l = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.reshape(S, H, G * n, W * B), plane(1)).reshape(S, H, G, n, d)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + torch.log(l)).squeeze(-1)
    take = i[None, :] < new[:, None]
    out = o.permute(0, 3, 1, 2, 4).reshape(S, n, H * G, d)[take].to(s["q"].dtype)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(S, n, H * G)[take]}


def _plain_append(s, c):
    B, N = c["block"], s["codes"].shape[2]
    qmax = QMAX[c["code"]]
    lens, starts = s["lens"].long(), s["starts"].long()
    new = starts[1:] - starts[:-1]
    T = s["k"].shape[0]
    t = torch.arange(T, device="cuda")
    r = torch.searchsorted(starts[1:], t, right=True)
    pos = (lens - new)[r] + t - starts[:-1][r]
    page, slot = s["tables"].long()[r, pos // B], pos % B
    k = s["k"].float()
    if c["rope"]:
        k = _plain_rotate(k, *_cos_sin(pos, s["inv_freq"]), False)
    slots = torch.arange(B, device="cuda")[None, :]
    first = torch.full((N,), B, dtype=torch.int64, device="cuda").scatter_reduce(0, page, slot, "amin")
    touched = torch.unique(page)
    for plane, x in ((0, k), (1, s["v"].float())):
        codes, scales = s["codes"][0, plane], s["scales"][0, plane]
        a = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(dim=-1)
        amax = torch.zeros((N, a.shape[1]), device="cuda").index_reduce_(0, page, a, "amax")[touched]
        part = (first[touched] > 0)[:, None]
        was = torch.where(part, scales[touched], 0.0)
        now = torch.maximum(torch.maximum(was, amax / qmax), torch.full((), TINY, device="cuda"))
        old = _of_codes(codes[touched], c["code"]) * (was / now)[:, None, :, None]
        keep = (slots < first[touched][:, None])[:, :, None, None]
        codes[touched] = torch.where(keep, _to_codes(old, c["code"]), codes[touched])
        scales[touched] = now
        codes[page, slot] = _to_codes(x * (1.0 / scales[page])[..., None], c["code"])


def _plain_pages(s, c):
    B = c["block"]
    tables, lens, refs = s["tables"], s["lens"], s["refs"]
    N, W = refs.shape[0], tables.shape[1]
    w = torch.arange(W, device="cuda")[None, :]
    if c["mode"] == "branch":
        kids, dad, n = s["children"].long(), s["parents"].long(), s["counts"].long()
        # fork
        held = lens[dad].long()
        used = w < ((held + B - 1) // B)[:, None]
        tables[kids] = torch.where(used, tables[dad], tables[kids])
        lens[kids] = lens[dad]
        refs.index_add_(0, tables[kids][used].long(), torch.ones_like(tables[kids][used]))
        # extend: a shared, partly filled last page is replaced, then fresh pages follow
        last = tables[kids].gather(1, ((held - 1).clamp(min=0) // B)[:, None])[:, 0].long()
        cow = (held % B != 0) & (n > 0) & (refs[last] > 1)
        lo = (held + B - 1) // B - cow.long()
        hi = (held + n + B - 1) // B
        take = (w >= lo[:, None]) & (w < hi[:, None])
        free = torch.nonzero(refs == 0)[:, 0]
        got = free[: int(take.sum())].to(torch.int32)
        rows = tables[kids]
        rows[take] = got
        tables[kids] = rows
        refs[got.long()] = 1
        refs.index_add_(0, last[cow], torch.full_like(last[cow], -1, dtype=torch.int32))
        lens[kids] = (held + n).to(torch.int32)
        src, dst = last[cow], rows.gather(1, lo[:, None])[:, 0].long()[cow]
        k = src.shape[0]
        s["n_pairs"].fill_(k)
        s["pairs"][:k, 0], s["pairs"][:k, 1] = src.to(torch.int32), dst.to(torch.int32)
        s["codes"][:, :, dst] = s["codes"][:, :, src]
        s["scales"][:, :, dst] = s["scales"][:, :, src]
        # free
        used = w < ((lens[kids].long() + B - 1) // B)[:, None]
        gone = tables[kids][used].long()
        refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
        lens[kids] = 0
        return
    tables.copy_(s["tables0"])
    refs.copy_(s["refs0"])
    live = refs > 0
    n = int(live.sum())
    src = torch.nonzero(live[n:])[:, 0] + n
    dst = torch.nonzero(~live[:n])[:, 0]
    new_id = torch.arange(N, dtype=torch.int32, device="cuda")
    new_id[src] = dst.to(torch.int32)
    used = w < ((lens.long() + B - 1) // B)[:, None]
    tables.copy_(torch.where(used, new_id[tables.long().clamp(min=0)], tables))
    refs[dst] = refs[src]
    refs[src] = 0
    k = src.shape[0]
    s["n_pairs"].fill_(k)
    s["pairs"][:k, 0], s["pairs"][:k, 1] = src.to(torch.int32), dst.to(torch.int32)
    s["codes"][:, :, dst] = s["codes"][:, :, src]
    s["scales"][:, :, dst] = s["scales"][:, :, src]


# ---- the same outputs from the definitions in 64 bits ---------------------------------------

def exact(case, seed):
    global own
    c = case
    if c["op"] == "pages":
        return None  # whole numbers and copies of bytes
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if c["op"] == "rotary":
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           s["pos"].double()[:, None] * s["inv_freq"].double()[None, :])
        return {n: _turn(s[n].double(), turn.conj() if c["inverse"] else turn, c["interleaved"]) for n in ("q", "k")}
    if c["op"] == "append":
        return _exact_append(s, c)
    return _exact_attend(s, c)


def _turn(x, turn, interleaved):
    """Rotation as a product of complex numbers: turn [rows, pairs] of length 1."""
    n = turn.shape[-1]
    y = x.clone()
    if interleaved:
        z = torch.complex(x[..., 0:2 * n:2].contiguous(), x[..., 1:2 * n:2].contiguous()) * turn[:, None]
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :n].contiguous(), x[..., n:2 * n].contiguous()) * turn[:, None]
        y[..., :n], y[..., n:2 * n] = z.real, z.imag
    return y


def _exact_attend(s, c):
    H, G, d, B = c["kv_heads"], c["heads"] // c["kv_heads"], c["d"], c["block"]
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    out = torch.zeros((s["q"].shape[0], c["heads"], d), dtype=torch.float64, device="cuda")
    lse = torch.full((s["q"].shape[0], c["heads"]), float("-inf"), dtype=torch.float64, device="cuda")
    for r, k in enumerate(lens):
        a, b = starts[r], starts[r + 1]
        at = torch.arange(k, device="cuda")
        page, slot = s["tables"][r].long()[at // B], at % B
        for h in range(H):
            kk, vv = (_of_codes(s["codes"][0, p][page, slot, h], c["code"]).double()
                      * s["scales"][0, p, :, h].double()[page, None] for p in (0, 1))
            for i in range(a, b, 1024):
                e = min(b, i + 1024)
                pos = torch.arange(k - (b - i), k - (b - e), device="cuda")[:, None]
                x = s["q"][i:e, h * G:(h + 1) * G].double().transpose(0, 1) @ kk.T / math.sqrt(d)
                hide = torch.zeros((e - i, k), dtype=torch.bool, device="cuda")
                if c["causal"]:
                    hide |= at[None] > pos
                if c["window"]:
                    hide |= at[None] <= pos - c["window"]
                x[:, hide] = float("-inf")
                z = torch.logsumexp(x, dim=-1)
                lse[i:e, h * G:(h + 1) * G] = z.T
                some = torch.isfinite(z)
                p = torch.where(some[..., None], torch.exp(x - torch.where(some, z, 0.0)[..., None]), 0.0)
                out[i:e, h * G:(h + 1) * G] = (p @ vv).transpose(0, 1)
    return {"out": out, "lse": lse}


def _exact_append(s, c):
    B, q = c["block"], QMAX[c["code"]]
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    tables = s["tables"].tolist()
    scales, codes = s["scales"].double(), s["codes"].clone()
    for r, n in enumerate(lens):
        a, b = starts[r], starts[r + 1]
        p0 = n - (b - a)
        k, v = s["k"][a:b].double(), s["v"][a:b].double()
        if c["rope"]:
            at = torch.arange(p0, n, dtype=torch.float64, device="cuda")
            k = _turn(k, torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), at[:, None] * s["inv_freq"].double()), False)
        if b - a > 512 and p0 % B == 0 and n % B == 0:
            blocks = [(p0, n)]
        else:
            cut = [p0] + [x for x in range((p0 // B + 1) * B, n, B)] + [n]
            if len(cut) > 4:  # whole pages between the first and the last are alike
                cut = [p0, cut[1], cut[-2], n]
            blocks = [(x, y) for x, y in zip(cut, cut[1:]) if y > x]
        for x, y in blocks:
            pages = torch.tensor(tables[r][x // B:(y + B - 1) // B], device="cuda")
            for plane, rows in ((0, k), (1, v)):
                z = rows[x - p0:y - p0]
                if x % B == 0 and y - x > B:
                    z = z.reshape(len(pages), B, *z.shape[1:])
                else:
                    z = z[None]
                was = scales[0, plane, pages] if x % B else torch.zeros_like(scales[0, plane, pages])
                now = torch.maximum(was, z.abs().amax(dim=(1, 3)) / q).clamp(min=TINY)
                scales[0, plane, pages] = now
                if x % B:
                    held = codes[0, plane, pages, : x % B]
                    codes[0, plane, pages, : x % B] = _to_codes((_of_codes(held, c["code"]).double() * (was / now)[:, None, :, None]).float(), c["code"])
                codes[0, plane, pages, x % B: x % B + z.shape[1]] = _to_codes((z / now[:, None, :, None]).float(), c["code"])
    return {"codes": _of_codes(codes, c["code"]).double() if c["code"] == "e4m3" else None, "scales": scales}
