"""Measured cases of the 8-bit paged cache's later operators.

Three operators: attention of a batch whose sequences share long prefixes ("shared"), the
weight that attention gives each cached token ("weigh"), and eviction of the tokens that
received least ("evict", bookkeeping and the copies of what stays).  ``run`` computes each in
its plain form (elementary torch operations in 32 bits) or, with ``own``, through this
repository's package.

A cache holds codes [L, 2, N, B, H, d] of one byte (e4m3 or int8; plane 0 is K, 1 is V) and
float32 scales [L, 2, N, H]: a value is its code times the scale of its page and head.
Sequence r's token t lives in page tables[r, t // B], slot t % B.
"""
import math

import numpy as np
import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _shared(name, **k):
    c = dict(op="shared", groups=1, members=3, members_mix="same", prefix=300, prefix_mix="same", tail=6,
             tail_mix="same", new=1, new_mix="same", heads=32, kv_heads=8, d=128, block=16, code="e4m3",
             dtype="bf16", mix=1)
    c.update(k)
    return dict(c, name=name) if name else c


def _weigh(name, **k):
    c = dict(op="weigh", seqs=1, kv=1000, kv_mix="same", new=1, new_mix="same", heads=32, kv_heads=8, d=128,
             block=16, code="e4m3", dtype="bf16", window=0, begin=True, mix=1)
    c.update(k)
    return dict(c, name=name) if name else c


def _evict(name, **k):
    c = dict(op="evict", seqs=1, kv=777, kv_mix="same", keep=512, first=4, recent=64, layers=32, kv_heads=8,
             d=128, block=16, code="e4m3", mix=1)
    c.update(k)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one prompt answered three ways, one token each: latency
        _shared("shared_three_branches"),
        # 64 samples of one prompt, some hundred tokens into their answers
        _shared("shared_samples_64", members=64, prefix=8000, tail=500, tail_mix="ragged", mix=2),
        # a batch of forked requests: 48 prompts, 1 to 9 branches each, small heads, int8 codes, f16
        _shared("shared_many_prompts", groups=48, members=9, members_mix="ragged", prefix=2200,
                prefix_mix="lognormal", tail=200, tail_mix="ragged", heads=16, kv_heads=4, d=64, block=32,
                code="int8", dtype="f16", mix=5),
        # eight branches of a 128K context of a 32B-class model (64 query heads), 1 to 4 drafted tokens each
        _shared("shared_long_drafted", members=8, prefix=128000, tail=64, tail_mix="ragged", new=4,
                new_mix="ragged", heads=64, block=64, mix=3),
        # one user's decoded token: latency
        _weigh("weigh_one_token", kv=777, begin=False),
        # a decode step of a full server, ragged
        _weigh("weigh_decode_256", seqs=256, kv=2200, kv_mix="lognormal", mix=5),
        # the last 32 tokens of several prompts judge them before they are shortened, int8 codes, f16, small heads
        _weigh("weigh_last_rows", seqs=6, kv=16000, kv_mix="ragged", new=32, heads=16, kv_heads=4, d=64, block=32,
               code="int8", dtype="f16", mix=3),
        # an agentic turn: all 512 fresh tokens on a cached prefix of 30,720
        _weigh("weigh_turn_512", kv=31232, new=512),
        # one sequence of a small cache shortened: latency
        _evict("evict_one", layers=2),
        # a batch of prompts shortened to a quarter after they were read
        _evict("evict_prompts", seqs=8, kv=4096, kv_mix="ragged", keep=1024, recent=128, mix=2),
        # a 128K context shortened to an eighth, int8 codes
        _evict("evict_long", kv=128000, keep=16000, first=16, recent=1024, layers=8, block=64, code="int8"),
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
    base = dict(kv_heads=kv_heads, d=d, block=block, code=code, mix=mix)
    op = rng.choice(["shared", "shared", "weigh", "weigh", "evict"])
    if op == "shared":
        c = _shared("", heads=heads, dtype=dtype, **base)
        c.update(members=_log(rng, 2, 96), members_mix=rng.choice(["same", "ragged"]), prefix=_log(rng, 16, 128000),
                 tail=_log(rng, 1, 1000), tail_mix=rng.choice(["same", "ragged"]))
        if rng.random() < 0.4:
            c.update(groups=_log(rng, 2, 64), prefix_mix=rng.choice(["ragged", "lognormal"]), members=rng.randint(2, 12))
        if rng.random() < 0.3:
            c.update(new=rng.randint(2, 8), new_mix="ragged")
        return c
    if op == "weigh":
        c = _weigh("", heads=heads, dtype=dtype, begin=rng.random() < 0.5,
                   window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]), **base)
        kind = rng.choice(["token", "last", "turn"])
        if kind == "token":
            c.update(seqs=_log(rng, 1, 256), kv=_log(rng, 1, 131072), kv_mix=rng.choice(["same", "ragged", "lognormal"]))
        elif kind == "last":
            c.update(seqs=rng.randint(1, 8), kv=_log(rng, 64, 32768), kv_mix="ragged", new=rng.randint(8, 64))
        else:
            c.update(seqs=rng.randint(1, 4), kv=_log(rng, 64, 32768), new=_log(rng, 64, 2048))
            c["new"] = min(c["new"], c["kv"])
        return c
    c = _evict("", layers=rng.choice([2, 8, 32]), **base)
    c.update(seqs=_log(rng, 1, 32), kv=_log(rng, 64, 128000), kv_mix=rng.choice(["same", "ragged"]),
             first=rng.choice([0, 4, 16, 40]), recent=_log(rng, 1, 512))
    c["keep"] = max(1, int(c["kv"] * rng.uniform(0.05, 0.9)))
    return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def _fits(c):
    """Whether the plain form's temporaries and the state stay within a few GB."""
    if c["op"] == "evict":
        return _evict_pages(c) * c["block"] * c["kv_heads"] * c["d"] * 2 * c["layers"] <= 2300 << 20
    if c["op"] == "shared":
        t = _shared_sizes(c)
        S, rows, k = len(t["lens"]), int(t["rows"].max()), int(t["whole"].max())
        g, tail = c["groups"], int((t["lens"] - t["whole"][t["group"]]).max()) + c["block"]
        words = g * k * c["kv_heads"] * c["d"] + g * rows * c["heads"] * k
        return max(words, S * tail * c["kv_heads"] * c["d"]) * 4 <= 6 << 30
    kv, new = _lengths(c)
    s, k, n = len(kv), int(kv.max()), int(new.max())
    return s * k * c["kv_heads"] * c["d"] * 4 <= 9 << 30 and s * (c["heads"] // c["kv_heads"]) * n * k * 4 <= 3 << 30


# ---- sizes a case stands for (from the case alone) ------------------------------------

def _spread(mix, n, size, how, low=1):
    g = np.random.RandomState(mix)
    if how == "ragged":
        return np.maximum(low, g.randint(1, size + 1, n)).astype(np.int64)
    if how == "lognormal":
        return np.clip(np.rint(g.lognormal(math.log(size), 0.5, n)), max(1, size // 8), size * 4).astype(np.int64)
    return np.full(n, size, np.int64)


def _lengths(c):
    """(tokens held, fresh tokens) of each sequence: the fresh ones are the last held."""
    kv = _spread(c["mix"], c["seqs"], c["kv"], c["kv_mix"])
    new = _spread(c["mix"] + 1, c["seqs"], c["new"], c["new_mix"])
    return np.maximum(kv, new), new


def _shared_sizes(c):
    """Sequences of a "shared" case: their group, tokens and fresh tokens; the whole pages' tokens that a
    group shares, and its rows."""
    members = _spread(c["mix"], c["groups"], c["members"], c["members_mix"])
    prefix = _spread(c["mix"] + 1, c["groups"], c["prefix"], c["prefix_mix"])
    group = np.repeat(np.arange(c["groups"]), members)
    new = _spread(c["mix"] + 2, group.size, c["new"], c["new_mix"])
    tail = np.maximum(_spread(c["mix"] + 3, group.size, c["tail"], c["tail_mix"]), new)
    return {"members": members, "group": group, "new": new, "lens": prefix[group] + tail,
            "whole": prefix // c["block"] * c["block"], "rows": np.bincount(group, new, c["groups"]).astype(np.int64)}


def _evict_pages(c):
    kv = _spread(c["mix"], c["seqs"], c["kv"], c["kv_mix"])
    B = c["block"]
    return max(8, int(1.1 * (int((-(-kv // B)).sum()) + c["seqs"] * (-(-c["keep"] // B) + 1))))


def _pairs(c):
    """Visible (query, key) pairs summed over the sequences, and tokens any query sees."""
    kv, new = _lengths(c)
    pairs, seen = 0, 0
    for k, n in zip(kv.tolist(), new.tolist()):
        pos = np.arange(k - n, k, dtype=np.int64)
        lo = np.maximum(0, pos + 1 - c["window"]) if c["window"] else np.zeros(n, np.int64)
        pairs += int((pos + 1 - lo).sum())
        seen += int(k - lo.min())
    return pairs, seen


def work(case):
    c = case
    H, d, B = c["kv_heads"], c["d"], c["block"]
    if c["op"] == "shared":
        t = _shared_sizes(c)
        tails = t["lens"] - t["whole"][t["group"]]
        held = int(t["whole"].sum() + tails.sum())
        rows = int(t["new"].sum())
        pairs = int((t["new"] * t["lens"] - t["new"] * (t["new"] - 1) // 2).sum())
        b = held * H * d * 2 + 8 * H * -(-held // B) + rows * c["heads"] * (4 * d + 4)
        return {"bytes": b, "flops": 4 * pairs * c["heads"] * d}
    if c["op"] == "weigh":
        pairs, seen = _pairs(c)
        kv, new = _lengths(c)
        rows = int(new.sum())
        b = seen * H * d + 4 * H * -(-seen // B) + rows * c["heads"] * (2 * d + 4) + 8 * int(kv.sum())
        return {"bytes": b, "flops": 2 * pairs * c["heads"] * d}
    kv = _spread(c["mix"], c["seqs"], c["kv"], c["kv_mix"])
    cut = kv[kv > c["keep"]]
    moved = len(cut) * (c["keep"] - min(c["first"], c["keep"]) // B * B)
    b = moved * c["layers"] * 2 * 2 * H * d + 16 * H * c["layers"] * (moved // B) + 8 * int(cut.sum()) + 12 * c["seqs"]
    return {"bytes": b, "flops": 0}


# ---- inputs -----------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _fill_cache(g, N, c):
    """Codes and scales of one layer's pool holding normal values, some heads and channels larger."""
    B, H, d = c["block"], c["kv_heads"], c["d"]
    codes = torch.empty((1, 2, N, B, H, d), dtype=torch.uint8, device="cuda")
    scales = torch.empty((1, 2, N, H), dtype=torch.float32, device="cuda")
    gain = torch.exp(0.5 * torch.randn((2, 1, 1, H, 1), generator=g, device="cuda"))
    gain = gain * torch.exp(0.3 * torch.randn((2, 1, 1, H, d), generator=g, device="cuda"))
    step = max(1, (1 << 28) // (B * H * d))
    for p in range(2):
        for a in range(0, N, step):
            x = torch.randn((min(step, N - a), B, H, d), generator=g, device="cuda") * gain[p]
            s = x.abs().amax(dim=(1, 3)) / QMAX[c["code"]]
            scales[0, p, a:a + step] = s
            codes[0, p, a:a + step] = _to_codes(x / s[:, None, :, None], c["code"])
    return codes, scales


def _to_codes(x, code):
    x = x.clamp(-QMAX[code], QMAX[code])
    if code == "e4m3":
        return x.to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.round(x).to(torch.int8).view(torch.uint8)


def _of_codes(u8, code):
    return u8.view(_value_type(code)).float()


def _value_type(code):
    return torch.float8_e4m3fn if code == "e4m3" else torch.int8


def _tables(g, kv, B, N):
    """Block tables [S, W] of sequences of kv tokens from a shuffled pool of N pages."""
    n = -(-kv // B)
    perm = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
    W = max(1, int(n.max()))
    starts = _dev(np.concatenate([[0], np.cumsum(n)[:-1]]))
    w = torch.arange(W, device="cuda")[None, :]
    at = (starts[:, None] + w).clamp(max=N - 1)
    return torch.where(w < _dev(n)[:, None], perm[at], torch.full((), -1, dtype=torch.int32, device="cuda")).contiguous()


def _refs(tables, N):
    t = tables[tables >= 0].long()
    return torch.zeros(N, dtype=torch.int32, device="cuda").index_add_(0, t, torch.ones_like(t, dtype=torch.int32))


def _starts(new):
    return _dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))


def _cache(s, c):
    if own:
        from layer_wise_paged_gb300 import cache
        s["cache"] = cache.QuantCache(s["codes"], s["scales"], s["tables"], s["lens"], s["refs"], code=c["code"])
    return s


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    B, H, d = c["block"], c["kv_heads"], c["d"]
    if c["op"] == "evict":
        return _prepare_evict(c, s, g)
    dt = DTYPES[c["dtype"]]
    if c["op"] == "shared":
        t = _shared_sizes(c)
        kv, new, whole = t["lens"], t["new"], t["whole"]
        own_kv = kv - whole[t["group"]]
        N = int(math.ceil(1.25 * int((-(-own_kv // B)).sum() + (whole // B).sum())))
        # a group's whole pages, then each sequence's own
        both = _tables(g, np.concatenate([whole, own_kv]), B, N)
        first, rest = both[: c["groups"]], both[c["groups"]:]
        W = int((-(-kv // B)).max())
        w = torch.arange(W, device="cuda")[None, :]
        group, n = _dev(t["group"]), _dev(whole // B)[_dev(t["group"])][:, None]
        one = first[group].gather(1, w.clamp(max=first.shape[1] - 1).expand(len(kv), W))
        two = rest.gather(1, (w - n).clamp(min=0, max=rest.shape[1] - 1))
        s["tables"] = torch.where(w < n, one, torch.where(w < _dev(-(-kv // B))[:, None], two, -1)).contiguous()
        s["groups"] = _starts(t["members"])
        s["shared"] = _dev(whole.astype(np.int32))
        s["max_rows"], s["max_whole"] = int(t["rows"].max()), int(whole.max())
        s["max_tail"] = int(own_kv.max())
    else:
        kv, new = _lengths(c)
        N = int(math.ceil(1.25 * int((-(-kv // B)).sum())))
        s["tables"] = _tables(g, kv, B, N)
    s["codes"], s["scales"] = _fill_cache(g, N, c)
    s["lens"] = _dev(kv.astype(np.int32))
    s["starts"] = _starts(new)
    s["refs"] = _refs(s["tables"], N)
    s["max_new"] = int(new.max())
    T = int(new.sum())
    # q beside k and v, as a fused projection leaves them
    s["q"] = torch.randn((T, c["heads"] + 2 * H, d), generator=g, device="cuda").to(dt)[:, : c["heads"]]
    s["lse"] = torch.empty((T, c["heads"]), dtype=torch.float32, device="cuda")
    if c["op"] == "shared":
        s["out"] = torch.empty((T, c["heads"], d), dtype=dt, device="cuda")
        return _cache(s, c)
    _fill_lse(s, c)
    cap = s["tables"].shape[1] * B
    s["mass"] = torch.rand((c["seqs"], cap), generator=g, device="cuda") * 0.1
    s["mass_out"] = torch.zeros((c["seqs"], cap), dtype=torch.float32, device="cuda")
    return _cache(s, c)


def _prepare_evict(c, s, g):
    B, H, d, L = c["block"], c["kv_heads"], c["d"], c["layers"]
    kv = _spread(c["mix"], c["seqs"], c["kv"], c["kv_mix"])
    N = _evict_pages(c)
    # any codes but e4m3's NaN, int8's -128
    r = torch.randint(0, 254, (L, 2, N, B, H, d), generator=g, device="cuda", dtype=torch.uint8)
    s["codes"] = r + (r > 126) if c["code"] == "e4m3" else r - 127
    s["scales"] = torch.rand((L, 2, N, H), generator=g, device="cuda") + 0.5
    s["tables"] = _tables(g, kv, B, N)
    s["lens"] = _dev(kv.astype(np.int32))
    s["refs"] = _refs(s["tables"], N)
    # a few tokens receive most of the weight, some none at all
    m = torch.exp(2 * torch.randn((c["seqs"], s["tables"].shape[1] * B), generator=g, device="cuda"))
    s["mass"] = m * (torch.rand(m.shape, generator=g, device="cuda") > 0.1)
    for k in ("tables", "lens", "refs", "mass"):
        s[k + "0"] = s[k].clone()
    s["slots"] = torch.arange(c["seqs"], dtype=torch.int32, device="cuda")
    s["keep"] = torch.full((c["seqs"],), c["keep"], dtype=torch.int32, device="cuda")
    return _cache(s, c)


# ---- one pass -----------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if c["op"] == "shared":
        if own:
            s["cache"].attend_shared(0, s["q"], s["starts"], s["groups"], s["shared"], out=s["out"], lse=s["lse"],
                                     max_new=s["max_new"])
            return {"out": s["out"], "lse": s["lse"]}
        return _plain_shared(s, c)
    if c["op"] == "weigh":
        if own:
            s["cache"].weigh(0, s["q"], s["starts"], s["lse"], s["mass"], out=s["mass_out"], begin=c["begin"],
                             window=c["window"], max_new=s["max_new"])
        else:
            _plain_weigh(s, c)
        return {"mass": s["mass_out"]}
    # the program's snapshot of its bookkeeping, so that there is something to evict
    for k in ("tables", "lens", "refs", "mass"):
        s[k].copy_(s[k + "0"])
    if own:
        s["cache"].evict(s["slots"], s["keep"], s["mass"], first=c["first"], recent=c["recent"])
        s["cache"].move_tokens()
    else:
        _plain_evict(s, c)
    out = {k: s[k] for k in ("tables", "lens", "refs", "mass", "scales")}
    return dict(out, codes=s["codes"].view(_value_type(c["code"])))


def _plane(s, c, p, pages):
    """Values [..., pages * B, H, d] of plane p in 32 bits."""
    B, H, d = c["block"], c["kv_heads"], c["d"]
    x = _of_codes(s["codes"][0, p][pages], c["code"]) * s["scales"][0, p][pages][..., None, :, None]
    return x.reshape(*pages.shape[:-1], pages.shape[-1] * B, H, d)


def _softmax_parts(q, k, v, see, d):
    """Maximum, sum and weighted values of rows q [n, H, r, d] over k, v [n, t, H, d] where see [n, 1, r, t]."""
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(d))
    x.masked_fill_(~see, float("-inf"))
    m = x.amax(dim=-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.full_like(m, -1e30), m)
    p = x.sub_(m).exp_()
    return m, p.sum(dim=-1, keepdim=True), torch.matmul(p, v.transpose(1, 2))


def _plain_shared(s, c):
    B, H, d, G = c["block"], c["kv_heads"], c["d"], c["heads"] // c["kv_heads"]
    lens, starts, groups, shared = (s[k].long() for k in ("lens", "starts", "groups", "shared"))
    T, S, n = s["q"].shape[0], lens.shape[0], s["max_new"]
    group = torch.searchsorted(groups[1:], torch.arange(S, device="cuda"), right=True)
    pages = s["tables"].long().clamp(min=0)
    q = s["q"].float().reshape(T, H, G, d)
    # the shared tokens, for all rows of a group at once
    n1 = s["max_rows"]
    i1 = torch.arange(n1, device="cuda")[None, :]
    r0, r1 = starts[groups[:-1]], starts[groups[1:]]
    rows1 = (r0[:, None] + i1).clamp(max=T - 1)
    p1 = pages[groups[:-1]][:, : max(1, s["max_whole"] // B)]
    see = (torch.arange(p1.shape[1] * B, device="cuda")[None, :] < shared[:, None])[:, None, None, :]
    q1 = q[rows1].permute(0, 2, 3, 1, 4).reshape(len(shared), H, G * n1, d)
    part1 = _softmax_parts(q1, _plane(s, c, 0, p1), _plane(s, c, 1, p1), see, d)
    # each sequence's own
    i2 = torch.arange(n, device="cuda")[None, :]
    new = starts[1:] - starts[:-1]
    rows2 = (starts[:-1, None] + i2).clamp(max=T - 1)
    base = shared[group]
    w = torch.arange(-(-s["max_tail"] // B), device="cuda")[None, :] + (base // B)[:, None]
    p2 = pages.gather(1, w.clamp(max=pages.shape[1] - 1))
    j = base[:, None] + torch.arange(p2.shape[1] * B, device="cuda")[None, :]
    pos = (lens - new)[:, None] + i2
    see = (j[:, None, :] <= pos[:, :, None]) & (j < lens[:, None])[:, None, :]
    q2 = q[rows2].permute(0, 2, 3, 1, 4).reshape(S, H, G * n, d)
    see = see[:, None].expand(S, G, n, -1).reshape(S, 1, G * n, -1)
    there = (j < lens[:, None])[:, :, None, None]
    k2, v2 = (torch.where(there, _plane(s, c, p, p2), 0.0) for p in (0, 1))
    part2 = _softmax_parts(q2, k2, v2, see, d)
    # row by row
    take1, take2 = i1 < (r1 - r0)[:, None], i2 < new[:, None]
    m1, l1, o1 = (x.reshape(len(shared), H, G, n1, -1).permute(0, 3, 1, 2, 4)[take1] for x in part1)
    m2, l2, o2 = (x.reshape(S, H, G, n, -1).permute(0, 3, 1, 2, 4)[take2] for x in part2)
    m = torch.maximum(m1, m2)
    a, b = torch.exp(m1 - m), torch.exp(m2 - m)
    l = l1 * a + l2 * b
    out = (o1 * a + o2 * b) / l
    return {"out": out.reshape(T, H * G, d).to(s["q"].dtype), "lse": (m + torch.log(l)).reshape(T, H * G)}


def _scores(s, c, h):
    """Scores of KV head h, [S, G, n, W * B] in 32 bits, -infinity where nothing is seen; the rows' numbers and
    which of them there are."""
    B, d, G, n = c["block"], c["d"], c["heads"] // c["kv_heads"], s["max_new"]
    lens, starts = s["lens"].long(), s["starts"].long()
    new = starts[1:] - starts[:-1]
    pages = s["tables"].long().clamp(min=0)
    S, W = pages.shape
    j = torch.arange(W * B, device="cuda")
    k = _of_codes(s["codes"][0, 0, :, :, h][pages], c["code"]) * s["scales"][0, 0, :, h][pages][:, :, None, None]
    k = torch.where((j[None, :] < lens[:, None])[:, :, None], k.reshape(S, W * B, d), 0.0)
    i = torch.arange(n, device="cuda")
    rows = (starts[:-1, None] + i[None, :]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][:, h * G:(h + 1) * G][rows].float().permute(0, 2, 1, 3).reshape(S, G * n, d)
    x = torch.matmul(q, k.transpose(1, 2)).mul_(1.0 / math.sqrt(d)).reshape(S, G, n, W * B)
    pos = (lens - new)[:, None] + i[None, :]
    see = j[None, None, :] <= pos[:, :, None]
    if c["window"]:
        see &= j[None, None, :] > pos[:, :, None] - c["window"]
    see &= (i[None, :] < new[:, None])[:, :, None]
    return x.masked_fill_(~see[:, None], float("-inf")), rows, i[None, :] < new[:, None]


def _fill_lse(s, c):
    G = c["heads"] // c["kv_heads"]
    for h in range(c["kv_heads"]):
        x, rows, there = _scores(s, c, h)
        s["lse"][:, h * G:(h + 1) * G] = torch.logsumexp(x, dim=-1).permute(0, 2, 1)[there]


def _plain_weigh(s, c):
    G = c["heads"] // c["kv_heads"]
    lens, new = s["lens"].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    total = None
    for h in range(c["kv_heads"]):
        x, rows, there = _scores(s, c, h)
        lse = s["lse"][:, h * G:(h + 1) * G][rows].permute(0, 2, 1)
        w = x.sub_(lse[..., None]).exp_().sum(dim=(1, 2))
        total = w if total is None else total + w
    j = torch.arange(total.shape[1], device="cuda")[None, :]
    old = torch.where(j >= (lens - new)[:, None], 0.0, s["mass"]) if c["begin"] else s["mass"]
    s["mass_out"].copy_(torch.where(j < lens[:, None], old + total, s["mass_out"]))


def _kept(s, c):
    """Which tokens stay, [S, cap]: all of a short sequence; else the first, the last and the heaviest."""
    lens, keep = s["lens"].long()[:, None], s["keep"].long()[:, None]
    S, cap = s["mass"].shape
    j = torch.arange(cap, device="cuda")[None, :]
    first = torch.clamp(keep, max=c["first"])
    recent = torch.clamp(keep - first, max=c["recent"])
    sure = (j < first) | (j >= lens - recent)
    key = torch.where(sure, float("inf"), s["mass"]).masked_fill_(j >= lens, float("-inf"))
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, j.expand(S, cap).contiguous())
    return ((rank < keep) | (lens <= keep)) & (j < lens)


def _plain_evict(s, c):
    B, N = c["block"], s["refs"].shape[0]
    kept = _kept(s, c)
    S, cap = kept.shape
    lens = s["lens"].long()
    cut = lens > s["keep"].long()
    held, n = (lens + B - 1) // B, (torch.minimum(lens, s["keep"].long()) + B - 1) // B
    u = torch.clamp(s["keep"].long(), max=c["first"]) // B  # pages that stay
    w = torch.arange(s["tables"].shape[1], device="cuda")[None, :]
    take = cut[:, None] & (w >= u[:, None]) & (w < n[:, None])
    gone = cut[:, None] & (w >= u[:, None]) & (w < held[:, None])
    old = s["tables"].clone()
    # kept tokens of shortened sequences, and where they go
    r, at = torch.nonzero(kept & cut[:, None], as_tuple=True)
    to = (torch.cumsum(kept, dim=1) - 1)[r, at]
    s["mass"][:] = torch.where(cut[:, None], torch.zeros_like(s["mass"]).index_put((r, to), s["mass"][r, at]), s["mass"])
    got = torch.nonzero(s["refs"] == 0)[:, 0][: int(take.sum())].to(torch.int32)
    s["tables"][take] = got
    s["refs"][got.long()] = 1
    dropped = old[gone].long()
    s["refs"].index_add_(0, dropped, torch.full_like(dropped, -1, dtype=torch.int32))
    s["lens"].copy_(torch.where(cut, s["keep"], s["lens"]))
    # their codes, under the largest of the scales that meet in a page
    moves = to >= (u * B)[r]
    r, at, to = r[moves], at[moves], to[moves]
    src, dst = old[r, at // B].long(), s["tables"][r, to // B].long()
    for l in range(c["layers"]):
        for p in range(2):
            codes, scales = s["codes"][l, p], s["scales"][l, p]
            was = scales[src]
            now = torch.zeros_like(scales).index_reduce_(0, dst, was, "amax")
            scales[got.long()] = now[got.long()]
            x = _of_codes(codes[src, at % B], c["code"]) * (was / now[dst])[..., None]
            codes[dst, to % B] = _to_codes(x, c["code"])


# ---- the same outputs from the definitions in 64 bits ---------------------------------------

def exact(case, seed):
    global own
    c = case
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if c["op"] == "shared":
        return _exact_attention(s, c)
    return _exact_weigh(s, c) if c["op"] == "weigh" else _exact_evict(s, c)


def _tokens_of(s, c, r, p, h):
    """Values [len, d] of sequence r, plane p, head h."""
    at = torch.arange(int(s["lens"][r]), device="cuda")
    page = s["tables"][r].long()[at // c["block"]]
    u8 = s["codes"][0, p, :, :, h][page, at % c["block"]]
    return u8.view(_value_type(c["code"])).double() * s["scales"][0, p, :, h].double()[page, None]


def _logits(s, c, r, h, a, b, k):
    """Scores [G, b - a, len] of rows a .. b of sequence r, -infinity where nothing is seen."""
    G, n, end = c["heads"] // c["kv_heads"], k.shape[0], int(s["starts"][r + 1])
    x = s["q"][a:b, h * G:(h + 1) * G].double().transpose(0, 1) @ k.T / math.sqrt(c["d"])
    ahead = torch.arange(n, device="cuda")[None, :] - torch.arange(n - (end - a), n - (end - b), device="cuda")[:, None]
    hide = ahead > 0
    if c.get("window"):
        hide |= ahead <= -c["window"]
    return x.masked_fill_(hide, float("-inf"))


def _exact_attention(s, c):
    """As if nothing were shared."""
    G, T = c["heads"] // c["kv_heads"], s["q"].shape[0]
    out = torch.zeros((T, c["heads"], c["d"]), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, c["heads"]), dtype=torch.float64, device="cuda")
    starts = s["starts"].tolist()
    for r in range(len(starts) - 1):
        a, b = starts[r], starts[r + 1]
        for h in range(c["kv_heads"]):
            x = _logits(s, c, r, h, a, b, _tokens_of(s, c, r, 0, h))
            lse[a:b, h * G:(h + 1) * G] = torch.logsumexp(x, dim=-1).T
            out[a:b, h * G:(h + 1) * G] = (torch.softmax(x, dim=-1) @ _tokens_of(s, c, r, 1, h)).transpose(0, 1)
    return {"out": out, "lse": lse}


def _exact_weigh(s, c):
    """From the lse that the inputs hold."""
    G = c["heads"] // c["kv_heads"]
    mass = s["mass_out"].double()
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    for r, n in enumerate(lens):
        a, b = starts[r], starts[r + 1]
        w = s["mass"][r, :n].double()
        if c["begin"]:
            w[n - (b - a):] = 0
        for h in range(c["kv_heads"]):
            k = _tokens_of(s, c, r, 0, h)
            for i in range(a, b, 512):
                e = min(b, i + 512)
                x = _logits(s, c, r, h, i, e, k)
                w += torch.exp(x - s["lse"][i:e, h * G:(h + 1) * G].double().T[..., None]).sum(dim=(0, 1))
        mass[r, :n] = w
    return {"mass": mass}


def _exact_evict(s, c):
    B, tables, lens = c["block"], s["tables"].tolist(), s["lens"].tolist()
    codes, scales, mass = s["codes"], s["scales"].double(), s["mass"].double()
    free = torch.nonzero(s["refs"] == 0)[:, 0].tolist()
    k, before = c["keep"], codes.clone()
    f = min(c["first"], k)
    e = min(c["recent"], k - f)
    u = f // B
    for r, n in enumerate(lens):
        if n <= k:
            continue
        m = s["mass"][r, f:n - e].cpu().numpy()
        middle = np.argsort(-m, kind="stable")[: k - f - e] + f
        at = _dev(np.concatenate([np.arange(f), np.sort(middle), np.arange(n - e, n)]))
        mass[r] = 0
        mass[r, :k] = s["mass"][r].double()[at]
        pages = torch.tensor([free.pop(0) for _ in range(-(-k // B) - u)], dtype=torch.int64, device="cuda")
        if not len(pages):
            continue
        # tokens by page; the last one again where the last page has room
        t = at[torch.arange(u * B, (u + len(pages)) * B, device="cuda").clamp(max=k - 1)].reshape(-1, B)
        src = torch.tensor(tables[r], device="cuda")[t // B]
        held = (torch.arange(u * B, (u + len(pages)) * B, device="cuda") < k).reshape(-1, B)
        for l in range(c["layers"]):
            for p in range(2):
                was = scales[l, p][src]                   # [pages, B, H]
                now = was.amax(dim=1, keepdim=True)
                scales[l, p, pages] = now[:, 0]
                x = before[l, p][src, t % B].view(_value_type(c["code"])).double() * (was / now)[..., None]
                codes[l, p, pages] = torch.where(held[..., None, None], _to_codes(x.float(), c["code"]), codes[l, p, pages])
    values = codes.view(_value_type(c["code"])).float() if c["code"] == "e4m3" else None
    return {"tables": None, "lens": None, "refs": None, "mass": mass, "scales": scales, "codes": values}
