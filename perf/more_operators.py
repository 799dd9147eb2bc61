"""Cases of what a serving step does around the paged cache: pages and index arrays
worked out on the GPU, norms of queries and keys with the rotation and the cache write
in one pass, attention with a sliding window and first tokens that stay visible, and
attention of a batch that shares a long prefix.

Shapes are those of the framework's own configurations: 32 query / 8 KV heads of 128
or 64 and the small 8 / 2 heads, verify chunks of K + 1 tokens, contexts of 512 to
16384, batches of 1 to 64.  With ``own`` False every operator is computed in plain
torch operations in 32 bits (angles in 64) and rounded once; with ``own`` True by the
package's calls.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ES = {"f32": 4, "bf16": 2, "e4m3": 1}
THETA, EPS = 500000.0, 1e-5


def listed():
    return [
        # pages and index arrays of one verify step (K = 5) of a batch, and the rejected rows' pages back
        {"name": "pages-verify-64x6", "op": "pages", "batch": 64, "q": 6, "ctx": 4096, "page": 16, "ragged": False},
        # the same for a wave of new prompts of different lengths
        {"name": "pages-prompts-64x16384", "op": "pages", "batch": 64, "q": 16384, "ctx": 0, "page": 16,
         "ragged": True},
        # one verify step of one sequence, from the fp32 q/k/v projection into a 16-bit cache
        {"name": "norm-append-1x6-bf16", "op": "append", "batch": 1, "q": 6, "ctx": 512, "heads": 32, "kv_heads": 8,
         "head_dim": 128, "page": 16, "in": "f32", "cache": "bf16"},
        # four prompts' rows into an 8-bit cache
        {"name": "norm-append-4x4000-e4m3", "op": "append", "batch": 4, "q": 4000, "ctx": 4096, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 64, "in": "bf16", "cache": "e4m3"},
        # plain decoding of 16 long contexts with the 1B-shaped heads: window of 1024, four first tokens
        {"name": "window-decode-16x1-16384", "op": "window", "batch": 16, "q": 1, "ctx": 16384, "heads": 32,
         "kv_heads": 8, "head_dim": 64, "page": 32, "cache": "bf16", "window": 1024, "sinks": 4, "ragged": False},
        # the verify step of 64 sequences over an 8-bit cache, window of 4096
        {"name": "window-verify-64x6-16384-e4m3", "op": "window", "batch": 64, "q": 6, "ctx": 16384, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 16, "cache": "e4m3", "window": 4096, "sinks": 4, "ragged": False},
        # chunks of new prompt tokens of different lengths over long contexts
        {"name": "window-chunk-4x512-16384", "op": "window", "batch": 4, "q": 512, "ctx": 16384, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 64, "cache": "bf16", "window": 2048, "sinks": 4, "ragged": True},
        # six long prompts of different lengths, packed
        {"name": "window-prompt-6x4096", "op": "prompt", "batch": 6, "len": 4096, "heads": 32, "kv_heads": 8,
         "head_dim": 128, "window": 1024, "sinks": 4},
        # the smallest shared batch: verify steps of four sequences behind a 512-token prompt
        {"name": "shared-verify-4x6-512", "op": "shared", "batch": 4, "q": 6, "groups": 1, "prefix": 512, "rest": 64,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 16, "cache": "bf16"},
        # plain decoding of 64 sequences behind one long prompt
        {"name": "shared-decode-64x1-16384", "op": "shared", "batch": 64, "q": 1, "groups": 1, "prefix": 16384,
         "rest": 512, "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 16, "cache": "bf16"},
        # verify steps behind four prompts, 8-bit cache
        {"name": "shared-verify-64x6-8192-e4m3", "op": "shared", "batch": 64, "q": 6, "groups": 4, "prefix": 8192,
         "rest": 300, "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 32, "cache": "e4m3"},
        # queries and keys of packed prompts, normed and rotated without a cache (the 1B-shaped heads)
        {"name": "norm-rope-16381", "op": "rows", "tokens": 16381, "heads": 32, "kv_heads": 8, "head_dim": 64,
         "in": "bf16", "out": "bf16", "interleaved": False, "first": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "append", "rows", "window", "window", "prompt", "shared", "shared"])
    hd = rng.choice([64, 128])
    hq, hkv = rng.choice([(8, 2), (32, 8), (32, 8), (12, 4), (16, 2), (7, 1)])
    page = rng.choice([16, 32, 64])
    cache = rng.choice(["bf16", "e4m3"])
    window, sinks = _log(rng, 16, 4096), rng.choice([0, 1, 4, 4, 16, 100])
    if op == "pages":
        b = _log(rng, 1, 512)
        q = rng.choice([1, 6, 9, _log(rng, 10, 16384)])
        q = max(1, min(q, 1000000 // b))
        return {"op": op, "batch": b, "q": q, "ctx": _log(rng, 1, 16384), "page": page, "ragged": rng.random() < 0.5}
    if op == "append":
        b = _log(rng, 1, 64)
        q = _log(rng, 1, max(2, 16000 // b))
        return {"op": op, "batch": b, "q": q, "ctx": q + _log(rng, 1, 4096), "heads": hq, "kv_heads": hkv,
                "head_dim": hd, "page": page, "in": rng.choice(["f32", "bf16"]), "cache": cache}
    if op == "rows":
        return {"op": op, "tokens": _log(rng, 1, 16384), "heads": hq, "kv_heads": hkv, "head_dim": hd,
                "in": rng.choice(["f32", "bf16"]), "out": rng.choice(["f32", "bf16"]),
                "interleaved": rng.random() < 0.5, "first": _log(rng, 1, 500000)}
    if op == "window":
        b = _log(rng, 1, 64)
        q = rng.choice([1, 2, 4, 6, 9, _log(rng, 10, 512)])
        q = min(q, max(1, 1024 // b))
        ctx = max(q, _log(rng, 64, 16384))
        return {"op": op, "batch": b, "q": q, "ctx": ctx, "heads": hq, "kv_heads": hkv, "head_dim": hd, "page": page,
                "cache": cache, "window": window, "sinks": sinks, "ragged": rng.random() < 0.5}
    if op == "prompt":
        b = _log(rng, 1, 16)
        return {"op": op, "batch": b, "len": _log(rng, 8, min(4096, 16384 // b)), "heads": hq, "kv_heads": hkv,
                "head_dim": hd, "window": window, "sinks": sinks}
    b = _log(rng, 2, 64)
    q = min(rng.choice([1, 2, 4, 6, 9, 40]), max(1, 512 // b))
    groups = rng.choice([1, 1, 2, min(5, b)])
    return {"op": op, "batch": b, "q": q, "groups": groups, "prefix": _log(rng, 64, 16384 // groups),
            "rest": q + _log(rng, 1, 512), "heads": hq, "kv_heads": hkv, "head_dim": hd, "page": page, "cache": cache}


def _lens(case):
    """(new tokens, context lengths) of a case's sequences, from the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    b = case["batch"]
    if case["op"] == "prompt":
        n = [rng.randint(max(1, case["len"] // 4), case["len"]) for _ in range(b)]
        n[rng.randrange(b)] = case["len"]
        return n, n
    q = [case["q"]] * b
    if case.get("ragged"):
        q = [_log(rng, 1, case["q"]) for _ in range(b)]
        q[rng.randrange(b)] = case["q"]
    if case["op"] == "shared":       # lengths behind the prefix
        rest = [rng.randint(max(n, case["rest"] // 4), max(n, case["rest"])) for n in q]
        return q, rest
    if case["op"] == "pages":        # lengths before the step
        return q, [rng.randint((case["ctx"] + 1) // 2, case["ctx"]) for _ in q]
    ctx = [max(n, rng.randint((case["ctx"] + 1) // 2, case["ctx"])) for n in q]
    ctx[rng.randrange(b)] = case["ctx"]
    return q, ctx


def _groups(case):
    """First sequence of every group, and the shared lengths (whole pages and others)."""
    rng = random.Random("g" + repr(sorted((k, v) for k, v in case.items() if k != "name")))
    g, b = case["groups"], case["batch"]
    first = [0] + sorted(rng.sample(range(1, b), g - 1)) + [b]
    shared = [case["prefix"]] + [rng.randint((case["prefix"] + 1) // 2, case["prefix"]) for _ in range(g - 1)]
    return first, shared


# ------------------------------------------------------------------ inputs
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rows(n, first):
    """Per packed row: its sequence, its index in the sequence's rows and its position."""
    seq = torch.repeat_interleave(torch.arange(len(n)), torch.tensor(n))
    idx = torch.cat([torch.arange(x) for x in n])
    pos = idx + torch.tensor(first)[seq]
    return seq.int().cuda(), idx.int().cuda(), pos.int().cuda()


def _cu(n):
    return _i32([sum(n[:i]) for i in range(len(n) + 1)])


def _kv_like(g, *shape):
    """Keys / values: normal, with a spread of channel scales as trained projections have."""
    x = torch.randn(*shape, generator=g, device="cuda")
    return x.mul_(torch.exp(0.4 * torch.randn(*shape[1:2], shape[-1], generator=g, device="cuda")).view(
        shape[1], *([1] * (len(shape) - 3)), shape[-1]))


def _encode(x):
    """8-bit rows: (codes, exponent byte e + 127), value = code * 2^e with the smallest e (held in
    -60..60) that keeps the row's largest magnitude within 448."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)
    e = (e - 9 + (m > 0.875).int()).clamp(-60, 60)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    codes = torch.ldexp(x, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _pools(case, per, lead, g):
    """The pools of a cache in use: shuffled pages, some not owned by any of the sequences.  per: pages
    of every sequence, of which the first lead[b] are those of sequence first[b]."""
    ps, h, d = case["page"], case["kv_heads"], case["head_dim"]
    own_pages = sum(n - (k if b != f else 0) for b, (n, (k, f)) in enumerate(zip(per, lead)))
    pages = own_pages + max(1, own_pages // 8)
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.zeros(len(per), max(per), dtype=torch.int32, device="cuda")
    at = 0
    for b, (n, (k, f)) in enumerate(zip(per, lead)):
        k = k if b != f else 0
        table[b, :k] = table[f, :k]
        table[b, k:n] = order[at:at + n - k]
        at += n - k
    s = {"table": table}
    for name in ("k", "v"):
        x = _kv_like(g, pages, h, ps, d)
        if case["cache"] == "e4m3":
            s[name], s[name + "_scale"] = _encode(x)
        else:
            s[name] = x.bfloat16()
        del x
    if own:
        import speculative_decoding_verification_step_gb300 as sv
        s["cache"] = sv.KVCache(s["k"], s["v"], table, s.get("k_scale"), s.get("v_scale"))
    return s


def _plan(dim, interleaved, s):
    """The rotation a program keeps: its frequencies (radians of the pairs per position)."""
    s["freq"] = (THETA ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)).cuda()
    s["inter"] = interleaved
    if own:
        import speculative_decoding_verification_step_gb300 as sv
        s["plan"] = sv.rope_plan(dim, THETA, interleaved=interleaved)


def _prepare_pages(case, g):
    n, lens = _lens(case)
    ps, b = case["page"], len(lens)
    had = [-(-c // ps) for c in lens]
    need = [-(-(c + m) // ps) - h for c, m, h in zip(lens, n, had)]
    pages = sum(had) + sum(need) + max(8, b // 2)
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((b, max(h + m for h, m in zip(had, need)) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, h in enumerate(had):
        table[i, :h] = order[at:at + h]
        at += h
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[:pages - at] = order[at:].flip(0)
    # accepted tokens that stay within the last page that a sequence had
    keep = [min(c + m // 2, h * ps) for c, m, h in zip(lens, n, had)]
    s = {"case": case, "table": table, "free": free, "n_free": _i32([pages - at]), "lens": _i32(lens),
         "counts": _i32(n), "keep": _i32(keep), "tokens": sum(n) + 64, "ps": ps}
    if own:
        import speculative_decoding_verification_step_gb300 as sv
        s["cache"] = sv.KVCache.empty(pages, ps, 1, 32, table)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    op = case["op"]
    if op == "pages":
        return _prepare_pages(case, g)
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    if op in ("append", "rows"):
        s["norm"] = torch.exp(0.3 * torch.randn(2, d, generator=g, device="cuda"))
    if op == "rows":
        x = torch.randn(case["tokens"], h + 2 * hk, d, generator=g, device="cuda")
        s["x"] = x.to(DT[case["in"]])[:, :h + hk]           # the q and k heads of a fused projection
        s["pos"] = (case["first"] + torch.arange(case["tokens"])).int().cuda()
        s["gain"] = torch.cat([s["norm"][0].expand(h, d), s["norm"][1].expand(hk, d)])   # of every head
        _plan(d, case["interleaved"], s)
        return s
    n, ctx = _lens(case)
    if op == "prompt":
        x = torch.cat([torch.randn(sum(n), h, d, generator=g, device="cuda"), _kv_like(g, sum(n), 2 * hk, d)],
                      1).bfloat16()
        s["q"], s["k"], s["v"] = x[:, :h], x[:, h:h + hk], x[:, h + hk:]
        s["cu"], s["max"] = _cu(n), max(n)
        s["seq"], s["idx"], _ = _rows(n, [0] * len(n))
        return s
    ps = case["page"]
    if op == "shared":
        first, shared = _groups(case)
        group = [sum(b >= f for f in first[1:-1]) for b in range(len(n))]
        ctx = [r + shared[x] for r, x in zip(ctx, group)]
        # (a prefix that ends inside a page: that page is copied for every sequence, and shared up to its start)
        whole = [x // ps for x in shared]
        s.update(_pools(case, [-(-c // ps) for c in ctx], [(whole[x], first[x]) for x in group], g))
        s["groups"], s["shared"], s["group"] = _i32(first), _i32([w * ps for w in whole]), _i32(group)
        s["longest"], s["rest"] = max(whole) * ps, max(c - whole[x] * ps for c, x in zip(ctx, group))
        gn = [sum(n[a:b]) for a, b in zip(first, first[1:])]
        s["grow"], s["gidx"], _ = _rows(gn, [0] * len(gn))   # per packed row: its group, its index in the group
        s["most"] = max(gn)
    else:
        s.update(_pools(case, [-(-c // ps) for c in ctx], [(0, b) for b in range(len(n))], g))
    s["seq"], s["idx"], s["pos"] = _rows(n, [c - m for c, m in zip(ctx, n)])
    if op == "append":
        x = torch.cat([torch.randn(sum(n), h, d, generator=g, device="cuda"), _kv_like(g, sum(n), 2 * hk, d)],
                      1).to(DT[case["in"]])
        s["q"], s["new_k"], s["new_v"] = x[:, :h], x[:, h:h + hk], x[:, h + hk:]
        _plan(d, False, s)
        return s
    s["q"] = torch.randn(sum(n), h, d, generator=g, device="cuda").bfloat16()
    s["cu"], s["lens"], s["max"] = _cu(n), _i32(ctx), max(n)
    return s


# ------------------------------------------------------------- plain forms
def _reserve(s):
    ps, table, free = s["ps"], s["table"], s["free"]
    lens, ask, left = s["lens"].long(), s["counts"].long().clamp_min(0), s["n_free"].long()
    cap = table.shape[1] * ps
    fits = (lens >= 0) & (lens + ask <= cap)
    ask = torch.where(fits, ask, 0)
    had = (lens + ps - 1) // ps
    need = torch.where(fits, (lens + ask + ps - 1) // ps - had, 0)
    served = fits & ((need == 0) | (need.cumsum(0) <= left)) & (ask.cumsum(0) <= s["tokens"])
    short = (need.sum() - left).clamp_min(0).int()
    ask, need = ask * served, need * served
    cu = torch.cat([ask.new_zeros(1), ask.cumsum(0)])
    i = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(cu[1:], i, right=True).clamp_max(len(ask) - 1)
    real = i < cu[-1]
    pos = torch.where(real, lens[seq] + i - cu[seq], -1)
    j = torch.arange(table.shape[1], device="cuda")
    mine = (j >= had[:, None]) & (j < (had + need)[:, None])
    rank = (need.cumsum(0) - need - had)[:, None] + j
    top = free[(left - 1 - rank).clamp(0, len(free) - 1)]
    table.copy_(torch.where(mine, top, table))
    s["n_free"].copy_(left - need.sum())
    return cu.int(), (lens + ask).int(), torch.where(real, seq, -1).int(), pos.int(), short.view(1)


def _release(s, lens):
    ps, table, free = s["ps"], s["table"], s["free"]
    lens, left = lens.long(), s["n_free"].long()
    keep = torch.minimum(s["keep"].long().clamp_min(0), lens)
    beg, end = (keep + ps - 1) // ps, (lens + ps - 1) // ps
    j = torch.arange(table.shape[1], device="cuda")
    drop = (j >= beg[:, None]) & (j < end[:, None])
    rank = ((end - beg).cumsum(0) - (end - beg) - beg)[:, None] + j
    more = torch.cat([free, free.new_zeros(1)])
    more[torch.where(drop, left + rank, len(free)).clamp_max(len(free))] = table
    free.copy_(more[:-1])
    table.masked_fill_(drop, -1)
    s["n_free"].copy_(left + (end - beg).sum())


def _normed(x, gain):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain


def _rotate(x, pos, s):
    """x [rows, heads, dim] in 32 bits, rotated."""
    a = pos.double().unsqueeze(1) * s["freq"]
    a = a - 2 * math.pi * torch.round(a / (2 * math.pi))
    c, n = torch.cos(a).float().unsqueeze(1), torch.sin(a).float().unsqueeze(1)
    y = torch.empty_like(x)
    h = x.shape[-1] // 2
    lo, hi = (slice(0, None, 2), slice(1, None, 2)) if s["inter"] else (slice(0, h), slice(h, None))
    u, v = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = u * c - v * n, v * c + u * n
    return y


def _keys(s, name, row, pos):
    """Cache rows in 32 bits at positions pos [b, keys] of the table's rows row [b]: [b, heads, keys, dim]."""
    ps = s["k"].shape[2]
    page = s["table"][row.long().unsqueeze(1), (pos // ps).clamp(0, s["table"].shape[1] - 1)].long()
    x = s[name][page, :, pos % ps].float()
    if name + "_scale" in s:
        x = torch.ldexp(x, s[name + "_scale"][page, :, pos % ps].int().unsqueeze(-1) - 127)
    return x.transpose(1, 2)


def _attend(q, k, v, see, scale):
    """q [b, m, hq, d] and k, v [b, hk, keys, d] in 32 bits, see [b, m, keys]: (out, lse)."""
    b, m, hq, d = q.shape
    hk = k.shape[1]
    q = q.view(b, m, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(scale).view(b, hk, hq // hk, m, -1)
    s.masked_fill_(~see.view(b, 1, 1, m, -1), -math.inf)
    top = s.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp_(s.sub_(top))
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hk, -1, p.shape[-1]), v).view(b, hk, hq // hk, m, d) / z.clamp_min(1e-30)
    lse = (top + torch.log(z)).squeeze(-1)
    return o.permute(0, 3, 1, 2, 4).reshape(b, m, hq, d), lse.permute(0, 3, 1, 2).reshape(b, m, hq)


def _padded(x, row, idx, b, m):
    y = x.new_zeros(b, m, *x.shape[1:], dtype=torch.float32)
    y[row.long(), idx.long()] = x.float()
    return y


def _windowed(s, case):
    """Keys of the first tokens and of the window of every sequence's rows, and no others."""
    m, w, first = s["max"], case["window"], case["sinks"]
    n, lens = (s["cu"][1:] - s["cu"][:-1]).long(), s["lens"].long()
    p = (lens - n)[:, None] + torch.arange(m, device="cuda")                # positions of the rows
    lo = (lens - n - w + 1).clamp_min(0)
    j = torch.cat([torch.arange(first, device="cuda").expand(len(n), first),
                   lo[:, None] + torch.arange(m + w - 1, device="cuda")], 1)
    once = torch.cat([torch.ones(first, dtype=torch.bool, device="cuda").expand(len(n), first),
                      (j[:, first:] >= first)], 1)                          # a first token inside the window
    live = (once & (j < lens[:, None]))[:, None]
    see = live & (j[:, None] <= p[..., None]) & ((j[:, None] > p[..., None] - w) | (j[:, None] < first))
    b = torch.arange(len(n), device="cuda")
    j = j.clamp_max(lens.amax() - 1)
    q = _padded(s["q"], s["seq"], s["idx"], len(n), m)
    return _attend(q, _keys(s, "k", b, j), _keys(s, "v", b, j), see, case["head_dim"] ** -0.5)


def _prompt(s, case):
    b, m, w = len(s["cu"]) - 1, s["max"], case["window"]
    q, k, v = (_padded(s[x], s["seq"], s["idx"], b, m) for x in ("q", "k", "v"))
    i = torch.arange(m, device="cuda")
    see = (i <= i[:, None]) & ((i > i[:, None] - w) | (i < case["sinks"]))
    return _attend(q, k.transpose(1, 2), v.transpose(1, 2), see.expand(b, m, m), case["head_dim"] ** -0.5)


def _shared(s, case):
    """The prefix of each group against all its rows, the rest of each sequence against its own."""
    b, m, scale = len(s["cu"]) - 1, s["max"], case["head_dim"] ** -0.5
    first, shared = s["groups"][:-1], s["shared"].long()
    j = torch.arange(s["longest"], device="cuda").expand(len(first), -1)
    see = (j < shared[:, None])[:, None].expand(-1, s["most"], -1)
    q = _padded(s["q"], s["grow"], s["gidx"], len(first), s["most"])
    o1, l1 = (x[s["grow"].long(), s["gidx"].long()]
              for x in _attend(q, _keys(s, "k", first, j), _keys(s, "v", first, j), see, scale))
    n, lens = (s["cu"][1:] - s["cu"][:-1]).long(), s["lens"].long()
    lo = shared[s["group"].long()]
    j = lo[:, None] + torch.arange(s["rest"], device="cuda")
    p = (lens - n)[:, None] + torch.arange(m, device="cuda")
    see = (j[:, None] <= p[..., None])
    rows = torch.arange(b, device="cuda")
    j = j.clamp_max(lens.amax() - 1)
    q = _padded(s["q"], s["seq"], s["idx"], b, m)
    o2, l2 = (x[s["seq"].long(), s["idx"].long()]
              for x in _attend(q, _keys(s, "k", rows, j), _keys(s, "v", rows, j), see, scale))
    lse = torch.logaddexp(l1, l2)
    w1, w2 = torch.exp(l1 - lse).unsqueeze(-1), torch.exp(l2 - lse).unsqueeze(-1)
    return (o1 * w1 + o2 * w2).bfloat16(), lse


def _run_own(s):
    import speculative_decoding_verification_step_gb300 as sv
    case = s["case"]
    op = case["op"]
    if op == "pages":
        step = sv.kv_reserve(s["cache"], s["lens"], s["counts"], s["free"], s["n_free"], s["tokens"])
        sv.kv_release(s["cache"], step[1], s["keep"], s["free"], s["n_free"])
        return (*step, s["table"], s["free"], s["n_free"])
    if op == "append":
        q = sv.qkv_append(s["cache"], s["q"], s["new_k"], s["new_v"], s["seq"], s["pos"], s["plan"], s["norm"][0],
                          s["norm"][1], eps=EPS)
        return (q, *_state(s))
    if op == "rows":
        return sv.rope_norm_rows(s["x"], s["pos"], s["plan"], s["gain"], eps=EPS, dtype=DT[case["out"]])
    if op == "window":
        return sv.attn_paged(s["q"], s["cache"], s["cu"], s["lens"], max_q=s["max"], window=case["window"],
                             sinks=case["sinks"])
    if op == "prompt":
        return sv.attn_prompt(s["q"], s["k"], s["v"], s["cu"], max_len=s["max"], window=case["window"],
                              sinks=case["sinks"])
    return sv.attn_shared(s["q"], s["cache"], s["cu"], s["lens"], s["shared"], groups=s["groups"], max_q=s["max"])


def _state(s):
    """The cache: its rows and, for 8 bits, the powers of two that scale them, as values."""
    if "k_scale" not in s:
        return s["k"], s["v"]
    return s["k"], s["v"], s["k_scale"].view(torch.float8_e8m0fnu), s["v_scale"].view(torch.float8_e8m0fnu)


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    op = case["op"]
    if op == "pages":
        step = _reserve(s)
        _release(s, step[1])
        return (*step, s["table"], s["free"], s["n_free"])
    if op == "rows":
        return _rotate(_normed(s["x"].float(), s["gain"]), s["pos"], s).to(DT[case["out"]])
    if op == "append":
        ps = case["page"]
        page = s["table"][s["seq"].long(), (s["pos"] // ps).long()].long()
        slot = (s["pos"] % ps).long()
        k = _rotate(_normed(s["new_k"].float(), s["norm"][1]), s["pos"], s)
        for name, x in (("k", k), ("v", s["new_v"].float())):
            if case["cache"] == "e4m3":
                codes, e = _encode(x)
                s[name].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
                s[name + "_scale"][page, :, slot] = e
            else:
                s[name][page, :, slot] = x.bfloat16()
        return (_rotate(_normed(s["q"].float(), s["norm"][0]), s["pos"], s).bfloat16(), *_state(s))
    if op == "shared":
        return _shared(s, case)
    o, lse = _windowed(s, case) if op == "window" else _prompt(s, case)
    at = s["seq"].long(), s["idx"].long()
    return o[at].bfloat16(), lse[at]


# ------------------------------------------------------------------- work
def _pairs(n, ctx, window, sinks):
    """(query, key) pairs that a sequence's n newest of ctx positions see, and the keys that any sees."""
    p = torch.arange(ctx - n, ctx)
    win = torch.minimum(p + 1, torch.tensor(window))
    lead = torch.clamp(p + 1 - win, max=sinks)
    lo = max(0, ctx - n - window + 1)
    return int((win + lead).sum()), ctx - lo + min(sinks, lo)


def work(case):
    op = case["op"]
    if op == "pages":
        n, lens = _lens(case)
        need = sum(-(-(c + m) // case["page"]) + -c // case["page"] for c, m in zip(lens, n))
        # lengths, counts and kept lengths in; cu, lengths and 8 bytes a token out; a page from the stack to the
        # table and back, and its entry cleared
        return {"bytes": 20 * len(n) + 8 * (sum(n) + 64) + 20 * need, "flops": 0}
    hq, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    if op == "rows":
        e = case["tokens"] * (hq + hk) * d
        return {"bytes": e * (ES[case["in"]] + ES[case["out"]]) + 4 * case["tokens"], "flops": 7 * e}
    n, ctx = _lens(case)
    t = sum(n)
    if op == "prompt":
        pairs = sum(_pairs(m, m, case["window"], case["sinks"])[0] for m in n)
        return {"bytes": t * d * 2 * (2 * hq + 2 * hk) + 4 * t * hq, "flops": 4 * pairs * hq * d}
    row = 2 * hk * (d * ES[case["cache"]] + (case["cache"] == "e4m3"))
    if op == "append":
        return {"bytes": t * ((hq + 2 * hk) * d * ES[case["in"]] + 2 * hq * d + row + 8),
                "flops": 7 * t * (hq + hk) * d}
    if op == "window":
        seen = [_pairs(m, c, case["window"], case["sinks"]) for m, c in zip(n, ctx)]
        pairs, keys = sum(x[0] for x in seen), sum(x[1] for x in seen)
    else:
        first, shared = _groups(case)
        group = [sum(b >= f for f in first[1:-1]) for b in range(len(n))]
        pairs = sum(m * (c + shared[g]) - m * (m - 1) // 2 for m, c, g in zip(n, ctx, group))
        keys = sum(ctx) + sum(shared)
    return {"bytes": keys * row + t * hq * (4 * d + 4) + 4 * (keys // case["page"]), "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ exact
def _turned(x, pos, s):
    """x in 64 bits as complex pairs, each turned by its angle."""
    a = torch.polar(torch.ones(1, dtype=torch.float64, device=x.device),
                    torch.outer(pos.double(), s["freq"]))[:, None, :]
    r = x.shape[-1]
    if s["inter"]:
        z = torch.view_as_complex(x.reshape(*x.shape[:-1], r // 2, 2).contiguous()) * a
        return torch.view_as_real(z).flatten(-2)
    z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:].contiguous()) * a
    return torch.cat([z.real, z.imag], -1)


def _unit(x, gain):
    x = x.double()
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * gain.double()


def _rounded8(x):
    """The nearest 4-bit-exponent, 3-bit-mantissa values (ties to even) of the rows after scaling each by
    a power of two, and those powers."""
    top = x.abs().amax(-1, keepdim=True)
    r = torch.where(top > 0, top, torch.full_like(top, 448.0)) / 448.0
    e = torch.round(torch.log2(r))                     # the smallest e with r <= 2^e, whichever way log2 rounds
    e = torch.where(r > torch.pow(2.0, e), e + 1, torch.where(r <= torch.pow(2.0, e - 1), e - 1, e)).clamp(-60, 60)
    y = x * torch.pow(2.0, -e)
    step = torch.pow(2.0, torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step, torch.pow(2.0, e).squeeze(-1)


def _values(s, name, page):
    x = s[name][page].double()
    if name + "_scale" in s:
        x = x * torch.pow(2.0, s[name + "_scale"][page].double() - 127).unsqueeze(-1)
    return x


def exact(case, seed):
    op = case["op"]
    if op == "pages":
        return None
    s = prepare(case, seed)
    if op == "rows":
        return _turned(_unit(s["x"], s["gain"]), s["pos"], s)
    ps = case.get("page", 1)
    if op == "append":
        at = s["table"].long().flatten()[s["seq"].long() * s["table"].shape[1] + s["pos"].long() // ps]
        slot = s["pos"].long() % ps
        new = {"k": _turned(_unit(s["new_k"], s["norm"][1]), s["pos"], s), "v": s["new_v"].double()}
        values, powers = [], []
        for name in ("k", "v"):
            x = s[name].double()
            if case["cache"] == "e4m3":
                e = torch.pow(2.0, s[name + "_scale"].double() - 127)
                x[at, :, slot], e[at, :, slot] = _rounded8(new[name])
                powers.append(e)
            else:
                x[at, :, slot] = new[name]
            values.append(x)
        return (_turned(_unit(s["q"], s["norm"][0]), s["pos"], s), *values, *powers)
    n, ctx = _lens(case)
    if op == "shared":
        ctx = [int(x) for x in s["lens"].tolist()]
    hq, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    q = s["q"].double()
    out = torch.zeros_like(q)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    window, sinks = case.get("window", 1 << 30), case.get("sinks", 0)
    r0 = 0
    for b in range(len(n)):
        if op == "prompt":
            k, v = (s[x][r0:r0 + n[b]].double().transpose(0, 1) for x in ("k", "v"))
        else:
            page = s["table"][b, :-(-ctx[b] // ps)].long()
            k, v = (_values(s, x, page).transpose(0, 1).reshape(hk, -1, d)[:, :ctx[b]] for x in ("k", "v"))
        p, j = torch.arange(ctx[b] - n[b], ctx[b], device="cuda")[:, None], torch.arange(ctx[b], device="cuda")
        see = (j <= p) & ((p - j < window) | (j < sinks))
        some = see.any(0)                                  # (what no row sees is left out)
        k, v, see = k[:, some], v[:, some], see[:, some]
        for h in range(hq):
            t = q[r0:r0 + n[b], h] @ k[h * hk // hq].T / math.sqrt(d)
            t = torch.where(see, t, -math.inf)
            lse[r0:r0 + n[b], h] = torch.logsumexp(t, -1)
            out[r0:r0 + n[b], h] = torch.softmax(t, -1) @ v[h * hk // hq]
        r0 += n[b]
    return out, lse
