"""Cases of the paged-cache operators: rotary positions, the cache's write and
read-back, attention of a chunk of new tokens over the paged cache, and causal
attention over packed prompts.

Shapes are those of the framework's own configurations: 32 query / 8 KV heads
of 128 or 64 and the small 8 / 2 heads, verify chunks of K + 1 tokens, contexts
of 512, 4096 and 16384, batches of 1 to 64.  With ``own`` False every operator
is computed in plain torch operations in 32 bits (angles in 64) and rounded
once; with ``own`` True by the package's calls.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ES = {"f32": 4, "bf16": 2, "e4m3": 1}
# rotary recipes: the 500000 base of the 1B / 8B shapes, plain or stretched 8x
# by wavelength for a context longer than the original 8192
THETA = 500000.0
STRETCH = {"factor": 8.0, "orig_ctx": 8192.0, "low": 1.0, "high": 4.0}


def listed():
    return [
        # queries and keys of one verify step of one sequence (K = 5), from the fp32 q/k/v projection
        {"name": "rope-verify-1x6", "op": "rope", "tokens": 6, "heads": 40, "head_dim": 128, "rot_dim": 128,
         "interleaved": False, "scaling": "plain", "first": 511, "in": "f32", "out": "bf16"},
        # a prompt far into a stretched context: interleaved pairs, half of every head rotated
        {"name": "rope-prompt-16381", "op": "rope", "tokens": 16381, "heads": 40, "head_dim": 64, "rot_dim": 32,
         "interleaved": True, "scaling": "parts", "first": 120000, "in": "bf16", "out": "bf16"},
        # the new rows of one verify step into a 16-bit cache: the smallest write
        {"name": "append-verify-1x6-bf16", "op": "append", "batch": 1, "q": 6, "ctx": 512, "kv_heads": 8,
         "head_dim": 128, "page": 16, "in": "f32", "cache": "bf16"},
        # four prompts' rows into an 8-bit cache
        {"name": "append-prompt-4x4000-e4m3", "op": "append", "batch": 4, "q": 4000, "ctx": 4096, "kv_heads": 8,
         "head_dim": 128, "page": 64, "in": "bf16", "cache": "e4m3"},
        # one short context read back in full precision
        {"name": "gather-1x500-bf16", "op": "gather", "batch": 1, "ctx": 500, "kv_heads": 8, "head_dim": 128,
         "page": 16, "cache": "bf16", "out": "f32"},
        # a batch of long 8-bit contexts read back, as before a change of layout or of cache type
        {"name": "gather-16x16384-e4m3", "op": "gather", "batch": 16, "ctx": 16384, "kv_heads": 8, "head_dim": 128,
         "page": 16, "cache": "e4m3", "out": "bf16"},
        # the verify step of one sequence (K = 5) at the end of a 512-token prompt
        {"name": "paged-verify-1x6-512", "op": "paged", "batch": 1, "q": 6, "ctx": 512, "heads": 32, "kv_heads": 8,
         "head_dim": 128, "page": 16, "cache": "bf16", "ragged": False},
        # plain decoding of 16 long contexts with the 1B-shaped heads
        {"name": "paged-decode-16x1-16384", "op": "paged", "batch": 16, "q": 1, "ctx": 16384, "heads": 32,
         "kv_heads": 8, "head_dim": 64, "page": 32, "cache": "bf16", "ragged": False},
        # the verify step of 64 sequences over an 8-bit cache
        {"name": "paged-verify-64x6-4096-e4m3", "op": "paged", "batch": 64, "q": 6, "ctx": 4096, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 16, "cache": "e4m3", "ragged": False},
        # chunks of new prompt tokens of different lengths over long contexts
        {"name": "paged-chunk-4x512-16384", "op": "paged", "batch": 4, "q": 512, "ctx": 16384, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 64, "cache": "bf16", "ragged": True},
        # three short prompts of the small heads, packed
        {"name": "prompt-3x130", "op": "prompt", "batch": 3, "len": 130, "heads": 8, "kv_heads": 2, "head_dim": 64},
        # six long prompts of different lengths, packed
        {"name": "prompt-6x4096", "op": "prompt", "batch": 6, "len": 4096, "heads": 32, "kv_heads": 8,
         "head_dim": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "gather", "paged", "paged", "paged", "prompt", "prompt"])
    hd = rng.choice([64, 128])
    hq, hkv = rng.choice([(8, 2), (32, 8), (32, 8), (12, 4), (16, 2), (7, 1)])
    page = rng.choice([16, 32, 64])
    cache = rng.choice(["bf16", "e4m3"])
    if op == "rope":
        return {"op": op, "tokens": _log(rng, 1, 16384), "heads": hq + hkv, "head_dim": hd,
                "rot_dim": rng.choice([hd, hd // 2, hd // 4]), "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(["plain", "parts"]), "first": _log(rng, 1, 500000),
                "in": rng.choice(["f32", "bf16"]), "out": rng.choice(["f32", "bf16"])}
    if op == "append":
        b = _log(rng, 1, 64)
        q = _log(rng, 1, max(2, 16000 // b))
        return {"op": op, "batch": b, "q": q, "ctx": q + _log(rng, 1, 4096), "kv_heads": hkv, "head_dim": hd,
                "page": page, "in": rng.choice(["f32", "bf16"]), "cache": cache}
    if op == "gather":
        b = _log(rng, 1, 16)
        return {"op": op, "batch": b, "ctx": _log(rng, 16, 100000 // b), "kv_heads": hkv, "head_dim": hd,
                "page": page, "cache": cache, "out": rng.choice(["f32", "bf16"])}
    if op == "paged":
        b = _log(rng, 1, 64)
        q = rng.choice([1, 2, 4, 6, 9, _log(rng, 10, 512)])
        q = min(q, max(1, 1024 // b))
        ctx = max(q, _log(rng, 64, min(16384, 262144 // b)))
        return {"op": op, "batch": b, "q": q, "ctx": ctx, "heads": hq, "kv_heads": hkv, "head_dim": hd,
                "page": page, "cache": cache, "ragged": rng.random() < 0.5}
    b = _log(rng, 1, 16)
    return {"op": op, "batch": b, "len": _log(rng, 8, min(4096, 16384 // b)), "heads": hq, "kv_heads": hkv,
            "head_dim": hd}


def _lens(case):
    """(new tokens, context lengths) of a case's sequences, from the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    b = case["batch"]
    if case["op"] == "prompt":
        n = [rng.randint(max(1, case["len"] // 4), case["len"]) for _ in range(b)]
        n[rng.randrange(b)] = case["len"]
        return n, n
    if case["op"] == "gather":
        n = [rng.randint(max(1, case["ctx"] // 2), case["ctx"]) for _ in range(b)]
        n[rng.randrange(b)] = case["ctx"]
        return n, n
    q = [case["q"]] * b
    if case.get("ragged"):
        q = [_log(rng, 1, case["q"]) for _ in range(b)]
        q[rng.randrange(b)] = case["q"]
    ctx = [max(n, rng.randint((case["ctx"] + 1) // 2, case["ctx"])) for n in q]
    ctx[rng.randrange(b)] = case["ctx"]
    return q, ctx


# ------------------------------------------------------------------ inputs
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rows(n, first):
    """Per packed row: its sequence, its index in the sequence's rows and its position."""
    seq = torch.repeat_interleave(torch.arange(len(n)), torch.tensor(n))
    idx = torch.cat([torch.arange(x) for x in n])
    pos = idx + torch.tensor(first)[seq]
    return seq.int().cuda(), idx.int().cuda(), pos.int().cuda()


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


def _pools(case, ctx, g):
    """The pools of a cache in use: shuffled pages, some not owned by any of the sequences."""
    ps, h, d = case["page"], case["kv_heads"], case["head_dim"]
    per = [-(-c // ps) for c in ctx]
    pages = sum(per) + max(1, sum(per) // 8)
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.zeros(len(ctx), max(per), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
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


def _plan(rot_dim, interleaved, scaling, s):
    """The rotation a program keeps: its frequencies (turns of the pairs per position)."""
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    f = THETA ** (-i / rot_dim)
    if scaling == "parts":
        turns = STRETCH["orig_ctx"] * f / (2 * math.pi)
        keep = ((turns - STRETCH["low"]) / (STRETCH["high"] - STRETCH["low"])).clamp(0, 1)
        f = f * (keep + (1 - keep) / STRETCH["factor"])
    s["freq"], s["rot"], s["inter"] = f.cuda(), rot_dim, interleaved
    if own:
        import speculative_decoding_verification_step_gb300 as sv
        more = STRETCH if scaling == "parts" else {}
        s["plan"] = sv.rope_plan(rot_dim, THETA, interleaved=interleaved, scaling=scaling, **more)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    op = case["op"]
    if op == "rope":
        h = case["heads"]
        x = torch.randn(case["tokens"], h + h // 4, case["head_dim"], generator=g, device="cuda")
        s["x"] = x.to(DT[case["in"]])[:, :h]           # the q and k heads of a fused projection
        s["pos"] = (case["first"] + torch.arange(case["tokens"])).int().cuda()
        _plan(case["rot_dim"], case["interleaved"], case["scaling"], s)
        return s
    n, ctx = _lens(case)
    if op == "prompt":
        h, hk = case["heads"], case["kv_heads"]
        x = torch.cat([torch.randn(sum(n), h, case["head_dim"], generator=g, device="cuda"),
                       _kv_like(g, sum(n), 2 * hk, case["head_dim"])], 1).bfloat16()
        s["q"], s["k"], s["v"] = x[:, :h], x[:, h:h + hk], x[:, h + hk:]
        s["cu"] = _i32([sum(n[:i]) for i in range(len(n) + 1)])
        s["max"] = max(n)
        s["seq"], s["idx"], _ = _rows(n, [0] * len(n))
        return s
    s.update(_pools(case, ctx, g))
    first = [c - m for c, m in zip(ctx, n)]
    s["seq"], s["idx"], s["pos"] = _rows(n, first)
    if op == "append":
        hk = case["kv_heads"]
        x = _kv_like(g, sum(n), 2 * hk, case["head_dim"]).to(DT[case["in"]])
        s["new_k"], s["new_v"] = x[:, :hk], x[:, hk:]
        _plan(case["head_dim"], False, "plain", s)
    if op == "paged":
        s["q"] = torch.randn(sum(n), case["heads"], case["head_dim"], generator=g, device="cuda").bfloat16()
        s["cu"] = _i32([sum(n[:i]) for i in range(len(n) + 1)])
        s["lens"] = _i32(ctx)
        s["max"] = max(n)
    return s


# ------------------------------------------------------------- plain forms
def _rotate(x, pos, s):
    """x [rows, heads, dim] in 32 bits, rotated."""
    a = pos.double().unsqueeze(1) * s["freq"]
    a = a - 2 * math.pi * torch.round(a / (2 * math.pi))
    c, n = torch.cos(a).float().unsqueeze(1), torch.sin(a).float().unsqueeze(1)
    r, y = s["rot"], x.clone()
    if s["inter"]:
        u, v = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = u * c - v * n, v * c + u * n
    else:
        u, v = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = u * c - v * n, v * c + u * n
    return y


def _decode(s, name, page, slot=None):
    x = s[name][page] if slot is None else s[name][page, :, slot]
    x = x.float()
    if name + "_scale" in s:
        e = s[name + "_scale"]
        e = (e[page] if slot is None else e[page, :, slot]).int() - 127
        x = torch.ldexp(x, e.unsqueeze(-1))
    return x


def _slots(s):
    ps = s["k"].shape[2]
    return s["table"][s["seq"].long(), (s["pos"] // ps).long()].long(), (s["pos"] % ps).long()


def _attend(q, k, v, n, seen, scale):
    """q [b, m, hq, d] and k, v [b, hk, keys, d] in 32 bits; row i of sequence b sees keys
    0 .. seen[b] - n[b] + i."""
    b, m, hq, d = q.shape
    hk = k.shape[1]
    q = q.view(b, m, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(scale).view(b, hk, hq // hk, m, -1)
    last = (seen - n).view(b, 1) + torch.arange(m, device=q.device)
    hide = torch.arange(k.shape[2], device=q.device) > last.unsqueeze(2)
    s.masked_fill_(hide.view(b, 1, 1, m, -1), -math.inf)
    top = s.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp_(s.sub_(top))
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hk, -1, p.shape[-1]), v).view(b, hk, hq // hk, m, d) / z.clamp_min(1e-30)
    lse = (top + torch.log(z)).squeeze(-1)
    return o.permute(0, 3, 1, 2, 4).reshape(b, m, hq, d), lse.permute(0, 3, 1, 2).reshape(b, m, hq)


def _padded(x, s, m):
    y = x.new_zeros(s["cu"].numel() - 1, m, *x.shape[1:], dtype=torch.float32)
    y[s["seq"].long(), s["idx"].long()] = x.float()
    return y


def _run_own(s):
    import speculative_decoding_verification_step_gb300 as sv
    op = s["case"]["op"]
    if op == "rope":
        return sv.rope_rows(s["x"], s["pos"], s["plan"], dtype=DT[s["case"]["out"]])
    if op == "append":
        sv.kv_append(s["cache"], s["new_k"], s["new_v"], s["seq"], s["pos"], s["plan"])
        return _state(s)
    if op == "gather":
        return sv.kv_gather(s["cache"], s["seq"], s["pos"], dtype=DT[s["case"]["out"]])
    if op == "paged":
        return sv.attn_paged(s["q"], s["cache"], s["cu"], s["lens"], max_q=s["max"])
    return sv.attn_prompt(s["q"], s["k"], s["v"], s["cu"], max_len=s["max"])


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
    if op == "rope":
        return _rotate(s["x"].float(), s["pos"], s).to(DT[case["out"]])
    if op == "append":
        page, slot = _slots(s)
        for name, x in (("k", _rotate(s["new_k"].float(), s["pos"], s)), ("v", s["new_v"].float())):
            if case["cache"] == "e4m3":
                codes, e = _encode(x)
                s[name].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
                s[name + "_scale"][page, :, slot] = e
            else:
                s[name][page, :, slot] = x.bfloat16()
        return _state(s)
    if op == "gather":
        page, slot = _slots(s)
        return tuple(_decode(s, name, page, slot).to(DT[case["out"]]) for name in ("k", "v"))
    d = case["head_dim"]
    if op == "paged":
        k, v = (_decode(s, name, s["table"].long()).transpose(1, 2).reshape(
            case["batch"], case["kv_heads"], -1, d) for name in ("k", "v"))
        seen = s["lens"]
    else:
        k, v = (_padded(s[name], s, s["max"]).transpose(1, 2) for name in ("k", "v"))
        seen = s["cu"][1:] - s["cu"][:-1]
    o, lse = _attend(_padded(s["q"], s, s["max"]), k, v, s["cu"][1:] - s["cu"][:-1], seen, d ** -0.5)
    at = s["seq"].long(), s["idx"].long()
    return o[at].bfloat16(), lse[at]


# ------------------------------------------------------------------- work
def work(case):
    op, d = case["op"], case["head_dim"]
    if op == "rope":
        e = case["tokens"] * case["heads"] * d
        return {"bytes": e * (ES[case["in"]] + ES[case["out"]]) + 4 * case["tokens"],
                "flops": 3 * case["tokens"] * case["heads"] * case["rot_dim"]}
    n, ctx = _lens(case)
    hk = case["kv_heads"]
    if op == "prompt":
        t, hq = sum(n), case["heads"]
        pairs = sum(m * (m + 1) // 2 for m in n)
        return {"bytes": t * d * 2 * (2 * hq + 2 * hk) + 4 * t * hq, "flops": 4 * pairs * hq * d}
    row = 2 * hk * (d * ES[case["cache"]] + (case["cache"] == "e4m3"))
    if op == "append":
        return {"bytes": sum(n) * (2 * hk * d * ES[case["in"]] + row + 8), "flops": 3 * sum(n) * hk * d}
    if op == "gather":
        return {"bytes": sum(n) * (row + 2 * hk * d * ES[case["out"]] + 8), "flops": 0}
    hq = case["heads"]
    pairs = sum(m * c - m * (m - 1) // 2 for m, c in zip(n, ctx))
    pages = sum(-(-c // case["page"]) for c in ctx)
    return {"bytes": sum(ctx) * row + sum(n) * hq * (4 * d + 4) + 4 * pages, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ exact
def _turned(x, pos, s):
    """x in 64 bits as complex pairs, each turned by its angle."""
    a = torch.polar(torch.ones(1, dtype=torch.float64, device=x.device),
                    torch.outer(pos.double(), s["freq"]))[:, None, :]
    r = s["rot"]
    head, rest = x[..., :r], x[..., r:]
    if s["inter"]:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], r // 2, 2).contiguous()) * a
        head = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(head[..., :r // 2].contiguous(), head[..., r // 2:].contiguous()) * a
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, rest], -1)


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


def _values(s, name):
    x = s[name].double()
    if name + "_scale" in s:
        x = x * torch.pow(2.0, s[name + "_scale"].double() - 127).unsqueeze(-1)
    return x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _turned(s["x"].double(), s["pos"], s)
    ps = case.get("page", 1)
    if op in ("append", "gather"):
        at = s["table"].long().flatten()[s["seq"].long() * s["table"].shape[1] + s["pos"].long() // ps]
        slot = s["pos"].long() % ps
    if op == "append":
        new = {"k": _turned(s["new_k"].double(), s["pos"], s), "v": s["new_v"].double()}
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
        return tuple(values + powers)
    if op == "gather":
        return tuple(_values(s, name)[at, :, slot] for name in ("k", "v"))
    n, ctx = _lens(case)
    hq, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    q = s["q"].double()
    out = torch.zeros_like(q)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    r0 = 0
    for b in range(len(n)):
        if op == "paged":
            page = s["table"][b, :-(-ctx[b] // ps)].long()
            part = {"table": s["table"], **{x: s[x][page] for x in ("k", "v", "k_scale", "v_scale") if x in s}}
            k, v = (_values(part, x).transpose(0, 1).reshape(hk, -1, d)[:, :ctx[b]] for x in ("k", "v"))
        else:
            k, v = (s[x][r0:r0 + n[b]].double().transpose(0, 1) for x in ("k", "v"))
        see = torch.ones(n[b], ctx[b], dtype=torch.bool, device="cuda").tril(ctx[b] - n[b])
        for h in range(hq):
            t = q[r0:r0 + n[b], h] @ k[h * hk // hq].T / math.sqrt(d)
            t = torch.where(see, t, -math.inf)
            lse[r0:r0 + n[b], h] = torch.logsumexp(t, -1)
            out[r0:r0 + n[b], h] = torch.softmax(t, -1) @ v[h * hk // hq]
        r0 += n[b]
    return out, lse
