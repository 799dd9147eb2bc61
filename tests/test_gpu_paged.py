"""Paged-cache operators against plain 64-bit forms: rotary positions, the
cache's write and read-back, chunk attention over the pages, packed prompts.

Tolerances count roundings.  A rounding is off by at most half a step of its
type (bf16 2^-8, fp32 2^-24, e4m3 2^-4 relative, and half of e4m3's smallest
step for its subnormals):
* rotation: the angle, a 32-bit fraction of a turn turned into fp32 (2^-24 of
  at most pi), sincospif (2 units, 2^-22), two products and one sum: under
  8 * 2^-23 of |a| + |b|, then the output's rounding;
* attention: a score is a sum of head_dim products, off by at most
  d = (head_dim + 8) 2^-24 scale sum|q k|; a weight by 2 d and, once for the
  product with v, by a bf16 rounding; so |out - ref| <= (2^-8 + 4 d + keys
  2^-23 + 2^-20) sum w|v| + 2^-8 |ref|, and lse is within 2 d + keys 2^-23 +
  2^-20 + |lse| 2^-22 (a fp32 sum of `keys` terms, exp2's 2^-22).
"""
import math

import pytest
import torch

import speculative_decoding_verification_step_gb300 as sv

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv.build()
    sv.lib()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ rotary
def _freqs(rot, theta, scaling="plain", factor=1.0, orig=0.0, low=1.0, high=4.0):
    f = []
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    for i in range(rot // 2):
        w = theta ** (-2.0 * i / rot)
        if scaling == "linear":
            w /= factor
        if scaling == "parts":
            keep = min(1.0, max(0.0, (orig * w / (2 * math.pi) - low) / (high - low)))
            w *= keep + (1 - keep) / factor
        f.append(w)
    return f


def _rope_ref(x, pos, freqs, inter, sign=1.0, mscale=1.0):
    """64-bit rotation by the complex product; also the pair sizes |a| + |b|."""
    x = x.to(F64)
    r = 2 * len(freqs)
    # angles in turns with integer positions: the fractional part is exact enough in 64 bits
    turns = torch.outer(pos.to(F64), torch.tensor(freqs, dtype=F64, device="cuda") / (2 * math.pi))
    ang = (turns - turns.round()) * (2 * math.pi) * sign
    z = torch.polar(torch.full_like(ang, mscale), ang)[:, None]
    y, size = x.clone(), x.abs()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if inter else (x[..., :r // 2], x[..., r // 2:r])
    w = torch.complex(a, b) * z
    s = a.abs() + b.abs()
    if inter:
        y[..., 0:r:2], y[..., 1:r:2] = w.real, w.imag
        size[..., 0:r:2], size[..., 1:r:2] = s, s
    else:
        y[..., :r // 2], y[..., r // 2:r] = w.real, w.imag
        size[..., :r // 2], size[..., r // 2:r] = s, s
    return y, size


ROPE = [  # tokens, heads, hd, rot, interleaved, in, out, plan options, first position
    (6, 40, 128, 128, False, torch.float32, torch.bfloat16, {}, 511),
    (1, 1, 64, 64, False, torch.bfloat16, torch.bfloat16, {}, 0),
    (33, 10, 64, 32, True, torch.bfloat16, torch.float32, {"scaling": "parts", "factor": 8.0, "orig_ctx": 8192.0}, 900000),
    (700, 40, 64, 16, False, torch.bfloat16, torch.bfloat16, {"scaling": "linear", "factor": 4.0}, 70000),
    (17, 3, 128, 128, True, torch.float32, torch.float32, {"scaling": "ntk", "factor": 4.0, "mscale": 1.25}, 3),
    (5, 7, 32, 6, False, torch.float32, torch.bfloat16, {}, 2 ** 31 - 10),      # odd split: one element at a time
    (5, 7, 34, 34, True, torch.bfloat16, torch.bfloat16, {}, 100),
    (4, 2, 256, 256, False, torch.float32, torch.float32, {"scaling": "parts", "factor": 32.0, "orig_ctx": 4096.0, "high": 32.0}, 1 << 20),
]


@pytest.mark.parametrize("t,h,hd,rot,inter,tin,tout,opt,first", ROPE)
def test_rope_rows(t, h, hd, rot, inter, tin, tout, opt, first):
    g = _gen(t + h)
    wide = _randn(g, t, h + 2, hd).to(tin)
    x = wide[:, 1:h + 1]                       # a slice of a projection
    pos = (first + torch.arange(t, device="cuda")).int()
    plan = sv.rope_plan(rot, 500000.0, interleaved=inter, **opt)
    y = sv.rope_rows(x, pos, plan, dtype=tout)
    o = dict(opt)
    ms = o.pop("mscale", 1.0)
    f = _freqs(rot, 500000.0, o.get("scaling", "plain"), o.get("factor", 1.0), o.get("orig_ctx", 0.0),
               o.get("low", 1.0), o.get("high", 4.0))
    ref, size = _rope_ref(x, pos, f, inter, mscale=ms)
    # the reference's own angles: positions times 64-bit frequencies, 2^-52 relative
    tol = size * ms * (8 * 2.0 ** -23 + (first + t) * 2.0 ** -50) + ref.abs() * HALF[tout]
    err = (y.to(F64) - ref).abs()
    assert (err <= tol).all(), float((err - tol).max())
    if rot < hd and tin == tout:
        assert torch.equal(y[..., rot:], x[..., rot:])
    # the gradient: <rotated x, u> = <x, rotated-back u>, and a difference quotient of the same
    u = _randn(g, t, h, hd)
    back = sv.rope_rows(u, pos, plan, inverse=True)
    bref, bsize = _rope_ref(u, pos, f, inter, sign=-1.0, mscale=ms)
    assert ((back.to(F64) - bref).abs() <= bsize * ms * (8 * 2.0 ** -23 + (first + t) * 2.0 ** -50)
            + bref.abs() * 2.0 ** -24).all()
    lhs = (ref * u.to(F64)).sum()
    rhs = (x.to(F64) * bref).sum()
    assert abs(lhs - rhs) <= 1e-10 * float((size * u.to(F64).abs()).sum())


def test_rope_rows_in_place_and_negative():
    g = _gen(3)
    x = _randn(g, 9, 4, 64).bfloat16()
    pos = _i32([-5, 0, 7, 7, 2 ** 31 - 1, -2 ** 31, 1, 2, 3])
    plan = sv.rope_plan(64, 10000.0)
    y = sv.rope_rows(x, pos, plan)
    ref, size = _rope_ref(x, pos, _freqs(64, 10000.0), False)
    far = pos.to(F64).abs()[:, None, None] * 2.0 ** -50
    assert ((y.to(F64) - ref).abs() <= size * (8 * 2.0 ** -23 + far) + ref.abs() * 2.0 ** -8).all()
    z = x.clone()
    assert sv.rope_rows(z, pos, plan, out=z) is z
    assert torch.equal(z, y)
    assert sv.rope_rows(x[:0], pos[:0], plan).shape == (0, 4, 64)


# ------------------------------------------------------------------- cache
def _times2(x, e):
    """x * 2^e, exact (a device pow or ldexp of 2 is not, in its last place)."""
    powers = torch.tensor([2.0 ** i for i in range(-140, 141)], dtype=F64, device=x.device)
    return x * powers[e.long() + 140]


def _round_e4m3(y):
    """Nearest e4m3 value (ties to even) of 64-bit values within +-448."""
    _, e = torch.frexp(y.abs().clamp_min(2.0 ** -6))      # y = m 2^e, 1/2 <= m < 1: steps of 2^(e - 4)
    return _times2(torch.round(_times2(y, 4 - e)), e - 4)


def _exponent(x):
    """Smallest e in -60..60 with max|x| <= 448 2^e (0 for zero rows)."""
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(top > 0, (e - 9 + (m > 0.875).int()), torch.zeros_like(e))
    return e.clamp(-60, 60)


def _cache(g, seqs, ctx, heads, ps, hd, dtype, extra=3):
    need = -(-ctx // ps)
    pages = seqs * need + extra
    table = torch.randperm(pages, generator=g, device="cuda")[:seqs * need].int().view(seqs, need).contiguous()
    return sv.KVCache.empty(pages, ps, heads, hd, table, dtype)


def _values(cache):
    out = []
    for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        v = x.to(F64)
        if s is not None:
            v = _times2(v, (s.int() - 127).clamp(-140, 140).unsqueeze(-1))
            v[s == 255] = math.nan
        out.append(v)
    return out


def _read(cache, values, seq, pos):
    page = cache.table.long()[seq.long(), (pos // cache.page_size).long()]
    return [v[page, :, (pos % cache.page_size).long()] for v in values]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("tin", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hd,heads,ps,n", [(32, 2, 16, 5), (64, 8, 32, 1), (128, 8, 16, 70), (128, 1, 256, 300),
                                           (64, 3, 64, 2500)])
def test_append_and_gather(dtype, tin, hd, heads, ps, n):
    g = _gen(hd + n)
    seqs, ctx = 3, max(n, 40)
    cache = _cache(g, seqs, ctx, heads, ps, hd, dtype)
    x = (_randn(g, n, 2 * heads + 1, hd) * torch.exp(2 * _randn(g, n, 1, 1))).to(tin)
    k, v = x[:, :heads], x[:, heads:2 * heads]
    seq = torch.randint(0, seqs, (n,), generator=g, device="cuda").int()
    pos = torch.randperm(ctx, generator=g, device="cuda")[:n].int()
    before = [t.clone() for t in _values(cache)]
    sv.kv_append(cache, k, v, seq, pos)
    got = _read(cache, _values(cache), seq, pos)
    for y, src in zip(got, (k, v)):
        s = src.to(F64)
        if dtype == "bf16":
            assert torch.equal(y, src.bfloat16().to(F64))
        else:
            e = _exponent(s).unsqueeze(-1)
            bad = int((y != _times2(_round_e4m3(_times2(s, -e)), e)).sum())
            assert bad == 0, bad
    # every other slot is as it was
    mask = torch.ones(before[0].shape[0], ps, dtype=torch.bool, device="cuda")
    mask[cache.table.long()[seq.long(), (pos // ps).long()], (pos % ps).long()] = False
    for y, z in zip(_values(cache), before):
        assert torch.equal(y.transpose(1, 2)[mask], z.transpose(1, 2)[mask])
    for out in (torch.bfloat16, torch.float32):
        for y, z in zip(sv.kv_gather(cache, seq, pos, dtype=out), got):
            assert y.dtype == out and torch.equal(y.to(F64), z)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("inter,rot,hd", [(False, 128, 128), (True, 64, 64), (False, 16, 32), (True, 8, 64),
                                          (False, 20, 64), (True, 30, 128)])
def test_append_rotates(dtype, inter, rot, hd):
    g = _gen(rot)
    n, heads = 37, 2
    cache = _cache(g, 2, 64, heads, 16, hd, dtype)
    k, v = _randn(g, n, heads, hd), _randn(g, n, heads, hd)
    seq = (torch.arange(n, device="cuda") % 2).int()
    pos = (torch.arange(n, device="cuda") // 2 + 20).int()
    sv.kv_append(cache, k, v, seq, pos, sv.rope_plan(rot, 500000.0, interleaved=inter))
    ref, size = _rope_ref(k, pos, _freqs(rot, 500000.0), inter)
    got, gv = _read(cache, _values(cache), seq, pos)
    rope = size * 8 * 2.0 ** -23
    if dtype == "bf16":
        assert ((got - ref).abs() <= ref.abs() * 2.0 ** -8 + 2 * rope).all()
        assert torch.equal(gv, v.bfloat16().to(F64))
    else:
        e = _exponent(ref)   # a row at a power's border may take the next one: twice the smallest step
        assert ((got - ref).abs() <= ref.abs() * 2.0 ** -4 + torch.pow(2.0, e.to(F64) - 9).unsqueeze(-1) + 2 * rope).all()


def test_append_skips_and_special_rows():
    g = _gen(8)
    cache = _cache(g, 2, 32, 1, 16, 32, "e4m3")
    cache.table[1, 1] = cache.k.shape[0]          # not a page of the pool
    cache.table[0, 1] = -7
    n = 8
    k = _randn(g, n, 1, 32)
    k[0] = 0
    k[1, 0, 3] = math.inf
    k[2, 0, 31] = math.nan
    k[3] *= 2.0 ** 100
    k[4] *= 2.0 ** -90
    k[5, 0, 0] = 448.0
    k[5, 0, 1:] /= 10
    v = _randn(g, n, 1, 32)
    before = [t.clone().view(torch.uint8) for t in (cache.k, cache.v)]
    skip_seq = _i32([-1, 2, 0, 0, 0, 1, 0, 1])
    skip_pos = _i32([0, 0, -1, 32, 16, 16, 31, 31])
    sv.kv_append(cache, k, v, skip_seq, skip_pos)
    assert all(torch.equal(t.view(torch.uint8), b) for t, b in zip((cache.k, cache.v), before))
    kk, vv = sv.kv_gather(cache, skip_seq, skip_pos)
    assert not kk.any() and not vv.any()
    seq, pos = _i32([0] * n), _i32(list(range(n)))
    sv.kv_append(cache, k, v, seq, pos)
    y, _ = sv.kv_gather(cache, seq, pos, dtype=torch.float32)
    assert not y[0].any()
    assert torch.isnan(y[1:4]).all()              # an infinity, a NaN, past 448 * 2^60
    assert not y[4].any()                         # under 2^-70
    assert y[5, 0, 0] == 448.0
    assert torch.isfinite(y[5:]).all()


def test_gather_one_side_of_nan_and_strided_pool():
    """k and v interleaved in one buffer [pages][2]...: a page stride twice a page."""
    g = _gen(9)
    both = _randn(g, 6, 2, 2, 16, 64).bfloat16()
    table = _i32([[5, 0], [2, 2]])                # a shared page
    cache = sv.KVCache(both[:, 0], both[:, 1], table)
    seq, pos = _i32([0, 0, 1, 1]), _i32([3, 20, 3, 19])
    k, v = sv.kv_gather(cache, seq, pos)
    for i, (p, s) in enumerate([(5, 3), (0, 4), (2, 3), (2, 3)]):
        assert torch.equal(k[i], both[p, 0, :, s]) and torch.equal(v[i], both[p, 1, :, s])


# --------------------------------------------------------------- attention
def _attend_ref(q, ks, vs, n, scale):
    """Rows q [n, hq, d] over keys ks, vs [keys, hk, d] in 64 bits: out, lse and
    the bounds' sums (sum w|v|, largest scale sum|q k|)."""
    keys, hk, _ = ks.shape
    hq = q.shape[1]
    rep = hq // hk
    q, ks, vs = q.to(F64), ks.to(F64).repeat_interleave(rep, 1), vs.to(F64).repeat_interleave(rep, 1)
    if keys == 0:
        z = torch.zeros_like(q)
        return z, torch.full(q.shape[:2], -math.inf, dtype=F64, device="cuda"), z, torch.zeros(1, 1, 1, device="cuda")
    s = torch.einsum("nhd,khd->hnk", q, ks) * scale
    size = torch.einsum("nhd,khd->hnk", q.abs(), ks.abs()) * scale
    see = torch.arange(keys, device="cuda")[None] <= (keys - n + torch.arange(n, device="cuda"))[:, None]
    s = s.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(s, -1)
    w = torch.where(see, torch.exp(s - lse.clamp_min(-1e300).unsqueeze(-1)), torch.zeros_like(s))
    dot = size.masked_fill(~see, 0).amax(-1)
    return (torch.einsum("hnk,khd->nhd", w, vs), lse.T, torch.einsum("hnk,khd->nhd", w, vs.abs()), dot.T.unsqueeze(-1))


def _check_rows(out, lse, ref, keys, d):
    o, l, wv, dot = ref
    assert torch.isfinite(out).all()
    delta = (d + 8) * 2.0 ** -24 * dot
    tol = (2.0 ** -8 + 4 * delta + keys * 2.0 ** -23 + 2.0 ** -20) * wv + 2.0 ** -8 * o.abs() + 1e-30
    err = (out.to(F64) - o).abs()
    assert (err <= tol).all(), float((err / tol).max())
    none = torch.isinf(l)
    assert torch.equal(none, torch.isinf(lse)) and (lse[none] < 0).all()
    lt = 2 * delta.expand(*l.shape, 1)[..., 0] + keys * 2.0 ** -23 + 2.0 ** -20 + l.abs() * 2.0 ** -22
    assert ((lse.to(F64) - l).abs()[~none] <= lt[~none]).all()


def _paged_case(seed, hq, hk, hd, ps, dtype, ns, lens, pad=0, poison=True, sharp=1.0):
    """A cache whose slots past the lengths hold NaN, its queries and its rows' values."""
    g = _gen(seed)
    seqs = len(ns)
    cache = _cache(g, seqs, max(max(lens), 1), hk, ps, hd, dtype)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x7f) if dtype == "e4m3" else t.fill_(math.nan if poison else 0.0)
    if dtype == "e4m3":
        cache.k_scale.fill_(255)
        cache.v_scale.fill_(255)
    rows = [(b, p) for b, c in enumerate(lens) for p in range(c)]
    if rows:
        seq, pos = _i32([r[0] for r in rows]), _i32([r[1] for r in rows])
        sv.kv_append(cache, _randn(g, len(rows), hk, hd) * sharp, _randn(g, len(rows), hk, hd), seq, pos)
    cu = [0]
    for n in ns:
        cu.append(cu[-1] + n)
    q = _randn(g, cu[-1] + pad, hq + 1, hd).bfloat16()[:, :hq]
    return cache, q, _i32(cu), _i32(lens)


def _paged_check(cache, q, cu, lens, ns, ctx, max_q=None, **kw):
    hd = q.shape[2]
    out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    got = sv.attn_paged(q, cache, cu, lens, max_q=max_q, out=out, lse=lse, **kw)
    assert got[0] is out and got[1] is lse
    values = _values(cache)
    r = 0
    for b, (n, c) in enumerate(zip(ns, ctx)):
        pos = torch.arange(c, device="cuda").int()
        k, v = _read(cache, values, torch.full_like(pos, b), pos)
        _check_rows(out[r:r + n], lse[r:r + n], _attend_ref(q[r:r + n], k, v, n, kw.get("scale") or hd ** -0.5), c, hd)
        r += n
    assert (out[r:] == 7.0).all() and (lse[r:] == 9.0).all()
    return out


PAGED = [  # hq, hk, hd, page, new tokens, contexts
    (32, 8, 128, 16, [6], [512]),
    (32, 8, 128, 16, [6, 6, 6], [513, 47, 1000]),
    (32, 8, 64, 32, [1] * 5, [1, 2, 16, 17, 3000]),
    (8, 2, 32, 16, [5, 1, 9], [5, 333, 64]),
    (4, 4, 64, 64, [1, 17, 16], [129, 17, 700]),
    (7, 1, 128, 32, [3, 5], [300, 5]),                # seven heads on one, odd row tiles
    (12, 4, 128, 256, [2, 0, 4], [40, 10, 600]),      # a sequence without new tokens
    (8, 2, 64, 16, [4, 3, 2], [2, 0, 1]),             # chunks longer than their contexts: empty rows
    (16, 2, 128, 16, [8], [8]),
    (2, 2, 64, 16, [1], [20000]),
    (32, 8, 128, 16, [40, 3], [200, 300]),
    (8, 2, 64, 64, [130, 257, 1], [500, 257, 100]),
    (32, 8, 128, 32, [129], [1500]),
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,hd,ps,ns,ctx", PAGED)
def test_attn_paged(hq, hk, hd, ps, ns, ctx, dtype):
    c, q, cu, lens = _paged_case(sum(ctx) + hd, hq, hk, hd, ps, dtype, ns, ctx, pad=2)
    _paged_check(c, q, cu, lens, ns, ctx)
    _paged_check(c, q, cu, lens, ns, ctx, max_q=max(ns))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [2, 70])
def test_attn_paged_sharp_scores(dtype, n):
    """Scores of +-hundreds: the exponents' reference moves all along the keys."""
    c, q, cu, lens = _paged_case(5, 8, 2, 64, 16, dtype, [n], [900], sharp=30.0)
    _paged_check(c, q, cu, lens, [n], [900])
    _paged_check(c, q, cu, lens, [n], [900], scale=0.01)


@pytest.mark.parametrize("n", [1, 6, 100])
@pytest.mark.parametrize("hd", [64, 128])
def test_attn_paged_subnormal_codes(hd, n):
    """Rows whose largest value no query sees: all that counts are e4m3's subnormal codes."""
    g = _gen(n)
    hq, hk, ctx = 8, 2, 200
    cache = _cache(g, 1, ctx, hk, 16, hd, "e4m3")
    k, v = (torch.randint(-7, 8, (ctx, hk, hd), generator=g, device="cuda").float() * 2.0 ** -9 for _ in range(2))
    k[..., 0] = v[..., 0] = 448.0
    pos = torch.arange(ctx, device="cuda").int()
    sv.kv_append(cache, k, v, torch.zeros_like(pos), pos)
    q = (_randn(g, n, hq, hd) * 64).bfloat16()
    q[..., 0] = 0
    kk, vv = sv.kv_gather(cache, torch.zeros_like(pos), pos, dtype=torch.float32)
    assert torch.equal(kk, k) and torch.equal(vv, v)
    out, lse = sv.attn_paged(q, cache, _i32([0, n]), _i32([ctx]))
    _check_rows(out, lse, _attend_ref(q, k, v, n, hd ** -0.5), ctx, hd)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd,n,g", [(64, 3, 2), (128, 6, 4), (128, 64, 4), (64, 200, 2)])
def test_attn_paged_batch_and_bad_indices(dtype, hd, n, g):
    """Many sequences of different lengths; table entries outside the pool read as
    zero rows, lengths past the table are cut, a broken cu row computes nothing."""
    seqs = 21 if n < 10 else 3
    ctx = [max(n, (37 * b * b) % 700) for b in range(seqs)]
    ns = [n] * seqs
    c, q, cu, lens = _paged_case(hd + n, 2 * g, 2, hd, 16, dtype, ns, ctx)
    _paged_check(c, q, cu, lens, ns, ctx, max_q=n)
    b = max(range(seqs), key=lambda i: ctx[i])
    for bad in (-3, c.k.shape[0], 2 ** 30):
        table = c.table.clone()
        t2 = table.clone()
        t2[b, 1] = bad
        c.table.copy_(t2)
        out, lse = sv.attn_paged(q, c, cu, lens, max_q=n)
        c.table.copy_(table)
        pos = torch.arange(ctx[b], device="cuda").int()
        k, v = _read(c, _values(c), torch.full_like(pos, b), pos)
        k[16:32], v[16:32] = 0, 0
        rows = slice(b * n, b * n + n)
        _check_rows(out[rows], lse[rows], _attend_ref(q[rows], k, v, n, hd ** -0.5), ctx[b], hd)
    cap = c.max_pages * 16
    cut = lens.clone()
    cut[b] = 2 ** 31 - 1
    if ctx[b] == cap:
        out, _ = sv.attn_paged(q, c, cu, lens)
        out2, _ = sv.attn_paged(q, c, cu, cut)
        assert torch.equal(out, out2)
    neg = lens.clone()
    neg[:] = -5
    out, lse = sv.attn_paged(q, c, cu, neg)
    assert not out.any() and torch.isinf(lse).all()
    broken = cu.clone()
    broken[1] = 10 ** 9
    keep = torch.full_like(q, 3.0, memory_format=torch.contiguous_format)
    out, _ = sv.attn_paged(q, c, broken, lens, out=keep)
    assert (out[:2 * n] == 3.0).all()


def test_attn_paged_max_q_leaves_rows():
    c, q, cu, lens = _paged_case(4, 8, 2, 64, 16, "bf16", [5, 2], [50, 60])
    full, _ = sv.attn_paged(q, c, cu, lens)
    out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
    sv.attn_paged(q, c, cu, lens, max_q=3, out=out, lse=False)
    assert torch.equal(out[:3], full[:3]) and (out[3:5] == 7.0).all() and torch.equal(out[5:], full[5:])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [3, 100])
def test_attn_paged_repeats_streams_and_graphs(dtype, n):
    """The same bits again, on another stream, and replayed from two graphs at once."""
    c, q, cu, lens = _paged_case(11, 32, 8, 128, 16, dtype, [n, n], [2000, 900 + n])
    out, lse = sv.attn_paged(q, c, cu, lens, max_q=n)
    for _ in range(3):
        a, b = sv.attn_paged(q, c, cu, lens, max_q=n)
        assert torch.equal(a, out) and torch.equal(b, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    for _ in range(2):
        o = torch.zeros_like(out)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            sv.attn_paged(q, c, cu, lens, max_q=n, out=o, lse=False)
            side.synchronize()
            o.zero_()
            with torch.cuda.graph(gr, stream=side):
                sv.attn_paged(q, c, cu, lens, max_q=n, out=o, lse=False)
        graphs.append(gr)
        outs.append(o)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graphs[0].replay()
    with torch.cuda.stream(other):
        graphs[1].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)
    # a replayed graph reads the lengths of the day
    lens.copy_(_i32([1000, 500 + n]))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], sv.attn_paged(q, c, cu, lens, max_q=n)[0])


LONG = [  # few rows per KV head over contexts that fill the GPU: hq, hk, hd, page, new tokens, contexts
    (32, 8, 128, 16, [6], [20000]),
    (32, 8, 128, 16, [6] * 5, [3001, 129, 9000, 0, 128]),
    (32, 8, 128, 64, [1, 1, 1], [4096, 7000, 3]),
    (16, 2, 64, 16, [5, 4, 5], [16384, 20001, 1]),    # 40 rows: two tiles of 20
    (32, 8, 64, 256, [1, 4], [6000, 5000]),
    (7, 1, 128, 32, [3, 5], [40000, 5]),              # seven heads on one
    (32, 8, 128, 32, [16, 0, 3], [5000, 10, 7000]),   # 64 rows, a sequence without new tokens
    (4, 4, 128, 16, [4] * 40, [3, 2, 0, 1000] + [130 * b for b in range(36)]),
    (64, 1, 128, 16, [1], [50000]),
    (32, 8, 128, 16, [9] * 16 + [1], [700, 9, 3, 1000] + [100 * b for b in range(13)]),   # 36 rows, items for all SMs
    (32, 8, 64, 64, [13, 16, 2] * 6, [90 * b for b in range(18)]),
    (32, 8, 128, 16, [3] * 40, [5000, 1, 0, 2] + [97 * b for b in range(36)]),            # more sequences than lanes
    (32, 8, 128, 128, [0, 6, 5, 0], [100, 4097, 8000, 0]),
    (8, 1, 64, 16, [1, 3], [17000, 250]),
    (32, 8, 128, 16, [6, 5] * 20, [5000, 1, 0, 5] + [97 * b for b in range(36)]),
    (8, 8, 128, 64, [9, 1, 16], [6000, 3, 9001]),                                         # 16 columns, one head each
    (32, 8, 128, 16, [6], [8192]),
    (32, 8, 128, 16, [2, 5] * 8, [1500, 0, 193, 64] + [70 * b + 1 for b in range(12)]),  # three blocks a tile
    (32, 8, 64, 32, [6] * 16, [130 * b for b in range(16)]),
    (16, 16, 32, 16, [1] * 9, [300 * b + 7 for b in range(9)]),
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,hd,ps,ns,ctx", LONG)
def test_attn_paged_long(hq, hk, hd, ps, ns, ctx, dtype):
    c, q, cu, lens = _paged_case(sum(ctx) + hd, hq, hk, hd, ps, dtype, ns, ctx, pad=2)
    out = _paged_check(c, q, cu, lens, ns, ctx, max_q=max(ns))
    assert torch.equal(out, _paged_check(c, q, cu, lens, ns, ctx, max_q=max(ns)))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd", [64, 128])
def test_attn_paged_long_sharp_scores(hd, dtype):
    c, q, cu, lens = _paged_case(6, 16, 4, hd, 16, dtype, [3, 5], [12000, 900], sharp=30.0)
    _paged_check(c, q, cu, lens, [3, 5], [12000, 900], max_q=5)
    _paged_check(c, q, cu, lens, [3, 5], [12000, 900], max_q=5, scale=0.01)
    c, q, cu, lens = _paged_case(7, 32, 2, hd, 16, dtype, [2, 1], [17000, 129], sharp=30.0)
    _paged_check(c, q, cu, lens, [2, 1], [17000, 129])


@pytest.mark.parametrize("hd", [64, 128])
def test_attn_paged_long_wide_queries(hd):
    """Queries of many sizes beside one large element."""
    hq, hk, ctx = 8, 2, 30000
    c, q, cu, lens = _paged_case(8, hq, hk, hd, 16, "e4m3", [4], [ctx])
    g = _gen(3)
    q = (q.float() * 2.0 ** -torch.randint(0, 10, q.shape, generator=g, device="cuda")).bfloat16()
    q[..., 0] = 448.0
    q = torch.where(q.abs() < 448 * 2.0 ** -13, 0, q)
    _paged_check(c, q, cu, lens, [4], [ctx])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_paged_long_special_values(dtype):
    """A NaN query row is NaN alone; a NaN key reaches the rows that see it; pages
    outside the pool read as zero rows."""
    hq, hk, hd, ctx = 8, 2, 128, 25000
    c, q, cu, lens = _paged_case(9, hq, hk, hd, 16, dtype, [4], [ctx])
    clean, _ = sv.attn_paged(q, c, cu, lens)
    q2 = q.clone()
    q2[1, 5, 7] = math.nan
    out, _ = sv.attn_paged(q2, c, cu, lens)
    assert torch.isnan(out[1, 5]).all()
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1, 5] = False
    assert torch.equal(out[keep], clean[keep])
    table = c.table.clone()
    t2 = table.clone()
    t2[0, 700] = 2 ** 30
    t2[0, 3] = -1
    c.table.copy_(t2)
    out, lse = sv.attn_paged(q, c, cu, lens)
    c.table.copy_(table)
    pos = torch.arange(ctx, device="cuda").int()
    k, v = _read(c, _values(c), torch.zeros_like(pos), pos)
    for p in (3, 700):
        k[16 * p:16 * p + 16], v[16 * p:16 * p + 16] = 0, 0
    _check_rows(out, lse, _attend_ref(q, k, v, 4, hd ** -0.5), ctx, hd)
    bad = torch.full((1, hk, hd), math.nan, device="cuda")
    sv.kv_append(c, bad, bad, _i32([0]), _i32([ctx - 2]))   # tokens 2 and 3 see it
    out, _ = sv.attn_paged(q, c, cu, lens)
    assert torch.isnan(out[2:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd", [64, 128])
def test_attn_paged_long_bound_and_strides(hd, dtype):
    """Rows past max_q stay; outputs between other columns, tables and pools with strides of their own, shared pages."""
    hq, hk, ps, ctx, n = 16, 4, 32, 20000, 8
    c, q, cu, lens = _paged_case(31, hq, hk, hd, ps, dtype, [n, n], [ctx, 40])
    table = torch.full((2, c.max_pages + 5), -7, dtype=torch.int32, device="cuda")
    table[:, :c.max_pages] = c.table[0]                   # both read the first sequence's pages
    two = sv.KVCache(c.k, c.v, table[:, :c.max_pages], c.k_scale, c.v_scale)
    wide = torch.full((2 * n, hq, hd + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2 * n, hq), 9.0, device="cuda")
    lens = _i32([ctx, ctx - 3])
    sv.attn_paged(q, two, cu, lens, max_q=6, out=wide[..., :hd], lse=lse)
    assert (wide[..., hd:] == 5.0).all()
    values = _values(c)
    for b, m in enumerate([ctx, ctx - 3]):
        pos = torch.arange(m, device="cuda").int()
        k, v = _read(c, values, torch.zeros_like(pos), pos)
        ref = _attend_ref(q[b * n:b * n + n], k, v, n, hd ** -0.5)
        ref = tuple(x[:6] for x in ref)
        r = slice(b * n, b * n + 6)
        _check_rows(wide[r, :, :hd], lse[r], ref, m, hd)
        assert (wide[b * n + 6:b * n + n] == 5.0).all() and (lse[b * n + 6:b * n + n] == 9.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_pool_past_32_bit_offsets(dtype):
    """Pages whose first element lies past 2^32: write, read-back and the attention kernels."""
    hk, hd, ps, ctx = 8, 128, 16, 10000
    pages = (1 << 32) // (hk * ps * hd) + ctx // ps + 8
    c = None
    table = (pages - 1 - torch.randperm(ctx // ps, generator=_gen(5), device="cuda")).int().view(1, -1).contiguous()
    kw = dict(device="cuda")
    if dtype == "e4m3":
        k, v = (torch.empty(pages, hk, ps, hd, dtype=torch.uint8, **kw).view(torch.float8_e4m3fn) for _ in range(2))
        c = sv.KVCache(k, v, table, *(torch.empty(pages, hk, ps, dtype=torch.uint8, **kw) for _ in range(2)))
    else:
        c = sv.KVCache(*(torch.empty(pages, hk, ps, hd, dtype=torch.bfloat16, **kw) for _ in range(2)), table)
    g = _gen(6)
    pos = torch.arange(ctx, device="cuda").int()
    k, v = _randn(g, ctx, hk, hd).bfloat16(), _randn(g, ctx, hk, hd).bfloat16()
    sv.kv_append(c, k, v, torch.zeros_like(pos), pos)
    kk, vv = sv.kv_gather(c, torch.zeros_like(pos), pos, dtype=torch.float32)
    if dtype == "bf16":
        assert torch.equal(kk, k.float()) and torch.equal(vv, v.float())
    for n in (1, 6, 100):
        q = _randn(g, n, 32, hd).bfloat16()
        out, lse = sv.attn_paged(q, c, _i32([0, n]), _i32([ctx]), max_q=n)
        _check_rows(out, lse, _attend_ref(q, kk, vv, n, hd ** -0.5), ctx, hd)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_paged_workspace(dtype):
    """With and without a workspace, and with one too small: right either way, nothing past its end."""
    ns, ctx, (hq, hk, hd) = [4, 3], [9000, 30000], (16, 4, 128)
    c, q, cu, lens = _paged_case(14, hq, hk, hd, 32, dtype, ns, ctx)
    L, n = sv.lib(), sum(ns)
    need = L.spec_attn_paged_workspace(c._ref, n, 4, hq)
    assert (need > 0) == (dtype == "e4m3")
    ws = torch.full((need + 256,), 0x5a, dtype=torch.uint8, device="cuda")
    for size in (0, max(need - 16, 0), need):
        out, lse = torch.zeros(n, hq, hd, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, hq, device="cuda")
        assert L.spec_attn_paged(c._ref, q.data_ptr(), q.stride(0), q.stride(1), cu.data_ptr(), lens.data_ptr(), n, 4, hq, 0.0,
                                 out.data_ptr(), hq * hd, hd, lse.data_ptr(), ws.data_ptr() if size else None, size,
                                 torch.cuda.current_stream().cuda_stream) == 0
        values, r = _values(c), 0
        for b, (k, m) in enumerate(zip(ns, ctx)):
            pos = torch.arange(m, device="cuda").int()
            kk, vv = _read(c, values, torch.full_like(pos, b), pos)
            _check_rows(out[r:r + k], lse[r:r + k], _attend_ref(q[r:r + k], kk, vv, k, hd ** -0.5), m, hd)
            r += k
        if size < need:
            assert (ws == 0x5a).all()
    assert (ws[need:] == 0x5a).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2, _ = sv.attn_paged(q, c, cu, lens, max_q=4, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out2, out)


@pytest.mark.parametrize("dtype,n", [("bf16", 4), ("e4m3", 4), ("e4m3", 6), ("e4m3", 8)])
def test_attn_paged_long_overlaps_and_graphs(dtype, n):
    """Calls on two streams at once and replayed graphs give the bits of one call alone."""
    ns, ctx = [n] * 3, [9000, 4000, 17000]
    c, q, cu, lens = _paged_case(12, 32, 8, 128, 16, dtype, ns, ctx)
    q2 = q.flip(0).contiguous()
    ref, ref2 = (sv.attn_paged(x, c, cu, lens, max_q=n)[0] for x in (q, q2))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got, got2 = [], []
    for _ in range(4):
        with torch.cuda.stream(a):
            got.append(sv.attn_paged(q, c, cu, lens, max_q=n)[0])
        with torch.cuda.stream(b):
            got2.append(sv.attn_paged(q2, c, cu, lens, max_q=n)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, ref) for x in got) and all(torch.equal(x, ref2) for x in got2)
    gr, o = torch.cuda.CUDAGraph(), torch.zeros_like(ref)
    with torch.cuda.graph(gr):
        sv.attn_paged(q, c, cu, lens, max_q=n, out=o)
    for new in (ctx, [1, 17000, 4], [0, 0, 0], [17000, 17000, 17000]):
        lens.copy_(_i32(new))
        gr.replay()
        torch.cuda.synchronize()
        # (as bits: the longer lengths reach slots that hold NaN)
        assert torch.equal(o.view(torch.int16), sv.attn_paged(q, c, cu, lens, max_q=n)[0].view(torch.int16))


PROMPT = [  # hq, hk, hd, lengths
    (8, 2, 64, [130, 1, 77]),
    (32, 8, 128, [17]),
    (8, 2, 32, [100, 33]),
    (7, 1, 128, [64, 0, 65, 200]),
    (12, 4, 64, [600, 129, 3]),
    (4, 4, 128, [1025]),
    (32, 8, 128, [900, 1500]),
    (16, 2, 64, [2000]),
]


@pytest.mark.parametrize("hq,hk,hd,ns", PROMPT)
def test_attn_prompt(hq, hk, hd, ns):
    g = _gen(sum(ns))
    total = sum(ns)
    x = _randn(g, total + 3, hq + 2 * hk, hd).bfloat16()
    x[total:] = math.nan                          # rows behind the last sequence
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    cu = [0]
    for n in ns:
        cu.append(cu[-1] + n)
    for bound in (None, max(ns)):
        out = torch.full((total + 3, hq, hd), 7.0, device="cuda", dtype=torch.bfloat16)
        lse = torch.full((total + 3, hq), 9.0, device="cuda")
        sv.attn_prompt(q, k, v, _i32(cu), max_len=bound, out=out, lse=lse)
        for b, n in enumerate(ns):
            r = slice(cu[b], cu[b + 1])
            if n:
                _check_rows(out[r], lse[r], _attend_ref(q[r], k[r], v[r], n, hd ** -0.5), n, hd)
        assert (out[total:] == 7.0).all() and (lse[total:] == 9.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd", [64, 128])
def test_attn_paged_chunks_repeat(hd, dtype):
    """Chunks over contexts of many lengths, few enough for two blocks an item: the
    same bits every time, beside other work, and right."""
    ns, ctx = [256, 130, 64, 1], [5000, 3333, 6001, 700]
    c, q, cu, lens = _paged_case(21, 16, 4, hd, 64, dtype, ns, ctx)
    ref = _paged_check(c, q, cu, lens, ns, ctx, max_q=256)
    side, noise = torch.cuda.Stream(), torch.zeros(1 << 26, device="cuda")
    torch.cuda.synchronize()
    got = []
    for i in range(60):
        with torch.cuda.stream(side):
            noise.add_(1.0)
        got.append(sv.attn_paged(q, c, cu, lens, max_q=256)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, ref) for x in got)


def test_prompt_neighbours_do_not_leak():
    """A sequence that holds NaN leaves its neighbours alone."""
    g = _gen(2)
    for ns in ([40, 50, 30], [300, 333, 290]):
        x = _randn(g, sum(ns), 4, 64).bfloat16()
        cu = _i32([0, ns[0], ns[0] + ns[1], sum(ns)])
        q, k, v = x[:, :2], x[:, 2:3], x[:, 3:]
        ref, _ = sv.attn_prompt(q, k, v, cu)
        x[ns[0]:ns[0] + ns[1]] = math.nan
        out, _ = sv.attn_prompt(q, k, v, cu)
        assert torch.equal(out[:ns[0]], ref[:ns[0]]) and torch.equal(out[ns[0] + ns[1]:], ref[ns[0] + ns[1]:])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd,ps", [(128, 16), (64, 64)])
def test_decode_loop(dtype, hd, ps):
    """The operators as a program runs them together: prompts packed and written,
    then verify steps of 4 tokens and a plain one, all against one 64-bit run."""
    g = _gen(hd)
    hq, hk = 8, 2
    prompts = [37, 90]
    ctx = 160
    cache = _cache(g, 2, ctx, hk, ps, hd, dtype)
    plan = sv.rope_plan(hd, 500000.0)
    freqs = _freqs(hd, 500000.0)
    lens = [0, 0]
    for chunk in (prompts, [4, 4], [1, 1], [4, 0], [64, 3]):
        n = sum(chunk)
        qkv = _randn(g, n, hq + 2 * hk, hd).bfloat16()
        seq = _i32([b for b in range(2) for _ in range(chunk[b])])
        pos = _i32([lens[b] + i for b in range(2) for i in range(chunk[b])])
        q = sv.rope_rows(qkv[:, :hq], pos, plan)
        sv.kv_append(cache, qkv[:, hq:hq + hk], qkv[:, hq + hk:], seq, pos, plan)
        qref, qsize = _rope_ref(qkv[:, :hq], pos, freqs, False)
        assert ((q.to(F64) - qref).abs() <= qsize * 2.0 ** -19 + qref.abs() * 2.0 ** -8).all()
        kref, ksize = _rope_ref(qkv[:, hq:hq + hk], pos, freqs, False)
        kk, vv = sv.kv_gather(cache, seq, pos, dtype=torch.float32)
        if dtype == "bf16":
            assert ((kk.to(F64) - kref).abs() <= ksize * 2.0 ** -19 + kref.abs() * 2.0 ** -8).all()
            assert torch.equal(vv, qkv[:, hq + hk:].float())
        else:
            assert ((kk.to(F64) - kref).abs() <= ksize * 2.0 ** -19 + kref.abs() * 2.0 ** -4 + kref.abs().amax(-1, keepdim=True) * 2.0 ** -16).all()
        lens = [a + b for a, b in zip(lens, chunk)]
        cu = _i32([0, chunk[0], n])
        _paged_check(cache, q, cu, _i32(lens), chunk, lens, max_q=max(chunk))
        if lens == prompts and dtype == "bf16":   # the prompt form of the same rows
            k16 = kk.bfloat16()
            out, lse = sv.attn_prompt(q, k16, vv.bfloat16(), cu)
            for r, c in ((slice(0, chunk[0]), chunk[0]), (slice(chunk[0], n), chunk[1])):
                _check_rows(out[r], lse[r], _attend_ref(q[r], k16[r], vv[r], c, hd ** -0.5), c, hd)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_cache_of_one_page_and_one_sequence(dtype):
    """Strides of dimensions of one entry mean nothing: expanded and sliced ones are as good as packed."""
    g = _gen(41)
    hq, hk, hd, n = 8, 2, 64, 11
    c, q, cu, lens = _paged_case(41, hq, hk, hd, 16, dtype, [n], [n])
    page = int(c.table[0, 0])
    one = lambda t: None if t is None else t[page:page + 1].expand(1, *t.shape[1:])
    odd = lambda t: None if t is None else one(t).as_strided(t[:1].shape, (3,) + t.stride()[1:], t.stride(0) * page)
    zero = _i32([0])
    for f in (one, odd):
        for table in (zero.expand(1, 1), zero.as_strided((1, 1), (7, 1))):
            alone = sv.KVCache(f(c.k), f(c.v), table, f(c.k_scale), f(c.v_scale))
            _paged_check(alone, q, cu, lens, [n], [n])
    # rows of a table that is wider than what it is used for
    both = torch.stack([c.table[0], c.table[0] * 0 - 1]).repeat_interleave(2, 0)
    for rows in (both[:1], both[::2][:1]):
        _paged_check(sv.KVCache(c.k, c.v, rows, c.k_scale, c.v_scale), q, cu, lens, [n], [n])


# --------------------------------------- 8-bit rows of very different sizes
def _filled(g, k, v, ps):
    """An e4m3 cache of one sequence's rows k, v [keys, heads, dim], and what it holds of them."""
    n, hk, hd = k.shape
    c = _cache(g, 1, n, hk, ps, hd, "e4m3")
    pos = torch.arange(n, device="cuda").int()
    sv.kv_append(c, k, v, torch.zeros_like(pos), pos)
    return c, *_read(c, _values(c), torch.zeros_like(pos), pos)


SPREADS = {  # exponents of the value rows, [keys]
    "early": lambda g, n, s: torch.where(torch.arange(n, device="cuda") < 20, s, 0),
    "late": lambda g, n, s: torch.where(torch.arange(n, device="cuda") > n - 20, s, 0),
    "down": lambda g, n, s: (s * (1 - torch.arange(n, device="cuda") / n)).int() - s // 2,
    "mixed": lambda g, n, s: torch.randint(-(s // 2), s // 2 + 1, (n,), generator=g, device="cuda"),
    "zeros": lambda g, n, s: torch.full((n,), -s, device="cuda"),
}


# (no more than keeps a row's exponent within the -60..60 of a write)
@pytest.mark.parametrize("kind,s", [(kind, s) for kind in SPREADS for s in (6, 12, 20, 30, 45, 60, 100)
                                    if s <= {"zeros": 50, "early": 60, "late": 60}.get(kind, 100)])
@pytest.mark.parametrize("hq,hk,hd,n", [(4, 4, 32, 1), (8, 2, 64, 4), (8, 2, 128, 1), (16, 4, 128, 6), (4, 1, 128, 8),
                                        (8, 1, 128, 20)])
def test_attn_paged_value_scales(hq, hk, hd, n, kind, s):
    """Value rows 2^s apart under scores so sharp that every query row rests on a few keys of its own:
    the small rows count for some queries as much as the large ones do for others."""
    g = _gen(s + hd + n)
    ctx = 333
    k, v = _randn(g, ctx, hk, hd) * 6.0, _randn(g, ctx, hk, hd)
    v = v * torch.pow(2.0, SPREADS[kind](g, ctx, s).float()).view(-1, 1, 1)
    if kind == "zeros":
        v[torch.rand(ctx, generator=g, device="cuda") < 0.3] = 0     # stored with exponent 0
    c, kk, vv = _filled(g, k, v, 16)
    q = _randn(g, n, hq, hd).bfloat16()
    out, lse = sv.attn_paged(q, c, _i32([0, n]), _i32([ctx]), max_q=n)
    ref = _attend_ref(q, kk, vv, n, hd ** -0.5)
    _check_rows(out, lse, ref, ctx, hd)


KERNELS = {  # one call for each way the attention is computed: new tokens, context, whether a workspace is wanted
    "few rows": (4, 300, False), "few rows of a long context": (4, 20000, True), "many rows": (100, 700, False),
}


@pytest.mark.parametrize("code", [0x7f, 0xff])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("kernel", list(KERNELS))
def test_nan_codes(kernel, hd, code):
    """A code that is no number (a cast of a caller's own puts it where a value overflows) reads as NaN
    everywhere: in K it takes the rows that see it, in V its column."""
    n, ctx, ws = KERNELS[kernel]
    hq, hk, ps = 8, 2, 16
    c, q, cu, lens = _paged_case(hd + n, hq, hk, hd, ps, "e4m3", [n], [ctx])
    assert (sv.lib().spec_attn_paged_workspace(c._ref, n, n, hq) > 0) == ws
    clean, clse = sv.attn_paged(q, c, cu, lens)
    at = lambda t, key, h, d: t.view(torch.uint8)[c.table[0, key // ps].long(), h, key % ps, d:d + 1]
    one = lambda key: (_i32([0]), _i32([key]))
    keep = at(c.v, 5, 1, 3).clone()
    at(c.v, 5, 1, 3).fill_(code)
    out, lse = sv.attn_paged(q, c, cu, lens)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[:, hq // 2:, 3] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad]) and torch.equal(lse, clse)
    for dt in (torch.bfloat16, torch.float32):
        k, v = sv.kv_gather(c, *one(5), dtype=dt)
        assert torch.isnan(v[0, 1, 3]) and int(torch.isnan(v).sum()) == 1 and not torch.isnan(k).any()
    at(c.v, 5, 1, 3).copy_(keep)
    for key, first in ((7, 0), (ctx - 1, n - 1), (ctx - 2, n - 2)):
        keep = at(c.k, key, 0, hd - 1).clone()
        at(c.k, key, 0, hd - 1).fill_(code)
        out, lse = sv.attn_paged(q, c, cu, lens)
        bad = torch.zeros_like(lse, dtype=torch.bool)
        bad[first:, :hq // 2] = True
        assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
        assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad], clse[~bad])
        at(c.k, key, 0, hd - 1).copy_(keep)
    # slots past the length may hold such codes and scales of any kind
    page, slot = c.table[0, ctx // ps if ctx % ps else 0].long(), slice(ctx % ps or ps, ps)
    for t, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        t.view(torch.uint8)[page, :, slot] = code
        s[page, :, slot] = 254
    out, lse = sv.attn_paged(q, c, cu, lens)
    assert torch.equal(out, clean) and torch.equal(lse, clse)


def test_gather_every_scale():
    """value = code * 2^(byte - 127) for every byte and code, rounded once."""
    hd = 64
    codes = torch.arange(256, device="cuda", dtype=torch.uint8).view(1, 4, 1, hd).expand(16, 4, 16, hd).contiguous()
    scale = torch.arange(256, device="cuda", dtype=torch.uint8).view(16, 1, 16).expand(16, 4, 16).contiguous()
    table = torch.arange(16, device="cuda").int().view(1, 16)
    f8 = codes.view(torch.float8_e4m3fn)
    c = sv.KVCache(f8, f8, table, scale, scale)
    pos = torch.arange(256, device="cuda").int()
    power = torch.tensor([2.0 ** (b - 127) for b in range(255)] + [math.nan], dtype=F64, device="cuda")
    want = power.view(256, 1, 1) * f8[0, :, 0].to(F64)
    for dt in (torch.float32, torch.bfloat16):
        ref = want.float().to(dt)                      # (exact in fp32 down to its smallest steps)
        for x in sv.kv_gather(c, torch.zeros_like(pos), pos, dtype=dt):
            assert torch.equal(torch.isnan(x), torch.isnan(ref)) and torch.equal(x[~x.isnan()], ref[~ref.isnan()])


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("kernel", list(KERNELS))
def test_attn_paged_every_scale(kernel, hd):
    """Powers of two that no write of the cache's own gives: the same scores and, but for the power, the
    same outputs as without."""
    n, ctx, ws = KERNELS[kernel]
    hq, hk, ps = 8, 2, 16
    c, q, cu, lens = _paged_case(hd + n, hq, hk, hd, ps, "e4m3", [n], [ctx])
    assert (sv.lib().spec_attn_paged_workspace(c._ref, n, n, hq) > 0) == ws
    g = _gen(hd)
    live = c.k_scale != 255
    for t in (c.k, c.v):           # codes of 1/64 to 1, which every power keeps within bf16
        t.copy_(torch.where(live.unsqueeze(-1), (torch.randint(1, 65, t.shape, generator=g, device="cuda") / 64.0)
                            * torch.randint(0, 2, t.shape, generator=g, device="cuda").mul(2).sub(1), math.nan))
    for kb, vb in ((127, 127), (0, 127), (1, 120), (37, 37), (60, 217), (217, 60), (127, 235), (217, 236), (127, 110)):
        c.k_scale.copy_(torch.where(live, kb, 255))
        c.v_scale.copy_(torch.where(live, vb, 255))
        scale = 2.0 ** (127 - kb) * hd ** -0.5
        out, lse = sv.attn_paged(q, c, cu, lens, scale=scale)
        pos = torch.arange(ctx, device="cuda").int()
        c.k_scale.copy_(torch.where(live, 127, 255))
        c.v_scale.copy_(torch.where(live, 127, 255))
        k, v = _read(c, _values(c), torch.zeros_like(pos), pos)
        out = out.to(F64) * 2.0 ** (127 - vb)
        _check_rows(out, lse, _attend_ref(q, k, v, n, hd ** -0.5), ctx, hd)


def _taken_blocks(call, shapes):
    """Pointers of blocks that the current stream has freed while its queued work still writes them, one
    of each shape, and the results of the call made meanwhile on a stream of its own."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty(s, dtype=dt, device="cuda") for s, dt in shapes]
    torch.cuda._sleep(20_000_000)
    for x in blocks:
        x.fill_(77)
    at = {x.data_ptr() for x in blocks}
    del blocks, x
    got = call(side.cuda_stream)
    torch.cuda.synchronize()
    return at, got


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_results_belong_to_the_given_stream(dtype):
    """With a raw stream given, results are not taken from memory that earlier work of the current
    stream still uses: that work would write over them."""
    n, ctx, hq, hk, hd = 4, 9000, 16, 4, 128
    c, q, cu, lens = _paged_case(52, hq, hk, hd, 32, dtype, [n], [ctx])
    plan = sv.rope_plan(hd, 10000.0)
    pos = torch.arange(n, device="cuda").int()
    seq = torch.zeros_like(pos)
    kv = q[:, :hk].contiguous()
    b16, f32 = torch.bfloat16, torch.float32
    calls = [
        (lambda s: sv.attn_paged(q, c, cu, lens, max_q=n, stream=s), [((n, hq, hd), b16), ((n, hq), f32)]),
        (lambda s: sv.attn_prompt(q, kv, kv, cu, stream=s), [((n, hq, hd), b16), ((n, hq), f32)]),
        (lambda s: sv.kv_gather(c, seq, pos, stream=s), [((n, hk, hd), b16)] * 2),
        (lambda s: (sv.rope_rows(q, pos, plan, stream=s),), [((n, hq, hd), b16)]),
    ]
    for call, shapes in calls:
        want = call(None)
        at, got = _taken_blocks(call, shapes)
        for x, y in zip(got, want):
            assert x.data_ptr() not in at and torch.equal(x, y)


def test_default_stream_by_its_handle():
    """Handle 0 is the default stream, and all that a call allocates is that stream's own memory."""
    n, ctx, hq, hk, hd = 4, 20000, 16, 4, 128
    c, q, cu, lens = _paged_case(53, hq, hk, hd, 32, "e4m3", [n], [ctx])
    assert sv.lib().spec_attn_paged_workspace(c._ref, n, n, hq) > 0
    want = sv.attn_paged(q, c, cu, lens, max_q=n)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = {s["address"] for s in torch.cuda.memory_snapshot()}
    got = sv.attn_paged(q, c, cu, lens, max_q=n, stream=0)
    with torch.cuda.stream(torch.cuda.Stream()):     # (whichever stream is current)
        got += sv.attn_paged(q, c, cu, lens, max_q=n, stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want + want))
    assert all(s["stream"] == 0 for s in torch.cuda.memory_snapshot() if s["address"] not in held)


# ------------------------------------------------------- waits that run out
def _give_up(call, q, steps):
    """The call with the hook armed at each of `steps`: every row is NaN or as without it, some are NaN,
    and the next call is right."""
    clean, clse = torch.full_like(q, 7.0, memory_format=torch.contiguous_format), torch.full(q.shape[:2], 9.0, device="cuda")
    call(clean, clse)
    for step in steps:
        out, lse = torch.full_like(clean, 5.0), torch.full_like(clse, 5.0)
        torch.cuda.synchronize()
        sv.inject_attention_timeout(step)
        try:
            call(out, lse)
        finally:
            sv.clear_faults()
        torch.cuda.synchronize()
        none = torch.isnan(lse)
        assert none.any(), step
        assert torch.isnan(out[none]).all()
        assert torch.equal(out[~none], clean[~none]) and torch.equal(lse[~none], clse[~none])
        call(out, lse)
        assert torch.equal(out, clean) and torch.equal(lse, clse)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype,ns,ctx", [("bf16", [256, 130, 64], [5000, 3333, 6001]), ("e4m3", [256, 130, 64], [5000, 3333, 6001]),
                                          ("bf16", [300], [700]), ("e4m3", [6, 3], [20000, 9000]), ("e4m3", [3], [30000])])
def test_waits_that_run_out(hd, dtype, ns, ctx):
    """Chunks (two blocks an item, and one) and few rows over long 8-bit contexts: a block that gives up
    early or late leaves NaN, and its products and copies in flight end before it does."""
    c, q, cu, lens = _paged_case(61, 16, 4, hd, 64, dtype, ns, ctx)
    _give_up(lambda o, l: sv.attn_paged(q, c, cu, lens, max_q=max(ns), out=o, lse=l), q, (1, 2, 3))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_items_taken_by_a_block_that_gives_up(dtype, hd):
    """Far more items than blocks at work: one that a block took over from the grid just before it gave
    up is written (as NaN) too, however often."""
    ns = [900, 1500, 1, 640] * 4 if dtype == "bf16" else [600, 256, 31, 500] * 5
    ctx = ns if dtype == "bf16" else [n + 300 for n in ns]
    c, q, cu, lens = _paged_case(62, 16, 8, hd, 64, dtype, ns, ctx)
    for step in (1, 3, 6, 9, 14, 20):
        _give_up(lambda o, l: sv.attn_paged(q, c, cu, lens, max_q=max(ns), out=o, lse=l), q, (step,) * 3)


@pytest.mark.parametrize("seqs,n,ctx,hq,hk,hd,ps", [
    (64, 16, 4096, 32, 8, 128, 16), (64, 9, 4096, 32, 8, 128, 16), (32, 6, 4096, 32, 8, 128, 16), (3, 4, 20000, 16, 4, 64, 16),
    (64, 16, 4096, 32, 8, 64, 64), (1, 16, 20000, 16, 4, 128, 32), (1, 64, 20000, 4, 4, 128, 32), (2, 40, 9000, 8, 4, 128, 16),
    (16, 1, 4096, 32, 8, 128, 64), (5, 30, 2048, 8, 2, 128, 16)])
def test_workspace_is_used_where_asked_for(seqs, n, ctx, hq, hk, hd, ps):
    """spec_attn_paged_workspace and the call go by one rule: bytes are asked for where the call uses
    them, and a call that asks for none leaves what it is given alone."""
    g = _gen(71)
    need = -(-ctx // ps)
    table = torch.randint(0, 64, (seqs, need), generator=g, device="cuda").int()
    c = sv.KVCache.empty(64, ps, hk, hd, table, "e4m3")
    for t in (c.k, c.v):
        t.copy_(_randn(g, *t.shape))
    q, lens = _randn(g, seqs * n, hq, hd).bfloat16(), _i32([ctx] * seqs)
    cu, L = _i32([n * b for b in range(seqs + 1)]), sv.lib()
    want = L.spec_attn_paged_workspace(c._ref, seqs * n, n, hq)
    ws = torch.full((max(want, 1 << 25),), 0x5a, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    assert L.spec_attn_paged(c._ref, q.data_ptr(), q.stride(0), q.stride(1), cu.data_ptr(), lens.data_ptr(), seqs * n, n, hq, 0.0,
                             out.data_ptr(), hq * hd, hd, None, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out, sv.attn_paged(q, c, cu, lens, max_q=n)[0])
    assert bool((ws != 0x5a).any()) == (want > 0)


def test_gradients_are_refused_or_whole():
    """Rows that require grad are refused; a Function of one's own has the rotation's gradient by `inverse`."""
    g = _gen(81)
    n, hq, hk, hd = 9, 8, 2, 64
    c, q, cu, lens = _paged_case(81, hq, hk, hd, 16, "bf16", [n], [40])
    pos, plan = torch.arange(n, device="cuda").int(), sv.rope_plan(hd, 10000.0)
    leaf, kv = q.clone().requires_grad_(), q[:, :hk].contiguous()
    seq = torch.zeros_like(pos)
    for call in (lambda: sv.rope_rows(leaf, pos, plan), lambda: sv.attn_paged(leaf, c, cu, lens),
                 lambda: sv.attn_prompt(leaf, kv, kv, cu), lambda: sv.attn_prompt(q, leaf[:, :hk], kv, cu),
                 lambda: sv.attn_prompt(q, kv, leaf[:, :hk], cu), lambda: sv.kv_append(c, leaf[:, :hk], kv, seq, pos),
                 lambda: sv.kv_append(c, kv, leaf[:, :hk], seq, pos)):
        with pytest.raises(sv.SpecError, match="requires grad"):
            call()
    with torch.no_grad():
        assert torch.equal(sv.attn_paged(leaf, c, cu, lens)[0], sv.attn_paged(q, c, cu, lens)[0])

    class Rotate(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return sv.rope_rows(x, pos, plan)

        @staticmethod
        def backward(ctx, dy):
            return sv.rope_rows(dy.contiguous(), pos, plan, inverse=True)

    x, u = _randn(g, n, hq, hd).requires_grad_(), _randn(g, n, hq, hd)
    (Rotate.apply(x) * u).sum().backward()
    ref, size = _rope_ref(u, pos, _freqs(hd, 10000.0), False, sign=-1.0)
    assert ((x.grad.to(F64) - ref).abs() <= size * (8 * 2.0 ** -23 + n * 2.0 ** -50) + ref.abs() * 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("seqs,n,ctx,hq,hk", [(2, 4, 320, 8, 2), (2, 3, 16384, 8, 1), (60, 12, 512, 32, 8), (3, 100, 512, 8, 2),
                                              (2, 250, 4096, 8, 2)])
def test_lengths_past_the_table(seqs, n, ctx, hq, hk, hd, dtype):
    """Lengths beyond what the table holds are cut there, in every kernel: few rows, few rows of a long
    8-bit context, 48 rows, many rows, many rows of few sequences."""
    ns = [n] * seqs
    c, q, cu, lens = _paged_case(91 + hd, hq, hk, hd, 64, dtype, [n] * seqs, [ctx] * seqs)
    assert c.max_pages * 64 == ctx
    out, lse = sv.attn_paged(q, c, cu, lens, max_q=n)
    b = seqs - 1
    pos = torch.arange(ctx, device="cuda").int()
    k, v = _read(c, _values(c), torch.full_like(pos, b), pos)
    _check_rows(out[b * n:], lse[b * n:], _attend_ref(q[b * n:], k, v, n, hd ** -0.5), ctx, hd)
    for far in (ctx + 1, ctx + 64, 2 * ctx, 2 ** 31 - 1):
        for which in (slice(None), slice(0, 1), slice(b, None)):
            past = lens.clone()
            past[which] = far
            o, l = sv.attn_paged(q, c, cu, past, max_q=n)
            assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_gather_one_side(dtype, out):
    """Either output alone, rows of NaN among the others, and the other output's memory left alone."""
    g = _gen(92)
    hk, hd, n = 3, 64, 50
    c = _cache(g, 2, 64, hk, 32, hd, dtype)
    x = _randn(g, n, 2 * hk, hd)
    x[7, 1, 3] = x[9, hk + 2, 5] = math.nan
    seq, pos = _i32([i % 2 for i in range(n)]), _i32([i // 2 for i in range(n)])
    sv.kv_append(c, x[:, :hk], x[:, hk:], seq, pos)
    k, v = sv.kv_gather(c, seq, pos, dtype=out)
    row = slice(None) if dtype == "e4m3" else 3
    assert torch.isnan(k[7, 1, row]).all() and torch.isnan(v[9, 2, slice(None) if dtype == "e4m3" else 5]).all()
    code, L = sv.SPEC_DTYPE_F32 if out == torch.float32 else sv.SPEC_DTYPE_BF16, sv.lib()
    bits = lambda t: t.view(torch.int32 if out == torch.float32 else torch.int16)
    for first in (True, False):
        y = torch.full((2, n, hk, hd), 7.0, dtype=out, device="cuda")
        p = [y[0].data_ptr(), None] if first else [None, y[1].data_ptr()]
        assert L.spec_kv_gather(c._ref, seq.data_ptr(), pos.data_ptr(), n, *p, code, torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(bits(y[0 if first else 1]), bits(k if first else v)) and (y[1 if first else 0] == 7.0).all()
