"""Attention with a sliding window and first tokens that stay visible, and attention of
sequences behind a shared prefix, against plain 64-bit forms.

Tolerances are those of the paged attention (they count the keys' roundings and one
bf16 rounding of a weight and of the output).  A row joined from parts has for each
part a factor 2^(m_i - M), off by 2 units (2^-22) and one product's rounding, in its
sums: parts times 2^-21 of sum w|v| at most, and the same of the row's sum; parts are
at most keys / 128 + 2, which the bound's keys * 2^-23 covers from 600 keys on, and
the 2^-20 for the two or three parts of fewer.
"""
import math

import pytest
import torch

import speculative_decoding_verification_step_gb300 as sv
from test_gpu_paged import (F64, _cache, _check_rows, _gen, _give_up, _i32, _paged_case, _paged_check, _randn, _read,
                            _values)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv.build()
    sv.lib()


def _see(n, ctx, window, sinks):
    p, j = torch.arange(ctx - n, ctx, device="cuda")[:, None], torch.arange(ctx, device="cuda")
    return (j <= p) & ((j > p - window) | (j < sinks) if window else j >= 0)


def _ref(q, ks, vs, see, scale):
    """Rows q [n, hq, d] over the keys ks, vs [keys, hk, d] that see [n, keys] names, in 64 bits:
    out, lse and the bounds' sums (sum w|v|, largest scale sum|q k|)."""
    rep = q.shape[1] // ks.shape[1]
    q, ks, vs = q.to(F64), ks.to(F64).repeat_interleave(rep, 1), vs.to(F64).repeat_interleave(rep, 1)
    some = see.any(0)                              # what no row sees may hold anything
    ks, vs, see = ks[some], vs[some], see[:, some]
    if see.shape[1] == 0:
        z = torch.zeros_like(q)
        return z, torch.full(q.shape[:2], -math.inf, dtype=F64, device="cuda"), z, torch.zeros(1, 1, 1, device="cuda")
    s = torch.einsum("nhd,khd->hnk", q, ks) * scale
    size = torch.einsum("nhd,khd->hnk", q.abs(), ks.abs()) * scale
    s = s.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(s, -1)
    w = torch.where(see, torch.exp(s - lse.clamp_min(-1e300).unsqueeze(-1)), torch.zeros_like(s))
    dot = size.masked_fill(~see, 0).amax(-1)
    return torch.einsum("hnk,khd->nhd", w, vs), lse.T, torch.einsum("hnk,khd->nhd", w, vs.abs()), dot.T.unsqueeze(-1)


def _evict(cache, ns, ctx, window, sinks):
    """What no row of the chunks sees becomes NaN; whole pages of it leave the table."""
    ps, c_table = cache.page_size, cache.table.long()
    for b, (n, c) in enumerate(zip(ns, ctx)):
        if not n or not c:
            continue
        lo = max(0, max(0, c - n) - window + 1)
        j = torch.arange(min(sinks, lo), lo, device="cuda")
        page, slot = c_table[b, j // ps], j % ps
        for t in (cache.k, cache.v):
            if t.dtype is torch.bfloat16:
                t[page, :, slot] = math.nan
        if cache.k_scale is not None:
            cache.k_scale[page, :, slot] = cache.v_scale[page, :, slot] = 255
        p = torch.arange(cache.max_pages, device="cuda")
        cache.table[b].masked_fill_((p * ps >= sinks) & ((p + 1) * ps <= lo), -1)


def _window_check(c, q, cu, lens, ns, ctx, window, sinks, values, max_q=None):
    hd = q.shape[2]
    out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    sv.attn_paged(q, c, cu, lens, max_q=max_q, out=out, lse=lse, window=window, sinks=sinks)
    r = 0
    for b, (n, m) in enumerate(zip(ns, ctx)):
        k, v = values[b]
        _check_rows(out[r:r + n], lse[r:r + n], _ref(q[r:r + n], k, v, _see(n, m, window, sinks), hd ** -0.5), m, hd)
        r += n
    assert (out[r:] == 7.0).all() and (lse[r:] == 9.0).all()
    return out, lse


def _all_values(c, ctx):
    values = _values(c)
    return [_read(c, values, torch.full((m,), b, dtype=torch.int32, device="cuda"), torch.arange(m, device="cuda").int())
            for b, m in enumerate(ctx)]


WINDOW = [  # hq, hk, hd, page, new tokens, contexts, window, sinks
    (32, 8, 128, 16, [6], [512], 100, 4),
    (32, 8, 128, 16, [6, 6, 6], [513, 47, 1000], 64, 0),
    (32, 8, 64, 32, [1] * 5, [1, 2, 16, 17, 3000], 16, 1),
    (8, 2, 32, 16, [5, 1, 9], [5, 333, 64], 1, 0),              # a row sees itself alone
    (4, 4, 64, 64, [1, 17, 16], [129, 17, 700], 33, 17),
    (7, 1, 128, 32, [3, 5], [300, 5], 10, 300),                 # more first tokens than keys
    (12, 4, 128, 256, [2, 0, 4], [40, 10, 600], 700, 3),        # a window past the contexts
    (8, 2, 64, 16, [4, 3, 2], [2, 0, 1], 2, 1),                 # chunks longer than their contexts: empty rows
    (8, 2, 64, 16, [2, 1, 1], [40, 25, 31], 15, 9),             # the first tokens end beside the window
    (2, 2, 64, 16, [1], [20000], 5000, 100),
    (16, 2, 128, 16, [4, 4], [20000, 9000], 4096, 4),
    (8, 2, 64, 64, [130, 257, 1], [500, 257, 100], 50, 4),
    (32, 8, 128, 32, [129], [1500], 200, 0),
    (32, 8, 128, 16, [40, 300, 3], [900, 2000, 300], 129, 140),  # first tokens over two steps of 128
    (4, 2, 128, 64, [200, 400], [200, 3000], 1, 1),
    (16, 4, 64, 16, [300], [5000], 700, 16),
    (32, 8, 128, 16, [128] * 4, [1000, 800, 300, 128], 128, 128),
    (8, 8, 128, 16, [400], [900], 2 ** 31 - 1, 2 ** 31 - 1),
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,hd,ps,ns,ctx,window,sinks", WINDOW)
def test_window_paged(hq, hk, hd, ps, ns, ctx, window, sinks, dtype):
    c, q, cu, lens = _paged_case(sum(ctx) + hd, hq, hk, hd, ps, dtype, ns, ctx, pad=2)
    values = _all_values(c, ctx)
    _evict(c, ns, ctx, window, sinks)
    a = _window_check(c, q, cu, lens, ns, ctx, window, sinks, values)
    b = _window_check(c, q, cu, lens, ns, ctx, window, sinks, values, max_q=max(ns))
    again = sv.attn_paged(q, c, cu, lens, max_q=max(ns), window=window, sinks=sinks)
    n = sum(ns)
    assert torch.equal(again[0][:n], b[0][:n]) and torch.equal(again[1][:n], b[1][:n])
    assert a[0].shape == b[0].shape


LONG = [  # few rows over long windows of 8-bit keys
    (32, 8, 128, 16, [6] * 24, [2500 + 37 * i for i in range(24)], 2100, 4),
    (32, 8, 128, 64, [4, 6, 5, 1] * 6, [3000 - 41 * i for i in range(24)], 2048, 130),
    (16, 4, 64, 32, [6, 3], [30000, 9000], 17000, 5),
    (16, 4, 128, 16, [8], [40000], 20001, 0),
    (4, 2, 128, 256, [16, 2], [20000, 18000], 17000, 300),
    (16, 2, 64, 16, [1, 2], [40000, 16500], 16400, 1),
]


@pytest.mark.parametrize("hq,hk,hd,ps,ns,ctx,window,sinks", LONG)
def test_window_few_rows_long(hq, hk, hd, ps, ns, ctx, window, sinks):
    c, q, cu, lens = _paged_case(sum(ctx), hq, hk, hd, ps, "e4m3", ns, ctx, pad=1)
    n = sum(ns)
    assert sv.lib().spec_attn_paged_window_workspace(c._ref, n + 1, max(ns), hq, window, sinks) > 0
    values = _all_values(c, ctx)
    _evict(c, ns, ctx, window, sinks)
    a = _window_check(c, q, cu, lens, ns, ctx, window, sinks, values, max_q=max(ns))
    for _ in range(3):
        again = sv.attn_paged(q, c, cu, lens, max_q=max(ns), window=window, sinks=sinks)
        assert torch.equal(again[0][:n], a[0][:n]) and torch.equal(again[1][:n], a[1][:n])
    if n < 30:
        rows = q[:n]
        _give_up(lambda o, l: sv.attn_paged(rows, c, cu, lens, max_q=max(ns), out=o, lse=l, window=window, sinks=sinks), rows, (1, 3))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 6, 40, 200])
def test_window_of_everything(dtype, n):
    """A window as long as the contexts is plain attention, and window 0 is the call without one."""
    ns, ctx = [n, n], [700, 513]
    c, q, cu, lens = _paged_case(77, 16, 4, 128, 32, dtype, ns, ctx)
    _paged_check(c, q, cu, lens, ns, ctx, max_q=n, window=700)
    ref = sv.attn_paged(q, c, cu, lens, max_q=n)
    for kw in (dict(window=0), dict(window=0, sinks=5)):
        got = sv.attn_paged(q, c, cu, lens, max_q=n, **kw)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [6, 130])
def test_window_bounds_and_bad_indices(dtype, n):
    """max_q leaves rows, lengths past the table are cut, bad entries read as zeros, broken row starts
    are skipped, and neighbours are as they were."""
    ns, ctx = [n, n, n], [300, 700, 450]
    c, q, cu, lens = _paged_case(31, 8, 2, 64, 16, dtype, ns, ctx)
    kw = dict(window=100, sinks=4)
    ref, rl = sv.attn_paged(q, c, cu, lens, max_q=n, **kw)
    out, lse = torch.full_like(ref, 3.0), torch.full_like(rl, 3.0)
    sv.attn_paged(q, c, cu, lens, max_q=2, out=out, lse=lse, **kw)
    assert (out.view(3, n, 8, 64)[:, 2:] == 3.0).all() and torch.isfinite(out.float()).all()
    for bad in ([0, n, 2 * n, 10 ** 6], [-5, n, 2 * n, 3 * n], [0, n, n, 3 * n]):
        got, _ = sv.attn_paged(q, c, _i32(bad), lens, max_q=n, out=torch.full_like(ref, 3.0), **kw)
        same = slice(n, 2 * n) if bad[2] == 2 * n else slice(0, n)
        assert torch.equal(got[same], ref[same])
    saved = c.table.clone()
    c.table[0, :] = 2 ** 30
    c.table[1, 30:] = -3
    got, gl = sv.attn_paged(q, c, cu, lens, max_q=n, **kw)
    assert torch.equal(got[2 * n:], ref[2 * n:]) and (got[:n] == 0).all()
    assert torch.isfinite(gl[:n]).all()                       # keys of zeros: scores of 0
    c.table.copy_(saved)
    cap = c.max_pages * 16
    over, want = (sv.attn_paged(q, c, cu, _i32([300, x, 450]), max_q=n, **kw)[0] for x in (2 ** 31 - 1, cap))
    assert torch.equal(over.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("hq,hk,hd,ns,window,sinks", [
    (8, 2, 64, [130, 1, 77], 20, 4),
    (32, 8, 128, [17], 5, 1),
    (8, 2, 32, [100, 33], 1, 0),
    (7, 1, 128, [64, 0, 65, 200], 50, 60),
    (12, 4, 64, [600, 129, 3], 128, 0),
    (4, 4, 128, [1025], 300, 4),
    (32, 8, 128, [900, 1500], 129, 130),
    (16, 2, 64, [2000], 1000, 7),
    (32, 8, 128, [2100], 64, 16),
])
def test_window_prompt(hq, hk, hd, ns, window, sinks):
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
        sv.attn_prompt(q, k, v, _i32(cu), max_len=bound, out=out, lse=lse, window=window, sinks=sinks)
        for b, n in enumerate(ns):
            r = slice(cu[b], cu[b + 1])
            if n:
                _check_rows(out[r], lse[r], _ref(q[r], k[r], v[r], _see(n, n, window, sinks), hd ** -0.5), n, hd)
        assert (out[total:] == 7.0).all() and (lse[total:] == 9.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd", [64, 128])
def test_window_waits_that_run_out(hd, dtype):
    ns, ctx = [256, 130, 64], [5000, 3333, 6001]
    c, q, cu, lens = _paged_case(63, 16, 4, hd, 64, dtype, ns, ctx)
    _give_up(lambda o, l: sv.attn_paged(q, c, cu, lens, max_q=256, out=o, lse=l, window=1500, sinks=4), q, (1, 2, 5))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 6, 40, 200])
def test_window_far_past_everything(dtype, n):
    """The longest table there is, and windows and first tokens near 2^31: no place of a walk leaves 32 bits."""
    ns, ctx = [n, n], [700, 513]
    c, q, cu, lens = _paged_case(78, 16, 4, 128, 256, dtype, ns, ctx)
    t = torch.full((2, 0x7fffff00 // 256), -1, dtype=torch.int32, device="cuda")
    t[:, :c.max_pages] = c.table
    values = _all_values(c, ctx)
    far = sv.KVCache(c.k, c.v, t, c.k_scale, c.v_scale)
    for window, sinks in ((0x7ffffeff, 0x7fffffff), (2 ** 30 + 1, 0), (2 ** 30 + 1, 2 ** 31 + 7), (0x7ffffeff, 5)):
        _window_check(far, q, cu, lens, ns, ctx, window, sinks, values, max_q=n)
    _window_check(far, q, cu, lens, ns, ctx, 100, 2 ** 31 - 1, values, max_q=n)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_more_past_32_bit_offsets(dtype):
    """Pages that lie past 2^31 elements: written by qkv_append, read in a window and behind a shared prefix."""
    hk, ps, hd, hq = 8, 256, 128, 32
    pages = 2 ** 31 // (hk * ps * hd) + 12
    if torch.cuda.mem_get_info()[0] < 4 * pages * hk * ps * hd * (2 if dtype == "bf16" else 1):
        pytest.skip("not enough memory")
    g = _gen(17)
    table = torch.full((3, 4000), -1, dtype=torch.int32, device="cuda")
    table[:, :4] = pages - 12 + torch.randperm(12, generator=g, device="cuda").int().view(3, 4)
    table[1:, :2] = table[0, :2]
    c = sv.KVCache.empty(pages, ps, hk, hd, table, dtype)
    ctx, ns = [900, 700, 1000], [6, 6, 6]
    plan, gain = sv.rope_plan(hd, 500000.0), torch.exp(0.3 * _randn(g, hd))
    for b, m in enumerate(ctx):
        pos = torch.arange(m, device="cuda").int()
        x = _randn(g, m, hq + 2 * hk, hd).bfloat16()
        live = pos if b == 0 else torch.where(pos < 2 * ps, -1, pos)     # (the shared pages are written once)
        sv.qkv_append(c, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], torch.full_like(pos, b), live, plan, gain, gain)
    q = _randn(g, 18, hq, hd).bfloat16()
    cu, lens, values = _i32([0, 6, 12, 18]), _i32(ctx), _all_values(c, ctx)
    assert all(v.abs().amax() > 0 for kv in values for v in kv)
    _window_check(c, q, cu, lens, ns, ctx, 300, 4, values, max_q=6)
    assert _shares(c, 1, 18, 6, hq)
    _shared_check(c, q, cu, lens, ns, ctx, _i32([2 * ps]), None, 6)


# ------------------------------------------------------------ shared prefixes
def _shared_case(seed, hq, hk, hd, ps, dtype, ns, first, shared, rests, pad=0):
    """Sequences whose rows of the table begin alike within a group; slots past the lengths hold NaN.
    first: the groups' first sequences and the end; rests: positions of every sequence behind the prefix."""
    g = _gen(seed)
    group = [max((i for i, f in enumerate(first[:-1]) if f <= b), default=-1) if b < first[-1] else -1 for b in range(len(ns))]
    lens = [(max(shared[x], 0) if x >= 0 else 0) + r for x, r in zip(group, rests)]
    cache = _cache(g, len(ns), max(max(lens), 1), hk, ps, hd, dtype)
    for b, x in enumerate(group):
        if x >= 0:
            k = -(-max(shared[x], 0) // ps)
            cache.table[b, :k] = cache.table[first[x], :k]
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x7f) if dtype == "e4m3" else t.fill_(math.nan)
    if dtype == "e4m3":
        cache.k_scale.fill_(255)
        cache.v_scale.fill_(255)
    rows = [(b, p) for b, n in enumerate(lens) for p in range(n)]
    if rows:
        seq, pos = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in zip(*rows))
        slot = cache.table[seq.long(), (pos // ps).long()].long() * ps + pos % ps
        _, inv = torch.unique(slot, return_inverse=True)         # one writer a slot
        once = torch.full((int(inv.max()) + 1,), len(rows), device="cuda").scatter_reduce(
            0, inv, torch.arange(len(rows), device="cuda"), "amin")
        seq, pos = seq[once], pos[once]
        sv.kv_append(cache, _randn(g, len(once), hk, hd), _randn(g, len(once), hk, hd), seq, pos)
    cu = [0]
    for n in ns:
        cu.append(cu[-1] + n)
    q = _randn(g, cu[-1] + pad, hq + 1, hd).bfloat16()[:, :hq]
    return cache, q, _i32(cu), _i32(lens), lens


def _wide(c):
    """The cache with a table whose width makes sharing pay for any of these batches (the lengths are
    the device's own; entries past them name nothing)."""
    t = torch.full((c.seqs, max(c.max_pages, 900000 // c.page_size)), -1, dtype=torch.int32, device="cuda")
    t[:, :c.max_pages] = c.table
    return sv.KVCache(c.k, c.v, t, c.k_scale, c.v_scale)


def _shares(c, groups, n, max_q, hq):
    """Whether a call of these sizes shares anything: the prefixes' parts need room of their own."""
    L = sv.lib()
    return (L.spec_attn_shared_workspace(c._ref, groups, n, max_q, hq)
            > L.spec_attn_paged_workspace(c._ref, n, max_q, hq) + 256 * n)


def _shared_check(c, q, cu, lens, ns, ctx, shared, groups, max_q):
    hd = q.shape[2]
    out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    got = sv.attn_shared(q, c, cu, lens, shared, groups=groups, max_q=max_q, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    r = 0
    for b, ((k, v), n, m) in enumerate(zip(_all_values(c, ctx), ns, ctx)):
        k, v = k[:m], v[:m]
        _check_rows(out[r:r + n], lse[r:r + n], _ref(q[r:r + n], k, v, _see(n, m, 0, 0), hd ** -0.5), m, hd)
        r += n
    assert (out[r:] == 7.0).all() and (lse[r:] == 9.0).all()
    return out, lse


SHARED = [  # hq, hk, hd, page, new tokens, groups, shared, positions behind the prefix
    (32, 8, 128, 16, [6] * 4, [0, 4], [512], [6, 50, 64, 17]),
    (32, 8, 128, 16, [1] * 9, [0, 9], [3000], [1, 2, 16, 17, 33, 100, 1, 5, 300]),
    (8, 2, 64, 32, [1, 4, 9, 2], [0, 2, 4], [640, 1024], [1, 20, 9, 700]),
    (8, 2, 64, 64, [3, 3, 3, 3, 3], [1, 3], [129], [10, 4, 5, 300, 3]),           # three outside the group
    (7, 1, 128, 32, [3, 5, 1], [0, 3], [777], [40, 30, 60]),                      # ends inside a page
    (12, 4, 128, 256, [2, 0, 4, 1], [0, 4], [512], [40, 10, 60, 1]),              # a sequence without new tokens
    (16, 2, 128, 16, [8] * 5, [0, 1, 5], [100, 2000], [8, 8, 9, 10, 300]),        # a group of one
    (8, 8, 64, 16, [1, 60, 2], [0, 3], [300], [1, 60, 300]),                      # 60 rows a KV head
    (32, 8, 64, 16, [2] * 40, [0, 10, 20, 30, 40], [400, 16, 0, 2000], [2 + i for i in range(40)]),
    (128, 1, 128, 16, [1] * 6, [0, 6], [700], [1, 9, 20, 33, 1, 64]),             # too many rows a KV head
    (64, 1, 128, 16, [1] * 6, [0, 6], [700], [1, 9, 20, 33, 1, 64]),              # a tile holds two tokens
    (120, 2, 64, 32, [1] * 5, [0, 5], [900], [1, 9, 20, 33, 1]),                  # 60 rows: a tile of 120
    (4, 4, 128, 16, [1] * 300, [0, 300], [256], [1 + i % 40 for i in range(300)]),  # two row pairs a head
    (6, 2, 64, 16, [1, 1], [0, 2], [-5], [30, 40]),
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,hd,ps,ns,first,shared,rests", SHARED)
def test_shared(hq, hk, hd, ps, ns, first, shared, rests, dtype):
    c, q, cu, lens, ctx = _shared_case(sum(rests) + hd, hq, hk, hd, ps, dtype, ns, first, shared, rests, pad=3)
    sh, gr = _i32(shared), _i32(first)
    c = _wide(c)
    assert _shares(c, len(shared), q.shape[0], max(ns), hq) == (max(ns) * hq // hk <= 64)
    a = _shared_check(c, q, cu, lens, ns, ctx, sh, gr, max(ns))
    if first == [0, len(ns)]:
        b = sv.attn_shared(q, c, cu, lens, sh, max_q=max(ns))
        n = sum(ns)
        assert torch.equal(a[0][:n], b[0][:n]) and torch.equal(a[1][:n], b[1][:n])
    # a number past what every row sees is cut there (within the table's alike pages), a smaller one is as good
    for less in ([max(0, s - 37) for s in shared], [s // 3 for s in shared]):
        _shared_check(c, q, cu, lens, ns, ctx, _i32(less), gr, max(ns))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd", [64, 128])
def test_shared_is_cut_to_what_rows_see(dtype, hd):
    """Sequences that name the same pages all along, of different lengths: the shortest one's new
    tokens bound what is shared, whatever the call says."""
    ns, ctx = [2, 1, 3, 0], [900, 400, 650, 3]
    g = _gen(hd)
    c = _cache(g, 4, 900, 2, 16, hd, dtype)
    c.table.copy_(c.table[:1].expand_as(c.table).clone())
    pos = torch.arange(900, device="cuda").int()
    sv.kv_append(c, _randn(g, 900, 2, hd), _randn(g, 900, 2, hd), torch.zeros_like(pos), pos)
    c = _wide(c)
    assert _shares(c, 1, 6, 3, 8)
    q = _randn(g, 6, 8, hd).bfloat16()
    cu, lens = _i32([0, 2, 3, 6, 6]), _i32(ctx)
    for shared in (399, 400, 900, 2 ** 31 - 1, 384, 1, 0):
        _shared_check(c, q, cu, lens, ns, ctx, _i32([shared]), None, 3)
    _shared_check(c, q, cu, _i32([900, 1, 650, 3]), ns, [900, 1, 650, 3], _i32([500]), None, 3)    # nothing left


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_shared_bad_indices(dtype):
    """Groups and row starts that make no sense: nothing outside the rows is written, sequences of sound
    groups are as they were."""
    ns, first, shared = [4] * 6, [0, 3, 6], [600, 300]
    c, q, cu, lens, ctx = _shared_case(5, 16, 4, 128, 16, dtype, ns, first, shared, [20] * 6, pad=2)
    c = _wide(c)
    assert _shares(c, 2, 26, 4, 16)
    ref, _ = sv.attn_shared(q, c, cu, lens, _i32(shared), groups=_i32(first), max_q=4)
    call = lambda g, cu=cu, t=None: sv.attn_shared(q, c, cu, lens, _i32(shared), groups=_i32(g), max_q=4,
                                                   out=torch.full_like(ref, 7.0))[0]
    for g in ([0, 3, 7], [-1, 3, 6], [0, 3, 2 ** 31 - 1], [3, 6, 0], [5, 2, 6], [0, 6, 3], [-2 ** 31, 0, 2 ** 31 - 1]):
        assert (call(g)[24:] == 7.0).all()
    out = call([3, 3, 6])
    plain, _ = sv.attn_paged(q, c, cu, lens, max_q=4)
    assert torch.allclose(out[:12].float(), plain[:12].float(), rtol=2 ** -6, atol=2 ** -6)     # (in no group: whole)
    assert torch.equal(call([0, 3, 6])[:24], ref[:24])
    for bad in ([0, 4, 8, 12, 16, 20, 10 ** 6], [-9, 4, 8, 12, 16, 20, 24], [0, 20, 4, 12, 16, 20, 24]):
        assert (call(first, cu=_i32(bad))[24:] == 7.0).all()
    c.table[:3, 5] = 2 ** 30                                     # a page outside the pool reads as zeros
    got = call(first)
    assert torch.equal(got[12:24], ref[12:24]) and torch.isfinite(got[:12].float()).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_shared_streams_graphs_workspaces(dtype):
    """The same bits on streams beside one another, replayed with new lengths and prefixes, and with a
    workspace that holds anything; without one the call is attn_paged."""
    ns, first, shared = [3] * 8, [0, 5, 8], [2000, 900]
    c, q, cu, lens, ctx = _shared_case(9, 32, 8, 128, 16, dtype, ns, first, shared, [30, 200] * 4)
    narrow = c
    c = _wide(c)
    assert _shares(c, 2, 24, 3, 32)
    sh, gr = _i32(shared), _i32(first)
    q2 = q.flip(0).contiguous()
    call = lambda x, **kw: sv.attn_shared(x, c, cu, lens, sh, groups=gr, max_q=3, **kw)
    ref, ref2 = call(q), call(q2)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got, got2 = [], []
    for _ in range(10):
        with torch.cuda.stream(a):
            got.append(call(q))
        got2.append(call(q2, stream=b.cuda_stream))
    torch.cuda.synchronize()
    for x, want in [(x, ref) for x in got] + [(x, ref2) for x in got2]:
        assert torch.equal(x[0], want[0]) and torch.equal(x[1], want[1])
    L, n = sv.lib(), 24
    need = L.spec_attn_shared_workspace(c._ref, 2, n, 3, 32)
    ws = torch.full((need + 256,), 0xff, dtype=torch.uint8, device="cuda")
    plain = sv.attn_paged(q, c, cu, lens, max_q=3)
    # where sharing does not pay the call is attn_paged
    assert not _shares(narrow, 2, n, 3, 32)
    for x, y in zip(sv.attn_shared(q, narrow, cu, lens, sh, groups=gr, max_q=3), sv.attn_paged(q, narrow, cu, lens, max_q=3)):
        assert torch.equal(x, y)
    for size in (0, max(0, need - 16), need):
        out, lse = torch.zeros(n, 32, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 32, device="cuda")
        assert L.spec_attn_shared(c._ref, q.data_ptr(), q.stride(0), q.stride(1), cu.data_ptr(), lens.data_ptr(),
                                  gr.data_ptr(), 2, sh.data_ptr(), n, 3, 32, 0.0, out.data_ptr(), 32 * 128, 128,
                                  lse.data_ptr(), ws.data_ptr() if size else None, size,
                                  torch.cuda.current_stream().cuda_stream) == 0
        if size == need:
            assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
        else:
            assert torch.allclose(out.float(), plain[0].float(), rtol=2 ** -6, atol=2 ** -6)
    assert (ws[need:] == 0xff).all()
    graph, o = torch.cuda.CUDAGraph(), torch.zeros_like(ref[0])
    with torch.cuda.graph(graph):
        call(q, out=o)
    for new, less in ((shared, 0), ([640, 0], 0), ([1999, 17], 5), ([0, 0], 0), ([5000, 5000], 1)):
        sh.copy_(_i32(new))
        lens.copy_(_i32([x - less for x in ctx]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, call(q)[0])


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_shared_waits_that_run_out(dtype, hd):
    """A prefix block that gives up leaves NaN in the rows of all parts of its run, also of those that it
    did not come to."""
    ns, first, shared = [4] * 40, [0, 30, 40], [3000, 900]
    c, q, cu, lens, ctx = _shared_case(19, 16, 4, hd, 16, dtype, ns, first, shared, [9] * 40)
    c = _wide(c)
    assert _shares(c, 2, 160, 4, 16)
    sh, gr = _i32(shared), _i32(first)
    _give_up(lambda o, l: sv.attn_shared(q, c, cu, lens, sh, groups=gr, max_q=4, out=o, lse=l), q, (1, 2))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd,ps", [(128, 16), (64, 64)])
def test_serving_loop(dtype, hd, ps):
    """The calls as a program runs them together: a prompt for all sequences, then verify steps whose
    pages are reserved and given back on the device, rows normed, rotated and written in one call, and
    attention behind the prompt and in a window, all against 64-bit forms of the cache's values."""
    g = _gen(hd)
    hq, hk, seqs, width = 8, 2, 5, 640 // ps + 2
    prompt = 512
    shared_pages = prompt // ps
    table = torch.full((seqs, 250000 // ps), -1, dtype=torch.int32, device="cuda")   # (wide: sharing pays)
    pool = shared_pages + seqs * (width - shared_pages)
    c = sv.KVCache.empty(pool, ps, hk, hd, table, dtype)
    table[:, :shared_pages] = torch.arange(shared_pages, device="cuda").int()
    free = torch.arange(shared_pages, pool, device="cuda").int()
    n_free = _i32([pool - shared_pages])
    plan, gq, gk = sv.rope_plan(hd, 500000.0), *(torch.exp(0.3 * _randn(g, hd)) for _ in range(2))

    def rows(n, seq, pos):
        x = _randn(g, n, hq + 2 * hk, hd).bfloat16()
        return sv.qkv_append(c, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], seq, pos, plan, gq, gk)

    pos = torch.arange(prompt, device="cuda").int()
    rows(prompt, torch.zeros_like(pos), pos)                     # the prompt, once
    lens, shared = _i32([prompt] * seqs), _i32([prompt])
    held = n_free.item()
    for counts, kept in (([6] * 5, [1, 6, 3, 2, 4]), ([6, 1, 0, 6, 6], [2, 1, 0, 6, 1]), ([40] * 5, [40, 1, 17, 33, 2])):
        cap = sum(counts) + 7
        cu, now, seq, pos, lacking = sv.kv_reserve(c, lens, _i32(counts), free, n_free, cap)
        assert lacking.item() == 0 and now.tolist() == [a + b for a, b in zip(lens.tolist(), counts)]
        q = rows(cap, seq, pos)
        _shared_check(c, q, cu, now, counts, now.tolist(), shared, None, max(counts))
        _window_check(c, q, cu, now, counts, now.tolist(), 50, 4, _all_values(c, now.tolist()), max_q=max(counts))
        lens = lens + _i32(kept)
        sv.kv_release(c, now, lens, free, n_free)
        pages = sum(-(-x // ps) - shared_pages for x in lens.tolist())
        assert n_free.item() == held - pages
    sv.kv_release(c, lens, _i32([prompt] * seqs), free, n_free)
    assert n_free.item() == held and sorted(free.tolist()) == list(range(shared_pages, pool))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd", [64, 128])
def test_shared_workspace_alignment(dtype, hd):
    """Workspaces at any multiple of 16 bytes: the same bits, and nothing outside the bytes asked for."""
    ns, first, shared = [3] * 6, [0, 4, 6], [1500, 333]
    c, q, cu, lens, ctx = _shared_case(29, 16, 4, hd, 32, dtype, ns, first, shared, [7, 300] * 3)
    c = _wide(c)
    assert _shares(c, 2, 18, 3, 16)
    sh, gr, n = _i32(shared), _i32(first), 18
    ref = sv.attn_shared(q, c, cu, lens, sh, groups=gr, max_q=3)
    L = sv.lib()
    need = L.spec_attn_shared_workspace(c._ref, 2, n, 3, 16)
    ws = torch.empty(need + 512, dtype=torch.uint8, device="cuda")
    assert ws.data_ptr() % 256 == 0
    for at in (16, 32, 48, 112, 0):
        ws.fill_(0xff)
        out, lse = torch.zeros(n, 16, hd, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 16, device="cuda")
        assert L.spec_attn_shared(c._ref, q.data_ptr(), q.stride(0), q.stride(1), cu.data_ptr(), lens.data_ptr(),
                                  gr.data_ptr(), 2, sh.data_ptr(), n, 3, 16, 0.0, out.data_ptr(), 16 * hd, hd,
                                  lse.data_ptr(), ws.data_ptr() + at, need, torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
        assert (ws[:at] == 0xff).all() and (ws[at + need:] == 0xff).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd,ns,first,shared", [
    (128, [0, 2, 1, 0, 3], [0, 5], [400]),
    (64, [0, 0, 4, 4, 0, 0, 0, 1, 2], [0, 4, 9], [640, 77]),
    (128, [0, 1] + [0] * 40 + [1, 1], [0, 1, 44], [300, 512]),       # the second of the group; a group of none
])
def test_shared_behind_idle_sequences(dtype, hd, ns, first, shared):
    """Sequences without new tokens whose pages were given back (no length, cleared entries), the groups'
    first ones among them: the prefix is that of the others."""
    c, q, cu, lens, ctx = _shared_case(23 + hd, 16, 4, hd, 16, dtype, ns, first, shared, [n + 9 for n in ns], pad=2)
    for b, n in enumerate(ns):
        if n == 0:
            c.table[b], lens[b], ctx[b] = -1, 0, 0
    c = _wide(c)
    sh, gr = _i32(shared), _i32(first)
    assert _shares(c, len(shared), q.shape[0], max(ns), 16)
    _shared_check(c, q, cu, lens, ns, ctx, sh, gr, max(ns))
    c.table[torch.tensor(ns, device="cuda") == 0] = 2 ** 30
    _shared_check(c, q, cu, lens, ns, ctx, sh, gr, max(ns))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,hd,ps,ns,ctx,window,sinks", [
    (16, 4, 128, 64, [256, 130], [7000, 3000], 2500, 4),
    (8, 2, 64, 16, [500], [9000], 3000, 300),
    (32, 8, 128, 256, [100], [6000], 5000, 0),
    (8, 2, 128, 32, [300, 200], [2900, 150], 2100, 2000),        # first tokens over many steps; a chunk past its context
])
def test_window_keys_cut_between_two_blocks(hq, hk, hd, ps, ns, ctx, window, sinks, dtype):
    """Few chunks in a long window: two blocks share an item's keys."""
    c, q, cu, lens = _paged_case(sum(ctx) + hd, hq, hk, hd, ps, dtype, ns, ctx, pad=2)
    values = _all_values(c, ctx)
    _evict(c, ns, ctx, window, sinks)
    a = _window_check(c, q, cu, lens, ns, ctx, window, sinks, values, max_q=max(ns))
    n = sum(ns)
    for _ in range(3):
        again = sv.attn_paged(q, c, cu, lens, max_q=max(ns), window=window, sinks=sinks)
        assert torch.equal(again[0][:n], a[0][:n]) and torch.equal(again[1][:n], a[1][:n])
    rows = q[:n]
    _give_up(lambda o, l: sv.attn_paged(rows, c, cu, lens, max_q=max(ns), out=o, lse=l, window=window, sinks=sinks), rows, (1, 4))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd,groups,each", [(128, 9, 3), (64, 33, 2), (128, 70, 2), (64, 130, 3)])
def test_shared_many_groups(dtype, hd, groups, each):
    """More groups than a block's warps, or than a warp has lanes; some share nothing, some have no rows."""
    r = torch.Generator().manual_seed(groups)
    draw = lambda hi, n: torch.randint(0, hi, (n,), generator=r).tolist()
    shared = [0 if i % 7 == 3 else x for i, x in enumerate(draw(400, groups))]
    ns = [0 if b // each % 5 == 2 else 1 + x for b, x in enumerate(draw(3, groups * each))]
    rests = [n + x for n, x in zip(ns, draw(60, groups * each))]
    first = list(range(0, groups * each + 1, each))
    c, q, cu, lens, ctx = _shared_case(31 + groups, 8, 2, hd, 16, dtype, ns, first, shared, rests, pad=1)
    c = _wide(c)
    assert _shares(c, groups, q.shape[0], max(ns), 8)
    _shared_check(c, q, cu, lens, ns, ctx, _i32(shared), _i32(first), max(ns))
