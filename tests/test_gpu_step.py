"""What a step does around the paged cache against plain forms: pages and index
arrays (whole numbers, a loop over the sequences), head norms with rotation and
cache write (64 bits).

Tolerances of the norm: the sum of head_dim squares in fp32 is off by at most
(head_dim + 2) 2^-24 relative (all terms are positive), half of that in its root;
rsqrtf by 2 units, the quotient by head_dim and the sum with eps by one rounding
each, two products: y is off by at most n = (head_dim / 2 + 10) 2^-24 of itself,
and the rotation adds 8 * 2^-23 of |a| + |b| as for the rotation alone.  Then the
output's rounding, half a step.
"""
import pytest
import torch

import speculative_decoding_verification_step_gb300 as sv
from test_gpu_paged import F64, HALF, _freqs, _gen, _i32, _randn, _rope_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv.build()
    sv.lib()


# ------------------------------------------------------- pages and index arrays
def _reserve_ref(table, ps, lens, counts, free, left, tokens):
    table, lens = [list(r) for r in table], list(lens)
    left = max(0, min(left, len(free)))
    cu, seq, pos, asked, toks, top = [0], [], [], 0, 0, left
    for b, (n, want) in enumerate(zip(lens, counts)):
        want = max(0, want)
        got = 0
        if n >= 0 and n + want <= len(table[b]) * ps:
            had, need = -(-n // ps), -(-(n + want) // ps) - -(-n // ps)
            asked += need
            toks += want
            if (need == 0 or asked <= left) and toks <= tokens:
                got = want
                for j in range(need):
                    top -= 1
                    table[b][had + j] = free[top]
        seq += [b] * got
        pos += range(n, n + got)
        lens[b] = n + got
        cu.append(cu[-1] + got)
    pad = [-1] * (tokens - len(seq))
    return table, top, cu, lens, seq + pad, pos + pad, max(0, asked - left)


def _release_ref(table, ps, lens, keep, free, left):
    table, free = [list(r) for r in table], list(free)
    left = max(0, min(left, len(free)))
    for b, (n, k) in enumerate(zip(lens, keep)):
        n = min(max(0, n), len(table[b]) * ps)
        k = min(max(0, k), n)
        for j in range(-(-k // ps), -(-n // ps)):
            if left < len(free):
                free[left] = table[b][j]
                left += 1
            table[b][j] = -1
    return table, free, left


def _pages(seqs, width, ps, pool, table=None):
    """A cache whose pools nothing touches: `pool` pages of the smallest rows."""
    t = torch.full((seqs, width), -1, dtype=torch.int32, device="cuda") if table is None else table
    return sv.KVCache.empty(pool, ps, 1, 32, t)


def _check_reserve(c, ps, lens, counts, free, left, tokens):
    table = c.table.tolist()
    f, n = _i32(free), _i32([left])
    got = sv.kv_reserve(c, _i32(lens), _i32(counts), f, n, tokens)
    want = _reserve_ref(table, ps, lens, counts, free, left, tokens)
    assert n.tolist() == [want[1]] and f.tolist() == free
    for x, y in zip(got, (want[2], want[3], want[4], want[5], [want[6]])):
        assert x.dtype is torch.int32 and x.tolist() == y
    assert c.table.tolist() == want[0]
    return got, f, n


RESERVE = [  # ps, table width, lengths, new tokens, pages in the stack, capacity
    (16, 4, [0], [1], 1, 1),
    (16, 4, [15, 16, 17], [1, 1, 1], 1, 3),                  # one of three crosses a page
    (16, 4, [0, 5, 63], [64, 0, 1], 4, 70),
    (16, 4, [60, 64, 0], [5, 1, 10], 9, 70),                 # two past the table's room
    (16, 8, [0, 0, 0, 3], [40, 40, 40, 2], 6, 200),          # the third lacks pages, the fourth needs none
    (16, 8, [0, 0, 0, 3], [40, 40, 40, 20], 6, 200),
    (32, 8, [10, 10, 10], [9, 9, 9], 8, 20),                 # the third has no room in the token arrays
    (16, 8, [-1, 7, 2 ** 31 - 1, 7], [3, -4, 1, 2 ** 31 - 1], 8, 32),   # no lengths, no counts
    (256, 3, [1, 2, 300], [0, 0, 0], 0, 5),
    (64, 5, [0, 100], [320, 100], 100, 420),
    (16, 4, [1, 1], [1, 1], 7, 0),                           # no tokens at all
]


@pytest.mark.parametrize("ps,width,lens,counts,left,tokens", RESERVE)
def test_reserve(ps, width, lens, counts, left, tokens):
    c = _pages(len(lens), width, ps, 128)
    free = [100 - i for i in range(max(left, 1) + 3)]
    _check_reserve(c, ps, lens, counts, free, left, tokens)


@pytest.mark.parametrize("seqs,most,left", [(511, 9, 10 ** 6), (512, 40, 700), (513, 300, 10 ** 6), (1500, 7, 900),
                                            (2, 20000, 10 ** 6), (40, 1500, 2000), (5, 60000, 10 ** 6), (600, 400, 5000),
                                            (9, 30000, 9000)])
def test_reserve_and_release_many(seqs, most, left):
    """More sequences than a block sums at once, more writes than a block makes, stacks that run short."""
    g = torch.Generator().manual_seed(seqs)
    ps, width = 16, 2 + 2 * most // 16
    draw = lambda hi: torch.randint(0, hi, (seqs,), generator=g).tolist()
    lens, counts = draw(most), draw(most + 1)
    pool = min(left, seqs * width)
    free = torch.randperm(pool, generator=g).tolist()
    table = torch.randint(0, 50, (seqs, width), generator=g).int().cuda()
    c = _pages(seqs, width, ps, 64, table)
    got, f, n = _check_reserve(c, ps, lens, counts, free, pool, sum(counts) + 3)
    now, keep = got[1].tolist(), [x + y // 2 for x, y in zip(lens, counts)]
    want = _release_ref(c.table.tolist(), ps, now, keep, f.tolist(), n.item())
    sv.kv_release(c, got[1], _i32(keep), f, n)
    assert (c.table.tolist(), f.tolist(), n.tolist()) == (want[0], want[1], [want[2]])


@pytest.mark.parametrize("ps,width,lens,keep,stack,left", [
    (16, 4, [64], [0], 4, 0),
    (16, 4, [64, 33, 10], [17, 32, 10], 9, 3),
    (16, 4, [64, 64], [0, 0], 5, 1),                         # more than the stack holds
    (16, 4, [64, 64], [1, 0], 8, -7),
    (16, 4, [64], [3], 8, 99),                               # a count past the stack: full
    (32, 3, [500, -3, 96], [-5, 4, 200], 9, 0),              # past the table, no length, kept past it
])
def test_release(ps, width, lens, keep, stack, left):
    c = _pages(len(lens), width, ps, 64, torch.arange(len(lens) * width, device="cuda").int().view(-1, width))
    free = list(range(50, 50 + stack))
    want = _release_ref(c.table.tolist(), ps, lens, keep, free, left)
    f, n = _i32(free), _i32([left])
    sv.kv_release(c, _i32(lens), _i32(keep), f, n)
    assert (c.table.tolist(), f.tolist(), n.tolist()) == (want[0], want[1], [want[2]])


def test_pages_without_a_stack():
    """A stack of no entries: what needs no page is served, what does gets nothing, dropped pages are lost."""
    c = _pages(2, 4, 16, 64, torch.arange(8, device="cuda").int().view(2, 4))
    free, n = torch.empty(0, dtype=torch.int32, device="cuda"), _i32([5])
    cu, lens, seq, pos, lacking = sv.kv_reserve(c, _i32([3, 15]), _i32([4, 2]), free, n, 9)
    assert (cu.tolist(), lens.tolist(), lacking.tolist(), n.tolist()) == ([0, 4, 4], [7, 15], [1], [0])
    assert seq.tolist() == [0] * 4 + [-1] * 5 and pos.tolist() == [3, 4, 5, 6] + [-1] * 5
    sv.kv_release(c, _i32([64, 64]), _i32([0, 17]), free, n)
    assert c.table.tolist() == [[-1] * 4, [4, 5, -1, -1]] and n.tolist() == [0]


def test_no_tokens():
    """A step of nothing writes nothing and returns what has no rows."""
    c = _pages(2, 4, 16, 8)
    x = torch.zeros(0, 6, 32, dtype=torch.bfloat16, device="cuda")
    none, plan = torch.empty(0, dtype=torch.int32, device="cuda"), sv.rope_plan(32, 10000.0)
    gain = torch.ones(32, device="cuda")
    assert sv.qkv_append(c, x[:, :4], x[:, 4:5], x[:, 5:], none, none, plan, gain, gain).shape == (0, 4, 32)
    assert sv.rope_norm_rows(x, none, plan, gain).shape == (0, 6, 32)
    zero, n = _i32([0, 0]), _i32([3])
    cu, lens, seq, pos, lacking = sv.kv_reserve(c, zero, zero, _i32([1, 2, 3]), n, 0)
    assert cu.tolist() == [0, 0, 0] and lens.tolist() == [0, 0] and seq.numel() == pos.numel() == 0
    q = torch.zeros(0, 4, 32, dtype=torch.bfloat16, device="cuda")
    for out, lse in (sv.attn_paged(q, c, cu, lens, window=5, sinks=1), sv.attn_shared(q, c, cu, lens, _i32([3])),
                     sv.attn_prompt(q, q[:, :1], q[:, :1], cu, window=5)):
        assert out.shape == (0, 4, 32) and lse.shape == (0, 4)


def test_pages_replayed_and_strided():
    """A captured step, replayed: the stack, the table and the lengths move on from where they are."""
    ps, seqs, width = 16, 3, 8
    wide = torch.full((seqs, width + 5), -7, dtype=torch.int32, device="cuda")
    table = wide[:, 2:2 + width]
    table.fill_(-1)
    c = _pages(seqs, width, ps, 64, table)
    free, n = torch.arange(40, device="cuda").int(), _i32([40])
    lens, counts, keep = _i32([0, 15, 31]), _i32([5, 6, 7]), _i32([0, 0, 0])
    had = (lens + ps - 1) // ps
    for b in range(seqs):
        table[b, :had[b]] = torch.arange(50 + 2 * b, 50 + 2 * b + int(had[b]), device="cuda").int()
    start = wide.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        state = [x.clone() for x in (wide, free, n, lens)]
        for _ in range(2):                                   # (allocations settle before the capture)
            r = sv.kv_reserve(c, lens, counts, free, n, 20)
            sv.kv_release(c, r[1], lens + 1, free, n)
        for x, y in zip((wide, free, n, lens), state):
            x.copy_(y)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = sv.kv_reserve(c, lens, counts, free, n, 20)
        keep.copy_(lens + 2)
        sv.kv_release(c, r[1], keep, free, n)
        lens.copy_(keep)
    t, f, left, ln = start[:, 2:2 + width].tolist(), list(range(40)), 40, [0, 15, 31]
    for _ in range(6):
        graph.replay()
        t, left, cu, now, seq, pos, lacking = _reserve_ref(t, ps, ln, [5, 6, 7], f, left, 20)
        ln = [x + 2 for x in ln]
        t, f, left = _release_ref(t, ps, now, ln, f, left)
        assert (table.tolist(), free.tolist(), n.tolist(), lens.tolist()) == (t, f, [left], ln)
        assert [x.tolist() for x in r] == [cu, now, seq, pos, [lacking]]
    assert (wide[:, :2] == -7).all() and (wide[:, 2 + width:] == -7).all()


# ------------------------------------------------------- norms and rotation
def _norm_ref(x, gain, eps):
    x = x.to(F64)
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * gain.to(F64)


def _normed(x, pos, gain, eps, rot, inter, theta=500000.0):
    """(64-bit norm and rotation, the bound of fp32's errors before the output's rounding)."""
    d = x.shape[-1]
    y = _norm_ref(x, gain, eps) if gain is not None else x.to(F64)
    n = (d / 2 + 10) * 2.0 ** -24 if gain is not None else 0.0
    if not rot:
        return y, y.abs() * n
    ref, size = _rope_ref(y, pos, _freqs(rot, theta), inter)
    far = pos.to(F64).abs()[:, None, None] * 2.0 ** -50
    return ref, size * (8 * 2.0 ** -23 + n + far)


NORM = [  # tokens, heads, hd, rot, interleaved, in, out, gain of each head, first position
    (6, 40, 128, 128, False, torch.float32, torch.bfloat16, True, 511),
    (1, 1, 64, 64, False, torch.bfloat16, torch.bfloat16, False, 0),
    (33, 10, 64, 32, True, torch.bfloat16, torch.float32, True, 900000),
    (700, 40, 64, 16, False, torch.bfloat16, torch.bfloat16, True, 70000),
    (17, 3, 128, 128, True, torch.float32, torch.float32, False, 3),
    (300, 9, 32, 32, False, torch.float32, torch.bfloat16, True, 5),
    (257, 33, 256, 64, False, torch.bfloat16, torch.bfloat16, False, 1 << 20),
    (5, 7, 96, 96, False, torch.bfloat16, torch.bfloat16, True, 77),       # no power of two: element by element
    (5, 7, 32, 6, False, torch.float32, torch.bfloat16, False, 2 ** 31 - 10),
    (4, 2, 512, 256, True, torch.float32, torch.float32, True, 9),
    (3, 5, 2, 2, False, torch.float32, torch.float32, True, 9),
]


@pytest.mark.parametrize("t,h,hd,rot,inter,tin,tout,each,first", NORM)
def test_rope_norm_rows(t, h, hd, rot, inter, tin, tout, each, first):
    g = _gen(t + hd)
    x = (_randn(g, t, h + 2, hd) * torch.exp(2 * _randn(g, t, h + 2, 1))).to(tin)[:, 1:h + 1]
    pos = (first + torch.arange(t, device="cuda")).int()
    gain = torch.exp(0.3 * _randn(g, *((h, hd) if each else (hd,))))
    plan = sv.rope_plan(rot, 500000.0, interleaved=inter)
    for eps in (1e-5, 0.5):
        y = sv.rope_norm_rows(x, pos, plan, gain, eps=eps, dtype=tout)
        ref, tol = _normed(x, pos, gain, eps, rot, inter)
        err = (y.to(F64) - ref).abs()
        tol = tol + ref.abs() * HALF[tout] + 1e-37
        assert (err <= tol).all(), float((err / tol).max())


def test_rope_norm_rows_odd_rows():
    """Unaligned rows, in place, rows of zeros, of infinities and of NaN, squares past fp32, no tokens."""
    g = _gen(3)
    plan, pos = sv.rope_plan(64, 10000.0), torch.arange(9, device="cuda").int()
    gain = torch.exp(_randn(g, 64))
    x = _randn(g, 9, 4, 64)
    x[1], x[2, 1, 5], x[3, 2, 7], x[4, 3] = 0, float("inf"), float("nan"), 1e25
    y = sv.rope_norm_rows(x, pos, plan, gain)
    ok = torch.ones(9, 4, dtype=torch.bool, device="cuda")
    ok[2, 1] = ok[3, 2] = ok[4, 3] = False
    ref, tol = _normed(x, pos, gain, 1e-5, 64, False, 10000.0)
    assert ((y.to(F64) - ref).abs() <= tol + ref.abs() * 2.0 ** -24 + 1e-37)[ok].all()
    assert (y[1] == 0).all() and y[2, 1].isnan().any() and y[3, 2].isnan().all() and (y[4, 3] == 0).all()
    z = x.clone()
    assert sv.rope_norm_rows(z, pos, plan, gain, out=z) is z and torch.equal(z.nan_to_num(7.0), y.nan_to_num(7.0))
    odd = torch.empty(9 * 4 * 65 + 1, device="cuda")[1:].view(9, 4, 65)[..., :64]       # no 16-byte alignment
    odd.copy_(x)
    w = sv.rope_norm_rows(odd, pos, plan, gain)
    assert ((w.to(F64) - ref).abs() <= tol + ref.abs() * 2.0 ** -24 + 1e-37)[ok].all()
    far = torch.empty(65, device="cuda")[1:]
    far.copy_(gain)
    assert torch.equal(sv.rope_norm_rows(x[:2], pos[:2], plan, far), sv.rope_norm_rows(odd[:2], pos[:2], plan, gain))
    assert sv.rope_norm_rows(x[:0], pos[:0], plan, gain).shape == (0, 4, 64)


QKV = [  # tokens, query heads, KV heads, hd, page, in, rot, interleaved, norms
    (6, 32, 8, 128, 16, torch.float32, 128, False, "qk"),
    (1, 8, 2, 64, 32, torch.bfloat16, 64, False, "qk"),
    (300, 32, 8, 64, 16, torch.bfloat16, 32, True, "qk"),
    (700, 7, 1, 128, 64, torch.bfloat16, 128, False, "q"),
    (65, 12, 4, 32, 256, torch.float32, 32, False, "k"),
    (40, 4, 4, 64, 16, torch.bfloat16, 0, False, "qk"),
    (50, 16, 2, 128, 16, torch.float32, 128, False, ""),
    (33, 5, 5, 64, 16, torch.float32, 24, False, "qk"),       # a rotated part of no whole chunks
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,hq,hk,hd,ps,tin,rot,inter,norms", QKV)
def test_qkv_append(n, hq, hk, hd, ps, tin, rot, inter, norms, dtype):
    g = _gen(n + hd)
    seqs = 3
    width = -(-n // ps) + 1
    table = torch.randperm(seqs * width + 2, generator=g, device="cuda")[:seqs * width].int().view(seqs, width)
    cache = sv.KVCache.empty(seqs * width + 2, ps, hk, hd, table.contiguous(), dtype)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x11)
    x = _randn(g, n, hq + 2 * hk, hd).to(tin)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    seq = torch.randint(0, seqs, (n,), generator=g, device="cuda").int()
    pos = torch.randperm(n, generator=g, device="cuda").int() + 3
    if n > 4:
        seq[1], pos[2], pos[3] = -1, -9, width * ps            # not written
    plan = sv.rope_plan(rot, 500000.0, interleaved=inter) if rot else None
    gq, gk = (torch.exp(0.3 * _randn(g, hd)) if c in norms else None for c in "qk")
    before = [t.view(torch.uint8).clone() for t in (cache.k, cache.v)]
    out = sv.qkv_append(cache, q, k, v, seq, pos, plan, gq, gk)
    ref, tol = _normed(q, pos, gq, 1e-5, rot, inter)
    assert out.dtype is torch.bfloat16
    assert ((out.to(F64) - ref).abs() <= tol + ref.abs() * 2.0 ** -8 + 1e-37).all()
    kk, vv = sv.kv_gather(cache, seq, pos, dtype=torch.float32)
    live = torch.ones(n, dtype=torch.bool, device="cuda")
    if n > 4:
        live[1:4] = False
    assert (kk[~live] == 0).all()
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -4
    for got, (ref, tol) in ((kk, _normed(k, pos, gk, 1e-5, rot, inter)), (vv, (v.to(F64), 0.0))):
        top = ref.abs().amax(-1, keepdim=True)
        small = top * 2.0 ** -17 if dtype == "e4m3" else 0.0   # half of the smallest step, 2^-10, of at least 224
        err = (got.to(F64) - ref).abs()
        assert (err <= tol + ref.abs() * half + small + 1e-37)[live].all()
    if gk is None and gq is None:                              # the same bits as the calls that it stands for
        other = sv.KVCache.empty(cache.k.shape[0], ps, hk, hd, cache.table, dtype)
        for t in (other.k, other.v):
            t.view(torch.uint8).fill_(0x11)
        sv.kv_append(other, k, v, seq, pos, plan)
        for a, b in ((cache.k, other.k), (cache.v, other.v)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(out, sv.rope_rows(q, pos, plan, dtype=torch.bfloat16))
    # nothing but the rows' slots
    mask = torch.ones(cache.k.shape[0], ps, dtype=torch.bool, device="cuda")
    mask[cache.table.long()[seq[live].long(), (pos[live] // ps).long()], (pos[live] % ps).long()] = False
    for t, old in zip((cache.k, cache.v), before):
        now = t.view(torch.uint8).view(t.shape[0], hk, ps, -1).transpose(1, 2)[mask]
        assert torch.equal(now, old.view(t.shape[0], hk, ps, -1).transpose(1, 2)[mask])


def test_qkv_append_in_place_and_streams():
    """q_out over q, calls on a raw stream and replayed from a graph: the same bits."""
    g = _gen(5)
    table = torch.arange(8, device="cuda").int().view(2, 4)
    mk = lambda: sv.KVCache.empty(8, 16, 2, 64, table, "bf16")
    x, seq, pos = _randn(g, 20, 12, 64).bfloat16(), _i32([0, 1] * 10), _i32([i // 2 for i in range(20)])
    plan, gain = sv.rope_plan(64, 10000.0), torch.exp(_randn(g, 64))
    call = lambda c, y, **kw: sv.qkv_append(c, y[:, :8], y[:, 8:10], y[:, 10:], seq, pos, plan, gain, gain, **kw)
    c = mk()
    ref = call(c, x)
    c2, y = mk(), x.clone()
    assert call(c2, y, out=y[:, :8]) is not None
    assert torch.equal(y[:, :8], ref) and torch.equal(y[:, 8:], x[:, 8:]) and torch.equal(c2.k, c.k)
    side = torch.cuda.Stream()
    c3 = mk()
    side.wait_stream(torch.cuda.current_stream())
    got = call(c3, x, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, ref) and torch.equal(c3.k, c.k) and torch.equal(c3.v, c.v)
    graph, c4 = torch.cuda.CUDAGraph(), mk()
    with torch.cuda.graph(graph):
        got = call(c4, x)
    graph.replay()
    assert torch.equal(got, ref) and torch.equal(c4.k, c.k)
    with pytest.raises(sv.SpecError):
        sv.qkv_append(c, x[:, :8], x[:, 8:10], x[:, 10:], seq, pos, plan, gain[:32], gain)
    with pytest.raises(sv.SpecError):
        sv.qkv_append(c, x[:, :8].float(), x[:, 8:10], x[:, 10:], seq, pos, plan, gain, gain)


# ------------------------------------------------------- results' allocation
@pytest.mark.parametrize("shape", [(0,), (7,), (5, 3), (0, 3), (4, 0), (6, 5, 64), (0, 5, 64), (6, 0, 64), (6, 5, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.int32, torch.uint8])
def test_results_are_packed_like_torchs_own(shape, dtype, monkeypatch):
    sv._torch()
    fast = sv._empty(0, torch.Size(shape), dtype)
    monkeypatch.setattr(sv, "_packed", None)       # torch without the short call
    slow = sv._empty(0, torch.Size(shape), dtype)
    for t in (fast, slow):
        assert t.shape == torch.Size(shape) and t.dtype == dtype and t.device == torch.device("cuda", 0)
        assert t.stride() == torch.empty(shape, dtype=dtype).stride()
    assert not fast.requires_grad


def test_calls_without_the_short_allocation(monkeypatch):
    x, pos = _randn(_gen(5), 9, 4, 64), _i32(list(range(9)))
    plan = sv.rope_plan(64, 10000.0)
    with_it = sv.rope_rows(x, pos, plan)
    monkeypatch.setattr(sv, "_packed", None)
    assert torch.equal(sv.rope_rows(x, pos, plan), with_it)


# ------------------------------------------------------- cleared entries
def _release_sound_ref(table, ps, lens, keep, free, left):
    """_release_ref over rows some of whose entries are cleared (negative) already: those are no pages."""
    table, free = [list(r) for r in table], list(free)
    left = max(0, min(left, len(free)))
    for b, (n, k) in enumerate(zip(lens, keep)):
        n = min(max(0, n), len(table[b]) * ps)
        k = min(max(0, k), n)
        for j in range(-(-k // ps), -(-n // ps)):
            if table[b][j] >= 0 and left < len(free):
                free[left] = table[b][j]
                left += 1
            table[b][j] = -1
    return table, free, left


@pytest.mark.parametrize("seqs,width,cleared,stack,left", [
    (1, 4, 0.5, 4, 0), (3, 40, 0.3, 200, 7), (3, 40, 1.0, 200, 7), (3, 400, 0.01, 2000, 100), (7, 300, 0.5, 900, 0),
    (1, 30000, 0.5, 40000, 17), (5, 9000, 0.002, 50000, 0), (9, 7000, 0.9, 3000, 1000), (513, 20, 0.2, 20000, 5),
    (1200, 9, 0.5, 4000, 3990), (1600, 40, 0.4, 70000, 1), (2, 8000, 0.0, 20000, 3),
])
def test_release_of_cleared_entries(seqs, width, cleared, stack, left):
    """What a program cleared itself, as the pages in front of a window, is not taken for a page; the others
    lie in the stack in order, in rows of one and of many blocks' work, in stacks with room and without."""
    g = torch.Generator().manual_seed(seqs + width)
    ps = 16
    table = torch.randperm(seqs * width, generator=g).int().view(seqs, width)
    gone = torch.rand(seqs, width, generator=g) < cleared
    table[gone] = torch.randint(-2 ** 31, 0, (int(gone.sum()),), generator=g).int()
    lens = torch.randint(width * ps // 2, width * ps + 40, (seqs,), generator=g).tolist()
    keep = [x if i % 5 == 3 else int(x * (i % 4) / 5) for i, x in enumerate(lens)]
    want = _release_sound_ref(table.tolist(), ps, lens, keep, list(range(stack)), left)
    c = _pages(seqs, width, ps, 64, table.cuda())
    f, n = _i32(list(range(stack))), _i32([left])
    sv.kv_release(c, _i32(lens), _i32(keep), f, n)
    assert n.tolist() == [want[2]] and f.tolist() == want[1] and c.table.tolist() == want[0]
    sv.kv_release(c, _i32(lens), _i32(keep), f, n)             # again: nothing is left to give back
    assert n.tolist() == [want[2]] and f.tolist() == want[1] and c.table.tolist() == want[0]


def test_pages_left_behind_by_a_window():
    """A program clears the entries in front of its window and gives their pages back itself; the sequence's
    release then leaves every page in the stack once, and what is reserved from it holds rows."""
    ps, pages = 16, 24
    table = torch.full((2, 64), -1, dtype=torch.int32, device="cuda")
    c = sv.KVCache.empty(pages, ps, 1, 32, table)
    free, n = torch.arange(pages, device="cuda").int(), _i32([pages])
    _, lens, *_ = sv.kv_reserve(c, _i32([0, 0]), _i32([200, 150]), free, n, 400)
    behind = table[0, :7].tolist()                             # positions in front of a window of 80
    left = n.item()
    free[left:left + 7] = _i32(behind)
    n.fill_(left + 7)
    table[0, :7] = -1
    sv.kv_release(c, lens, _i32([0, 0]), free, n)
    assert n.item() == pages and sorted(free.tolist()) == list(range(pages)) and (table == -1).all()
    cu, lens, seq, pos, lacking = sv.kv_reserve(c, _i32([0, 0]), _i32([190, 190]), free, n, 380)
    assert lacking.item() == 0 and n.item() == 0
    x = _randn(_gen(1), 380, 1, 32).bfloat16()
    sv.kv_append(c, x, x, seq, pos)
    k, v = sv.kv_gather(c, seq, pos)
    assert torch.equal(k, x) and torch.equal(v, x)


def test_release_of_few_and_many_by_turns():
    """Few dropped entries, then many, and again: what one block placed alone moves the others' places."""
    g = torch.Generator().manual_seed(11)
    ps, seqs, width, stack = 16, 2100, 30, 70000
    table = torch.randperm(seqs * width, generator=g).int().view(seqs, width)
    table[torch.rand(seqs, width, generator=g) < 0.3] = -1
    lens = [width * ps] * seqs
    drops = lambda b: b // 512 % 2 == 1 or b % 512 in (7, 100, 101)
    keep = [17 * (b % 20) if drops(b) else lens[b] for b in range(seqs)]
    want = _release_sound_ref(table.tolist(), ps, lens, keep, list(range(stack)), 40)
    c = _pages(seqs, width, ps, 64, table.cuda())
    f, n = _i32(list(range(stack))), _i32([40])
    sv.kv_release(c, _i32(lens), _i32(keep), f, n)
    assert n.tolist() == [want[2]] and f.tolist() == want[1] and c.table.tolist() == want[0]


@pytest.mark.parametrize("det", [False, True])
def test_results_under_deterministic_algorithms(det):
    """Torch fills what it allocates while deterministic algorithms are asked for: so with the results' rows
    that a call leaves as they were."""
    c = _pages(1, 4, 16, 8, _i32([[0, 1, 2, 3]]))
    q = torch.ones(5, 4, 32, dtype=torch.bfloat16, device="cuda")
    on, fill = torch.are_deterministic_algorithms_enabled(), torch.utils.deterministic.fill_uninitialized_memory
    try:
        torch.use_deterministic_algorithms(True)
        torch.utils.deterministic.fill_uninitialized_memory = det
        for _ in range(3):
            junk = [torch.full((5, 4, 32), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((5, 4), 3.0, device="cuda")]
            del junk                                     # (what the memory holds when the results take it)
            out, lse = sv.attn_paged(q, c, _i32([0, 2]), _i32([9]))
            assert torch.isfinite(out[:2].float()).all() and torch.isfinite(lse[:2]).all()
            if det:
                assert out[2:].isnan().all() and lse[2:].isnan().all()
    finally:
        torch.use_deterministic_algorithms(on)
        torch.utils.deterministic.fill_uninitialized_memory = fill


def test_results_under_modes():
    """Dispatch and function modes and profilers see the results' allocation, and a result made in inference mode is one."""
    from torch.overrides import TorchFunctionMode
    from torch.utils._python_dispatch import TorchDispatchMode
    seen = []

    class Dispatch(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            seen.append(str(func))
            return func(*args, **(kwargs or {}))

    class Function(TorchFunctionMode):
        def __torch_function__(self, func, types, args=(), kwargs=None):
            seen.append(getattr(func, "__name__", ""))
            return func(*args, **(kwargs or {}))

    x, pos, plan = _randn(_gen(5), 9, 4, 64), _i32(list(range(9))), sv.rope_plan(64, 10000.0)
    ref = sv.rope_rows(x, pos, plan)
    for mode in (Dispatch, Function):
        seen.clear()
        with mode():
            y = sv.rope_rows(x, pos, plan)
        assert any("empty" in s for s in seen), mode
        assert torch.equal(y, ref)
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as prof:
        sv.rope_rows(x, pos, plan)
    assert any(e.key == "aten::empty" for e in prof.key_averages())
    with torch.inference_mode():
        y = sv.rope_rows(x, pos, plan)
    assert y.is_inference() and not ref.is_inference() and torch.equal(y, ref)
