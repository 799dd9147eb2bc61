"""Argument checks of the paged-cache operators, none of which needs a GPU:
bad descriptions are refused with the documented codes before any device work,
calls without tokens succeed, and the rotary plan is plain arithmetic."""
import ctypes
import math

import pytest
import torch

import speculative_decoding_verification_step_gb300 as sv

P = 0x10000        # a 16-byte aligned address that no call may touch


@pytest.fixture(scope="module")
def L():
    sv.build()
    return sv.lib()


def _cache(**kw):
    a = dict(k=P, v=P, k_scale=P, v_scale=P, dtype=sv.SPEC_DTYPE_BF16, pages=4, page_size=16, n_kv_heads=2,
             head_dim=64, page_stride=0, scale_page_stride=0, table=P, table_stride=0, seqs=2, max_pages=2)
    a.update(kw)
    return sv.KVCacheDesc(**a)


BAD_CACHE = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(table=None), -1), (dict(dtype=0), -1), (dict(dtype=2), -1),
    (dict(dtype=3, k_scale=None), -1), (dict(head_dim=48), -3), (dict(head_dim=256), -3), (dict(page_size=24), -3),
    (dict(page_size=8), -3), (dict(page_size=512), -3), (dict(pages=0), -1), (dict(n_kv_heads=0), -1),
    (dict(seqs=0), -1), (dict(max_pages=0), -1), (dict(k=P + 8), -1), (dict(page_stride=100), -1),
    (dict(page_stride=2 * 16 * 64 + 4), -1), (dict(table_stride=1), -1), (dict(dtype=3, v_scale=P + 1), -1),
    (dict(dtype=3, scale_page_stride=33), -1), (dict(max_pages=2 ** 27, page_size=256), -1),
]


@pytest.mark.parametrize("change,code", BAD_CACHE)
def test_cache_refusals(L, change, code):
    c = ctypes.byref(_cache(**change))
    assert L.spec_kv_append(c, P, 128, 64, P, 128, 64, 1, P, P, 1, None, None) == code
    assert L.spec_kv_gather(c, P, P, 1, P, P, 1, None) == code
    assert L.spec_attn_paged(c, P, 256, 64, P, P, 1, 1, 4, 0.0, P, 256, 64, None, None, 0, None) == code
    assert L.spec_last_error(None)


def test_null_cache(L):
    assert L.spec_kv_append(None, P, 128, 64, P, 128, 64, 1, P, P, 1, None, None) == -1
    assert L.spec_kv_gather(None, P, P, 1, P, P, 1, None) == -1
    assert L.spec_attn_paged(None, P, 256, 64, P, P, 1, 1, 4, 0.0, P, 256, 64, None, None, 0, None) == -1
    assert L.spec_attn_paged_workspace(None, 1, 1, 4) == 0


def test_row_refusals(L):
    c = ctypes.byref(_cache())
    app = lambda **k: L.spec_kv_append(c, k.get("k", P), 128, 64, P, 128, 64, k.get("dtype", 1), k.get("seq", P), P,
                                       k.get("n", 1), k.get("plan"), None)
    assert app(k=None) == app(seq=None) == app(dtype=3) == app(n=-1) == -1
    assert app(n=0) == 0                                   # nothing to do: no device work
    plan = sv.rope_plan(128, 10000.0)                      # larger than the head
    assert app(plan=plan._ref) == -1
    assert L.spec_kv_gather(c, P, P, 1, P + 2, P, 1, None) == -1
    assert L.spec_kv_gather(c, None, P, 1, P, P, 1, None) == -1
    assert L.spec_kv_gather(c, P, P, 1, P, P, 3, None) == -1
    assert L.spec_kv_gather(c, P, P, 0, P, P, 1, None) == 0
    assert L.spec_kv_gather(c, P, P, 5, None, None, 1, None) == 0
    plan = sv.rope_plan(32, 10000.0)
    rope = lambda **k: L.spec_rope_rows(k.get("x", P), k.get("xd", 1), 256, 64, k.get("y", 2 * P), k.get("yd", 1),
                                        k.get("ys", 256), 64, k.get("pos", P), k.get("n", 1), k.get("h", 4),
                                        k.get("hd", 64), k.get("plan", plan._ref), 0, None)
    assert rope(x=None) == rope(y=None) == rope(pos=None) == rope(xd=3) == rope(yd=2) == rope(plan=None) == -1
    assert rope(n=-1) == rope(h=0) == rope(hd=16) == -1    # rot_dim 32 does not fit a head of 16
    assert rope(y=P, yd=0) == rope(y=P, ys=512) == -1      # in place with another dtype or stride
    assert rope(hd=65) == -3
    assert rope(n=0) == 0


def test_attention_refusals(L):
    c = ctypes.byref(_cache())
    att = lambda **k: L.spec_attn_paged(c, k.get("q", P), k.get("qs", 256), 64, k.get("cu", P), k.get("lens", P),
                                        k.get("n", 1), k.get("m", 1), k.get("h", 4), k.get("scale", 0.0),
                                        k.get("out", P), 256, k.get("oh", 64), None, k.get("ws"), k.get("wb", 0), None)
    assert att(q=None) == att(cu=None) == att(lens=None) == att(out=None) == -1
    assert att(q=P + 2) == att(qs=260) == att(oh=4) == att(n=-1) == att(m=-1) == -1
    assert att(ws=P + 4, wb=64) == att(ws=P, wb=-1) == -1
    assert att(scale=math.nan) == att(scale=math.inf) == att(scale=-1.0) == -1
    assert att(h=3) == att(h=0) == -3
    assert att(n=0) == att(m=0) == 0
    pr = lambda **k: L.spec_attn_prompt(k.get("q", P), 256, 64, k.get("k", P), 128, 64, k.get("v", P), k.get("vs", 128),
                                        64, k.get("cu", P), k.get("seqs", 1), k.get("n", 1), 1, k.get("h", 4), 2,
                                        k.get("hd", 64), 0.0, P, 256, 64, None, None)
    assert pr(q=None) == pr(k=None) == pr(v=None) == pr(cu=None) == pr(seqs=0) == pr(k=P + 4) == pr(vs=132) == -1
    assert pr(h=3) == pr(hd=96) == pr(hd=256) == -3
    assert pr(n=0) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_no_cpu_fallback(L):
    c = ctypes.byref(_cache())
    assert L.spec_attn_paged(c, P, 256, 64, P, P, 1, 1, 4, 0.0, P, 256, 64, None, None, 0, None) == -5
    assert L.spec_kv_gather(c, P, P, 1, P, P, 1, None) == -5


@pytest.mark.parametrize("kw", [dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=258), dict(theta=0.0), dict(theta=math.inf),
                                dict(scaling="linear", factor=0.0), dict(scaling="ntk", rot_dim=2),
                                dict(scaling="parts"), dict(scaling="parts", orig_ctx=10.0, low=4.0, high=4.0),
                                dict(mscale=-1.0), dict(scaling="other")])
def test_plan_refusals(L, kw):
    a = dict(rot_dim=64, theta=10000.0)
    a.update(kw)
    with pytest.raises(sv.SpecError):
        sv.rope_plan(a.pop("rot_dim"), a.pop("theta"), **a)


def test_plan_values(L):
    for scaling, more in (("plain", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=4.0)),
                          ("parts", dict(factor=8.0, orig_ctx=8192.0, low=1.0, high=4.0))):
        rot, theta = 64, 500000.0
        p = sv.rope_plan(rot, theta, scaling=scaling, mscale=0.0, **more)
        assert p.rot_dim == rot and p.mscale == 1.0
        base = theta * 4.0 ** (rot / (rot - 2)) if scaling == "ntk" else theta
        for i in range(rot // 2):
            f = base ** (-2.0 * i / rot)
            if scaling == "linear":
                f /= 4.0
            if scaling == "parts":
                keep = min(1.0, max(0.0, (8192.0 * f / (2 * math.pi) - 1.0) / 3.0))
                f *= keep + (1 - keep) / 8.0
            # two libraries' pow, a product and a quotient: a few units of the last place; the fraction
            # of a turn is rounded to a multiple of 2^-64, half of that off: pi 2^-64 radians
            assert abs(p.turn[i] / 2.0 ** 64 * 2 * math.pi - f) <= 8 * 2.0 ** -52 * f + math.pi * 2.0 ** -64


def test_binding_refusals(L):
    """Tensors that the calls cannot read are refused by name before the library is called."""
    x = torch.zeros(2, 2, 64)
    plan = sv.rope_plan(64, 10000.0)
    with pytest.raises(sv.SpecError):
        sv.rope_rows(x, torch.zeros(2, dtype=torch.int32), plan)           # not on a GPU
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(1, 4, dtype=torch.int32)
    for bad in (dict(k=k.half(), v=k.half()), dict(k=k, v=k[:3]), dict(k=k, v=k, k_scale=k), dict(k=k, v=k),
                dict(k=k.to(torch.float8_e4m3fn), v=k.to(torch.float8_e4m3fn)),
                dict(k=k.transpose(1, 2), v=k.transpose(1, 2))):
        with pytest.raises(sv.SpecError):
            sv.KVCache(bad["k"], bad["v"], table, bad.get("k_scale"))
    with pytest.raises(sv.SpecError):
        sv.KVCache(k, k, table.long())


def test_expanded_cache_refusals(L):
    """In the C structure a stride of 0 means packed: a tensor expanded along its first
    dimension would be read past its end, so it is refused."""
    page = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)
    codes, scale = page.to(torch.float8_e4m3fn), torch.zeros(1, 2, 16, dtype=torch.uint8)
    pool, pool8, scales = (x.repeat(4, *[1] * (x.dim() - 1)) for x in (page, codes.view(torch.uint8), scale))
    pool8 = pool8.view(torch.float8_e4m3fn)
    row, table = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(3, 4, dtype=torch.int32)
    wide = lambda x, n=4: x.expand(n, *x.shape[1:])
    for args in ((pool, pool, wide(row, 3)), (wide(page), wide(page), table), (pool, wide(page), table),
                 (pool8, pool8, table, wide(scale), wide(scale)), (pool8, pool8, table, scales, wide(scale)),
                 (wide(codes), wide(codes), table, scales, scales)):
        with pytest.raises(sv.SpecError, match="first stride of 0"):
            sv.KVCache(*args)


def test_timeout_hook_arguments(L):
    assert L.spec_inject_fault(None, sv.SPEC_FAULT_ATTN_TIMEOUT, -1) == -1
    assert L.spec_inject_fault(None, sv.SPEC_FAULT_ATTN_TIMEOUT, 2) == 0
    assert L.spec_inject_fault(None, sv.SPEC_FAULT_CLEAR, 0) == 0
    sv.inject_attention_timeout(0)


def test_gradients_are_not_dropped(L):
    """Nothing here records a backward pass: rows that require grad are refused by name while grad mode is on."""
    sv._torch()
    leaf = torch.zeros(2, 2, 64, dtype=torch.bfloat16, requires_grad=True)
    i, plan, cu = torch.zeros(2, dtype=torch.int32), sv.rope_plan(64, 10000.0), torch.tensor([0, 2], dtype=torch.int32)
    for t in (leaf, leaf * 1.0):
        for call in (lambda: sv.rope_rows(t, i, plan), lambda: sv.attn_prompt(t, t, t, cu), lambda: sv._rows3("k", t)):
            with pytest.raises(sv.SpecError, match="requires grad"):
                call()
            with torch.no_grad(), pytest.raises(sv.SpecError, match="a CUDA tensor"):   # taken as any other
                call()


def test_plan_mscale_past_fp32(L):
    """The factor is applied in fp32: one that is infinite there is refused."""
    with pytest.raises(sv.SpecError, match="mscale"):
        sv.rope_plan(64, 10000.0, mscale=1e39)
    assert sv.rope_plan(64, 10000.0, mscale=3e38).mscale > 2.9e38


def test_scale_past_fp32(L):
    """The scale is applied to exponents of two: one that is infinite there is refused."""
    c = ctypes.byref(_cache())
    for scale in (3e38, 2.4e38):
        assert L.spec_attn_paged(c, P, 256, 64, P, P, 1, 1, 4, scale, P, 256, 64, None, None, 0, None) == -1
        assert L.spec_attn_prompt(P, 256, 64, P, 128, 64, P, 128, 64, P, 1, 1, 1, 4, 2, 64, scale, P, 256, 64, None, None) == -1
