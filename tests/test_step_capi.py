"""Argument checks of the calls around a step (pages and index arrays, head norms
with the cache write), none of which needs a GPU: refused with the documented
codes before any device work; calls without tokens succeed."""
import ctypes
import math

import pytest
import torch

import speculative_decoding_verification_step_gb300 as sv
from test_paged_capi import BAD_CACHE, P, _cache


@pytest.fixture(scope="module")
def L():
    sv.build()
    return sv.lib()


def _reserve(L, c, **k):
    return L.spec_kv_reserve(c, k.get("lens", P), k.get("counts", P), k.get("free", P), k.get("left", P), k.get("cap", 4),
                             k.get("n", 8), k.get("cu", P), k.get("out", 2 * P), k.get("seq", P), k.get("pos", P),
                             k.get("lacking", P), None)


def _release(L, c, **k):
    return L.spec_kv_release(c, k.get("lens", P), k.get("keep", P), k.get("free", P), k.get("left", P), k.get("cap", 4), None)


def _qkv(L, c, **k):
    return L.spec_qkv_append(c, k.get("q", P), k.get("qs", 256), 64, k.get("k", P), 128, 64, k.get("v", P), 128, 64,
                             k.get("dtype", 1), k.get("seq", P), k.get("pos", P), k.get("n", 1), k.get("h", 4),
                             k.get("plan"), k.get("gq"), k.get("gk"), k.get("eps", 1e-5), k.get("out", 2 * P), 256, 64, None)


def _norm(L, **k):
    plan = k.get("plan", sv.rope_plan(32, 10000.0)._ref)
    return L.spec_rope_norm_rows(k.get("x", P), k.get("xd", 1), 256, 64, k.get("y", 2 * P), k.get("yd", 1),
                                 k.get("ys", 256), 64, k.get("pos", P), k.get("n", 1), k.get("h", 4), k.get("hd", 64),
                                 k.get("gain", P), k.get("gs", 0), k.get("eps", 1e-5), plan, None)


@pytest.mark.parametrize("change,code", BAD_CACHE)
def test_cache_refusals(L, change, code):
    c = ctypes.byref(_cache(**change))
    assert _reserve(L, c) == _release(L, c) == _qkv(L, c) == code
    assert L.spec_last_error(None)


def test_page_refusals(L):
    c = ctypes.byref(_cache())
    for name in ("lens", "counts", "free", "left", "cu", "out", "seq", "pos", "lacking"):
        assert _reserve(L, c, **{name: None}) == -1, name
    assert _reserve(L, c, cap=-1) == _reserve(L, c, n=-1) == _reserve(L, c, n=2 ** 31 - 1) == -1
    many = ctypes.byref(_cache(seqs=2 ** 30 + 1))
    assert _reserve(L, many) == _release(L, many) == -1
    assert _reserve(L, c, out=P) == -1                       # the new lengths over the old
    assert _reserve(L, None) == _release(L, None) == -1
    assert _reserve(L, c, free=None, cap=1) == _release(L, c, free=None, cap=1) == -1
    for name in ("lens", "keep", "free", "left"):
        assert _release(L, c, **{name: None}) == -1, name
    assert _release(L, c, cap=-1) == -1


def test_row_refusals(L):
    c = ctypes.byref(_cache())
    for name in ("q", "k", "v", "seq", "pos", "out"):
        assert _qkv(L, c, **{name: None}) == -1, name
    assert _qkv(L, c, n=-1) == _qkv(L, c, dtype=3) == _qkv(L, c, h=0) == _qkv(L, c, h=65536) == -1
    assert _qkv(L, c, eps=-1.0) == _qkv(L, c, eps=math.nan) == _qkv(L, c, eps=math.inf) == -1
    assert _qkv(L, c, plan=sv.rope_plan(128, 10000.0)._ref) == -1       # larger than the head
    assert _qkv(L, c, out=P, dtype=0) == _qkv(L, c, out=P, qs=512) == -1   # in place with another dtype or stride
    assert _qkv(L, c, n=0) == 0
    for name in ("x", "y", "pos", "gain", "plan"):
        assert _norm(L, **{name: None}) == -1, name
    assert _norm(L, n=-1) == _norm(L, h=0) == _norm(L, xd=3) == _norm(L, yd=2) == _norm(L, eps=-1e-9) == -1
    assert _norm(L, hd=16) == -1                             # rot_dim 32 does not fit
    assert _norm(L, hd=65) == _norm(L, hd=514) == _norm(L, hd=0) == -3
    assert _norm(L, y=P, yd=0) == _norm(L, y=P, ys=512) == -1
    assert _norm(L, n=0) == 0


def _window(L, c, **k):
    return L.spec_attn_paged_window(c, k.get("q", P), k.get("qs", 256), 64, k.get("cu", P), k.get("lens", P), k.get("n", 1),
                                    k.get("m", 1), k.get("h", 4), k.get("scale", 0.0), k.get("window", 8), k.get("sinks", 1),
                                    k.get("out", P), 256, 64, None, k.get("ws"), k.get("wb", 0), None)


def _prompt(L, **k):
    return L.spec_attn_prompt_window(k.get("q", P), 256, 64, k.get("k", P), 128, 64, k.get("v", P), k.get("vs", 128), 64,
                                     k.get("cu", P), k.get("seqs", 1), k.get("n", 1), 1, k.get("h", 4), 2, k.get("hd", 64),
                                     k.get("scale", 0.0), k.get("window", 8), k.get("sinks", 1), P, 256, 64, None, None)


def _shared(L, c, **k):
    return L.spec_attn_shared(c, k.get("q", P), k.get("qs", 256), 64, k.get("cu", P), k.get("lens", P), k.get("groups", P),
                              k.get("ng", 1), k.get("shared", P), k.get("n", 1), k.get("m", 1), k.get("h", 4),
                              k.get("scale", 0.0), k.get("out", P), 256, 64, None, k.get("ws"), k.get("wb", 0), None)


def test_attention_refusals(L):
    c = ctypes.byref(_cache())
    for call in (_window, _shared):
        for name in ("q", "cu", "lens", "out"):
            assert call(L, c, **{name: None}) == -1, name
        assert call(L, c, q=P + 2) == call(L, c, qs=260) == call(L, c, n=-1) == call(L, c, m=-1) == -1
        assert call(L, c, ws=P + 4, wb=64) == call(L, c, ws=P, wb=-1) == call(L, c, scale=math.nan) == -1
        assert call(L, c, scale=3e38) == call(L, c, scale=-1.0) == -1
        assert call(L, c, h=3) == call(L, c, h=0) == -3
        assert call(L, c, n=0) == call(L, c, m=0) == 0
        assert call(L, None) == -1
    for call in (lambda **k: _window(L, c, **k), lambda **k: _prompt(L, **k)):
        assert call(window=-1) == call(sinks=-1) == -1
    assert _shared(L, c, shared=None) == _shared(L, c, ng=0) == _shared(L, c, groups=None, ng=2) == -1
    for name in ("q", "k", "v", "cu"):
        assert _prompt(L, **{name: None}) == -1, name
    assert _prompt(L, seqs=0) == _prompt(L, vs=132) == -1 and _prompt(L, h=3) == _prompt(L, hd=96) == -3
    assert _prompt(L, n=0) == 0
    assert L.spec_attn_shared_workspace(None, 1, 1, 1, 4) == 0
    for bad in ((0, 1, 1, 4), (1, 0, 1, 4), (1, 1, 0, 4), (1, 1, 1, 3)):
        assert L.spec_attn_shared_workspace(c, *bad) == 0


@pytest.mark.parametrize("change,code", BAD_CACHE)
def test_attention_cache_refusals(L, change, code):
    c = ctypes.byref(_cache(**change))
    assert _window(L, c) == _shared(L, c) == code


def test_binding_refusals(L):
    sv._torch()
    plan, i, g = sv.rope_plan(64, 10000.0), torch.zeros(2, dtype=torch.int32), torch.ones(64)
    x = torch.zeros(2, 2, 64)
    with pytest.raises(sv.SpecError, match="CUDA"):
        sv.rope_norm_rows(x, i, plan, g)
    with pytest.raises(sv.SpecError, match="requires grad"):
        sv.rope_norm_rows(x.requires_grad_(), i, plan, g)
    for bad in (g[:32], g.double(), torch.ones(2, 2, 64)):
        with pytest.raises(sv.SpecError, match="gain"):
            sv._gain("gain", bad, (64,), -1)
    with pytest.raises(sv.SpecError, match="requires grad"):
        sv._gain("gain", torch.ones(64, requires_grad=True), (64,), -1)
    for bad in ((-1, 0), (0, -1), (-2 ** 40, 5)):
        with pytest.raises(sv.SpecError, match="negative"):
            sv._window(*bad)
    assert sv._window(2 ** 40, 7) == (0x7fffffff, 7)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_no_cpu_fallback(L):
    c = ctypes.byref(_cache())
    assert _reserve(L, c) == _release(L, c) == _qkv(L, c) == _norm(L) == -5
    assert _window(L, c) == _shared(L, c) == _prompt(L) == -5
