"""GB300 speculative-decoding verification step -- Python binding.

A thin ctypes layer over the C ABI in ``include/specverify.h``: it marshals
arguments and raises on error codes.  Every step of the path runs in the
CUDA library (``_lib/libspecverify.so``, built by ``build()``); there is no
CPU fallback, and using the binding without the built library raises.
Device memory (weights, logits) is passed as torch CUDA tensors, read by
pointer.
"""
import ctypes
import os

from ._build import LIB, build

__all__ = ["build", "lib", "SpecError", "SpecDecoder", "accept_rows", "sample_rows",
           "SPEC_DTYPE_F32", "SPEC_DTYPE_BF16", "SPEC_OPT_NO_GRAPH", "SPEC_OPT_TIMING",
           "SPEC_FLAG_RESID_ZERO", "SPEC_FLAG_ALL_ACCEPTED", "KVCache", "rope_plan", "rope_rows",
           "kv_append", "kv_gather", "attn_paged", "attn_prompt", "attn_shared", "rope_norm_rows", "qkv_append",
           "kv_reserve", "kv_release"]

SPEC_OK = 0
ERRORS = {-1: "SPEC_E_ARG", -2: "SPEC_E_VOCAB", -3: "SPEC_E_SHAPE", -4: "SPEC_E_CAPACITY",
          -5: "SPEC_E_CUDA", -6: "SPEC_E_OOM", -7: "SPEC_E_TIMEOUT", -8: "SPEC_E_STATE"}
SPEC_DTYPE_F32 = 0
SPEC_DTYPE_BF16 = 1
SPEC_DTYPE_Q4 = 2
SPEC_DTYPE_E4M3 = 3
SPEC_ROPE_MAX_DIM = 256
_ROPE_SCALING = {"plain": 0, "linear": 1, "ntk": 2, "parts": 3}
_DTYPES = {"f32": SPEC_DTYPE_F32, "bf16": SPEC_DTYPE_BF16, "q4": SPEC_DTYPE_Q4}
SPEC_MAX_BATCH = 64
SPEC_FLAG_RESID_ZERO = 0x1
SPEC_FLAG_ALL_ACCEPTED = 0x2
SPEC_OPT_NO_GRAPH = 0x1
SPEC_OPT_TIMING = 0x2
SPEC_OPT_PDL = 0x4
SPEC_OPT_NO_PERSIST = 0x8
SPEC_OPT_PHASE_TIMES = 0x10
SPEC_FAULT_CLEAR = 0
SPEC_FAULT_ALLOC = 1
SPEC_FAULT_WAIT_TIMEOUT = 2
SPEC_FAULT_ATTN_TIMEOUT = 3

_LAYER_FIELDS = ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "w_gate", "w_up", "w_down")


class LayerWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _LAYER_FIELDS]


class ModelDesc(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("d_model", ctypes.c_int), ("n_heads", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("ffn_dim", ctypes.c_int),
                ("vocab", ctypes.c_int), ("rope_theta", ctypes.c_float), ("rms_eps", ctypes.c_float),
                ("dtype", ctypes.c_int), ("embed", ctypes.c_void_p), ("final_norm", ctypes.c_void_p),
                ("lm_head", ctypes.c_void_p), ("layers", ctypes.POINTER(LayerWeights))]


class Opts(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("max_ctx", ctypes.c_int), ("temperature", ctypes.c_float),
                ("seed", ctypes.c_uint64), ("draft_mix_lambda", ctypes.c_float),
                ("cuda_stream", ctypes.c_void_p), ("flags", ctypes.c_int), ("draft_lookup", ctypes.c_int),
                ("draft_heads", ctypes.c_void_p)]


class Stats(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int64), ("ar_steps", ctypes.c_int64),
                ("tokens_emitted", ctypes.c_int64), ("drafts_accepted", ctypes.c_int64),
                ("accept_hist", ctypes.c_int64 * 17), ("context_len", ctypes.c_int32),
                ("kernels_per_step", ctypes.c_int32), ("kernels_per_ar_step", ctypes.c_int32),
                ("gemm_launches_per_verify", ctypes.c_int32),
                ("verify_weight_bytes", ctypes.c_double), ("draft_weight_bytes", ctypes.c_double),
                ("kv_bytes_per_token_target", ctypes.c_double),
                ("kv_bytes_per_token_draft", ctypes.c_double),
                ("timed_gemm_ms", ctypes.c_double), ("timed_gemm_bytes", ctypes.c_double),
                ("timed_gemm_launches", ctypes.c_int64)]

    def as_dict(self):
        d = {n: getattr(self, n) for n, _ in self._fields_}
        d["accept_hist"] = list(self.accept_hist)
        return d


class Profile(ctypes.Structure):
    _fields_ = [("draft_loop_ms", ctypes.c_double), ("verify_ms", ctypes.c_double),
                ("ar_ms", ctypes.c_double), ("iters", ctypes.c_int32),
                ("kernels_draft_loop", ctypes.c_int32), ("kernels_verify", ctypes.c_int32),
                ("kernels_ar", ctypes.c_int32), ("verify_forward_ms", ctypes.c_double),
                ("kernels_verify_forward", ctypes.c_int32)]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class KVCacheDesc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("dtype", ctypes.c_int), ("pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_stride", ctypes.c_int64), ("scale_page_stride", ctypes.c_int64),
                ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("seqs", ctypes.c_int),
                ("max_pages", ctypes.c_int)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("scaling", ctypes.c_int),
                ("theta", ctypes.c_double), ("factor", ctypes.c_double), ("orig_ctx", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("mscale", ctypes.c_double)]


class RopePlan(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("mscale", ctypes.c_float),
                ("reserved", ctypes.c_int), ("turn", ctypes.c_uint64 * (SPEC_ROPE_MAX_DIM // 2))]


_I32P = ctypes.POINTER(ctypes.c_int32)
_U32P = ctypes.POINTER(ctypes.c_uint32)
_F32P = ctypes.POINTER(ctypes.c_float)
_VP = ctypes.c_void_p
_INT = ctypes.c_int
_I64 = ctypes.c_int64

# name -> (restype, argtypes); every function declared in include/specverify.h
SIGNATURES = {
    "spec_init": (ctypes.c_int, [ctypes.POINTER(ModelDesc), ctypes.POINTER(ModelDesc), ctypes.c_int,
                                 ctypes.POINTER(Opts), ctypes.POINTER(_VP)]),
    "spec_free": (None, [_VP]),
    "spec_last_error": (ctypes.c_char_p, [_VP]),
    "spec_prefill": (ctypes.c_int, [_VP, _I32P, ctypes.c_int]),
    "spec_prefill_synthetic": (ctypes.c_int, [_VP, ctypes.c_int, ctypes.c_uint64]),
    "spec_seq_context": (ctypes.c_int, [_VP, ctypes.c_int, _I32P, _I32P]),
    "spec_step": (ctypes.c_int, [_VP, _I32P, _I32P, _U32P]),
    "spec_generate": (ctypes.c_int, [_VP, ctypes.c_int, _I32P, _I32P]),
    "spec_ar_step": (ctypes.c_int, [_VP, _I32P]),
    "spec_get_stats": (ctypes.c_int, [_VP, ctypes.POINTER(Stats)]),
    "spec_last_step_debug": (ctypes.c_int, [_VP, _F32P, _F32P, _I32P, _I32P, _I32P]),
    "spec_model_forward": (ctypes.c_int, [_VP, ctypes.c_int, _I32P, ctypes.c_int, ctypes.c_int, _VP]),
    "spec_accept_rows": (ctypes.c_int, [_VP, ctypes.c_int64, _VP, ctypes.c_int64, _VP, ctypes.c_int,
                                        ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_uint64,
                                        ctypes.c_uint64, _VP, _VP, _VP, _VP]),
    "spec_accept_rows_noalloc": (ctypes.c_int, [_VP, ctypes.c_int64, _VP, ctypes.c_int64, _VP,
                                                ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                ctypes.c_float, ctypes.c_uint64, ctypes.c_uint64,
                                                _VP, _VP, _VP, _VP]),
    "spec_sample_rows": (ctypes.c_int, [_VP, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_float, ctypes.c_uint64, ctypes.c_uint64,
                                        ctypes.c_int, _VP, _VP]),
    "spec_rope_plan": (ctypes.c_int, [_VP, _VP]),
    "spec_rope_rows": (ctypes.c_int, [_VP, _INT, _I64, _I64, _VP, _INT, _I64, _I64, _VP, _INT, _INT, _INT,
                                      _VP, _INT, _VP]),
    "spec_kv_append": (ctypes.c_int, [_VP, _VP, _I64, _I64, _VP, _I64, _I64, _INT, _VP, _VP, _INT, _VP, _VP]),
    "spec_kv_gather": (ctypes.c_int, [_VP, _VP, _VP, _INT, _VP, _VP, _INT, _VP]),
    "spec_qkv_append": (ctypes.c_int, [_VP, _VP, _I64, _I64, _VP, _I64, _I64, _VP, _I64, _I64, _INT, _VP, _VP, _INT,
                                       _INT, _VP, _VP, _VP, ctypes.c_float, _VP, _I64, _I64, _VP]),
    "spec_rope_norm_rows": (ctypes.c_int, [_VP, _INT, _I64, _I64, _VP, _INT, _I64, _I64, _VP, _INT, _INT, _INT,
                                           _VP, _I64, ctypes.c_float, _VP, _VP]),
    "spec_kv_reserve": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _INT, _INT, _VP, _VP, _VP, _VP, _VP, _VP]),
    "spec_kv_release": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _INT, _VP]),
    "spec_attn_paged": (ctypes.c_int, [_VP, _VP, _I64, _I64, _VP, _VP, _INT, _INT, _INT, ctypes.c_float,
                                       _VP, _I64, _I64, _VP, _VP, _I64, _VP]),
    "spec_attn_paged_workspace": (ctypes.c_int64, [_VP, _INT, _INT, _INT]),
    "spec_attn_prompt": (ctypes.c_int, [_VP, _I64, _I64, _VP, _I64, _I64, _VP, _I64, _I64, _VP, _INT, _INT,
                                        _INT, _INT, _INT, _INT, ctypes.c_float, _VP, _I64, _I64, _VP, _VP]),
    "spec_attn_paged_window": (ctypes.c_int, [_VP, _VP, _I64, _I64, _VP, _VP, _INT, _INT, _INT, ctypes.c_float,
                                              _INT, _INT, _VP, _I64, _I64, _VP, _VP, _I64, _VP]),
    "spec_attn_paged_window_workspace": (ctypes.c_int64, [_VP, _INT, _INT, _INT, _INT, _INT]),
    "spec_attn_prompt_window": (ctypes.c_int, [_VP, _I64, _I64, _VP, _I64, _I64, _VP, _I64, _I64, _VP, _INT, _INT,
                                               _INT, _INT, _INT, _INT, ctypes.c_float, _INT, _INT, _VP, _I64, _I64,
                                               _VP, _VP]),
    "spec_attn_shared": (ctypes.c_int, [_VP, _VP, _I64, _I64, _VP, _VP, _VP, _INT, _VP, _INT, _INT, _INT,
                                        ctypes.c_float, _VP, _I64, _I64, _VP, _VP, _I64, _VP]),
    "spec_attn_shared_workspace": (ctypes.c_int64, [_VP, _INT, _INT, _INT, _INT]),
    "spec_profile": (ctypes.c_int, [_VP, ctypes.c_int, ctypes.POINTER(Profile)]),
    "spec_phase_times": (ctypes.c_int, [_VP, ctypes.c_int, _VP, ctypes.c_int,
                                        ctypes.POINTER(ctypes.c_int)]),
    "spec_version": (ctypes.c_char_p, []),
    "spec_inject_fault": (ctypes.c_int, [_VP, ctypes.c_int, ctypes.c_int]),
    "spec_phase_list": (ctypes.c_int, [_VP, ctypes.c_int, _VP, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]),
    "spec_device_bytes_held": (ctypes.c_int64, []),
}

_lib = None


def lib():
    """The loaded CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError(f"{LIB} is missing: run build() first; this package has no CPU fallback")
        handle = ctypes.CDLL(LIB)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


class SpecError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{ERRORS.get(code, code)}: {msg}")
        self.code = code


def _check(rc, ctx=None):
    if rc != SPEC_OK:
        msg = lib().spec_last_error(ctx).decode(errors="replace")
        raise SpecError(rc, msg)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def model_desc(shape, weights):
    """ModelDesc for a shape (attributes n_layers, d_model, n_heads, n_kv_heads,
    head_dim, ffn_dim, vocab, rope_theta, rms_eps, dtype 'f32'|'bf16'|'q4') and a
    weights dict {'embed', 'final_norm', 'lm_head', 'layers': [dict]} of CUDA
    tensors ('q4': every matrix one uint8 buffer of packed codes followed by
    group-major bf16 scales, see include/specverify.h).  Returns (desc, keepalive)."""
    layers = (LayerWeights * shape.n_layers)()
    for i, lw in enumerate(weights["layers"]):
        for n in _LAYER_FIELDS:
            setattr(layers[i], n, lw[n].data_ptr())
    d = ModelDesc(shape.n_layers, shape.d_model, shape.n_heads, shape.n_kv_heads, shape.head_dim,
                  shape.ffn_dim, shape.vocab, shape.rope_theta, shape.rms_eps, _DTYPES[shape.dtype],
                  weights["embed"].data_ptr(), weights["final_norm"].data_ptr(),
                  weights["lm_head"].data_ptr(), layers)
    return d, (layers, weights)


class SpecDecoder:
    """One target/draft pair with K drafts per step over `batch` sequences
    (batch > 1: bf16 models, every sequence advancing independently);
    lookup = n > 0 drafts by prompt lookup (n-gram suffix match up to n
    tokens) instead of running the draft model; heads = a device tensor
    [K, d_model, d_model] in the target's arithmetic dtype drafts with
    self-draft heads on the target (draft_shape / draft_w then None)."""

    def __init__(self, target_shape, target_w, draft_shape, draft_w, k, max_ctx,
                 temperature=0.0, seed=0, mix_lambda=0.0, stream=None, flags=0, batch=1, lookup=0,
                 heads=None):
        self.k = k
        self.batch = batch
        self.vocab = target_shape.vocab
        self._td, self._tk = model_desc(target_shape, target_w)
        self._heads = heads
        if draft_shape is None:
            self._dd, self._dk = None, None
        else:
            self._dd, self._dk = model_desc(draft_shape, draft_w)
        opts = Opts(batch, max_ctx, temperature, seed, mix_lambda,
                    ctypes.c_void_p(stream) if stream else ctypes.c_void_p(0), flags, lookup,
                    ctypes.c_void_p(heads.data_ptr() if heads is not None else 0))
        h = ctypes.c_void_p()
        rc = lib().spec_init(ctypes.byref(self._td), ctypes.byref(self._dd) if self._dd is not None else None, k,
                             ctypes.byref(opts), ctypes.byref(h))
        _check(rc)
        self.ctx = h

    def close(self):
        if getattr(self, "ctx", None):
            lib().spec_free(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def prefill(self, tokens):
        """tokens: one prompt (batch 1) or `batch` prompts of one length."""
        rows = [list(tokens)] if self.batch == 1 and not hasattr(tokens[0], "__len__") else list(tokens)
        n = len(rows[0])
        flat = [int(t) for r in rows for t in r]
        arr = (ctypes.c_int32 * len(flat))(*flat)
        _check(lib().spec_prefill(self.ctx, arr, n), self.ctx)

    def prefill_synthetic(self, length, seed=0):
        """State of a prefill of `length` tokens with synthetic token ids and
        KV caches (benchmark workloads; the tokens carry no meaning)."""
        _check(lib().spec_prefill_synthetic(self.ctx, length, seed), self.ctx)

    def step(self):
        """Batch 1: (emitted tokens, flags).  Batch > 1: ([tokens of each
        sequence], [flags of each sequence])."""
        b = self.batch
        out = (ctypes.c_int32 * (b * (self.k + 1)))()
        cnt = (ctypes.c_int32 * b)()
        flags = (ctypes.c_uint32 * b)()
        _check(lib().spec_step(self.ctx, out, cnt, flags), self.ctx)
        rows = [list(out[i * (self.k + 1):i * (self.k + 1) + cnt[i]]) for i in range(b)]
        if b == 1:
            return rows[0], flags[0]
        return rows, list(flags)

    def seq_context(self, b):
        """Committed tokens of sequence b (the last is the pending token)."""
        import numpy as np
        n = ctypes.c_int32()
        _check(lib().spec_seq_context(self.ctx, b, None, ctypes.byref(n)), self.ctx)
        buf = np.zeros(max(1, n.value), dtype=np.int32)
        _check(lib().spec_seq_context(self.ctx, b, buf.ctypes.data_as(_I32P), ctypes.byref(n)), self.ctx)
        return buf[:n.value].copy()

    def generate(self, n_new):
        out = (ctypes.c_int32 * max(1, n_new))()
        got = ctypes.c_int32()
        _check(lib().spec_generate(self.ctx, n_new, out, ctypes.byref(got)), self.ctx)
        return list(out[:got.value])

    def ar_step(self):
        """Batch 1: the token; batch > 1: one token per sequence."""
        tok = (ctypes.c_int32 * self.batch)()
        _check(lib().spec_ar_step(self.ctx, tok), self.ctx)
        return tok[0] if self.batch == 1 else list(tok)

    def stats(self):
        s = Stats()
        _check(lib().spec_get_stats(self.ctx, ctypes.byref(s)), self.ctx)
        return s.as_dict()

    def profile(self, iters=20):
        """Graph-replayed phase times (ms): draft loop, verify pass, plain-decoding
        pass, and the verify pass's target forward alone."""
        pr = Profile()
        _check(lib().spec_profile(self.ctx, iters, ctypes.byref(pr)), self.ctx)
        return pr.as_dict()

    def phase_times(self, which):
        """Per-phase stamps of the last persistent run of forward `which`
        (0..K-1 draft passes, K verify, K+1 plain decoding): a list of dicts
        with kind, n, k, the earliest/latest arrival, the release, the latest
        end of X preparation and the latest end of streaming, in ns."""
        import numpy as np
        buf = np.zeros((1024, 8), dtype=np.int64)
        n = ctypes.c_int(0)
        _check(lib().spec_phase_times(self.ctx, which, buf.ctypes.data_as(_VP), 1024,
                                      ctypes.byref(n)), self.ctx)
        names = ("kind", "n", "k", "arrive_min_ns", "arrive_max_ns", "release_ns", "prep_max_ns",
                 "work_max_ns")
        return [dict(zip(names, (int(v) for v in row))) for row in buf[:n.value]]

    def last_step_debug(self, max_ctx):
        """(p_logits [K+1, V], q_logits [K, V], drafts [K], context tokens) as
        numpy; batch > 1: p [B, K+1, V], q [B, K, V], drafts [B, K] and
        sequence 0's context."""
        import numpy as np
        k, v, b = self.k, self.vocab, self.batch
        lead = () if b == 1 else (b,)
        p = np.zeros(lead + (k + 1, v), dtype=np.float32)
        q = np.zeros(lead + (k, v), dtype=np.float32)
        d = np.zeros(lead + (k,), dtype=np.int32)
        ctx = np.zeros(max_ctx, dtype=np.int32)
        n = ctypes.c_int32()
        _check(lib().spec_last_step_debug(self.ctx, p.ctypes.data_as(_F32P), q.ctypes.data_as(_F32P),
                                          d.ctypes.data_as(_I32P), ctx.ctypes.data_as(_I32P),
                                          ctypes.byref(n)), self.ctx)
        return p, q, d, ctx[:n.value].copy()

    def phase_list(self, which):
        """Phase geometry of persistent forward `which` (0..K-1 draft passes,
        K verify, K+1 plain decoding): a list of 8-tuples, see spec_phase_list."""
        import numpy as np
        buf = np.zeros((4096, 8), dtype=np.int64)
        n = ctypes.c_int(0)
        _check(lib().spec_phase_list(self.ctx, which, buf.ctypes.data_as(_VP), 4096, ctypes.byref(n)), self.ctx)
        return [tuple(int(v) for v in row) for row in buf[:n.value]]

    def inject_fault(self, kind, arg):
        """Test hook: arm (arg > 0) or disarm (0) a fault of this context
        (SPEC_FAULT_WAIT_TIMEOUT) -- see include/specverify.h."""
        _check(lib().spec_inject_fault(self.ctx, kind, arg), self.ctx)

    def model_forward(self, which, tokens, pos0, logits):
        """Forward of the target (0) or draft (1) over host token ids at
        positions pos0.. into logits (CUDA fp32 tensor [n, V])."""
        arr = (ctypes.c_int32 * len(tokens))(*[int(t) for t in tokens])
        _check(lib().spec_model_forward(self.ctx, which, arr, len(tokens), pos0, _ptr(logits)), self.ctx)


def inject_alloc_failure(n):
    """Test hook: the n-th device allocation of the next context creation fails."""
    _check(lib().spec_inject_fault(None, SPEC_FAULT_ALLOC, n))


def inject_attention_timeout(step):
    """Test hook: blocks of the tensor-memory attention kernels give up at their
    step-th 128 keys (0: disarm) -- see include/specverify.h."""
    _check(lib().spec_inject_fault(None, SPEC_FAULT_ATTN_TIMEOUT, step))


def clear_faults():
    _check(lib().spec_inject_fault(None, SPEC_FAULT_CLEAR, 0))


def device_bytes_held():
    """Device bytes held by every live context of this process."""
    return int(lib().spec_device_bytes_held())


def accept_rows(p_logits, q_logits, drafts, temperature, seed, step_base=0, stream=None,
                p_row_stride=None, q_row_stride=None, rows=None):
    """Fused acceptance over independent verify rows (CUDA tensors):
    p_logits [R, K+1, V] fp32, q_logits [R, K, V] fp32, drafts [R, K] int32.
    Returns (tokens [R, K+1] int32, counts [R] int32, flags [R] int32)."""
    import torch
    K = q_logits.shape[-2]
    V = p_logits.shape[-1]
    R = rows if rows is not None else p_logits.shape[0]
    dev = p_logits.device
    tokens = torch.empty((R, K + 1), dtype=torch.int32, device=dev)
    counts = torch.empty(R, dtype=torch.int32, device=dev)
    flags = torch.empty(R, dtype=torch.int32, device=dev)
    ps = p_row_stride if p_row_stride is not None else (K + 1) * V
    qs = q_row_stride if q_row_stride is not None else K * V
    st = stream if stream is not None else torch.cuda.current_stream().cuda_stream
    _check(lib().spec_accept_rows(_ptr(p_logits), ps, _ptr(q_logits), qs, _ptr(drafts), R, K, V,
                                  float(temperature), int(seed), int(step_base), _ptr(tokens),
                                  _ptr(counts), _ptr(flags), ctypes.c_void_p(st)))
    return tokens, counts, flags


def accept_rows_noalloc(p_logits, q_logits, drafts, temperature, seed, step_base=0, stream=None):
    """accept_rows for callers that cannot allocate device memory: the library's
    scratch comes from a fixed 4 MiB array instead of an allocator (outputs are
    still torch tensors here; C callers pass their own buffers)."""
    import torch
    K = q_logits.shape[-2]
    V = p_logits.shape[-1]
    R = p_logits.shape[0]
    dev = p_logits.device
    tokens = torch.empty((R, K + 1), dtype=torch.int32, device=dev)
    counts = torch.empty(R, dtype=torch.int32, device=dev)
    flags = torch.empty(R, dtype=torch.int32, device=dev)
    st = stream if stream is not None else torch.cuda.current_stream().cuda_stream
    _check(lib().spec_accept_rows_noalloc(_ptr(p_logits), (K + 1) * V, _ptr(q_logits), K * V,
                                          _ptr(drafts), R, K, V, float(temperature), int(seed),
                                          int(step_base), _ptr(tokens), _ptr(counts), _ptr(flags),
                                          ctypes.c_void_p(st)))
    return tokens, counts, flags


def sample_rows(logits, temperature, seed, step_base=0, position=1, stream=None, row_stride=None,
                rows=None):
    """Inverse-CDF draw per row of logits [R, V] (CUDA fp32); returns int32 [R]."""
    import torch
    V = logits.shape[-1]
    R = rows if rows is not None else logits.shape[0]
    out = torch.empty(R, dtype=torch.int32, device=logits.device)
    st = stream if stream is not None else torch.cuda.current_stream().cuda_stream
    rs = row_stride if row_stride is not None else V
    _check(lib().spec_sample_rows(_ptr(logits), rs, R, V, float(temperature), int(seed),
                                  int(step_base), int(position), _ptr(out), ctypes.c_void_p(st)))
    return out


# ---- paged-cache operators (see include/specverify.h) ----
# The calls run on the current stream of the tensors' device (or the raw
# stream given), with that device current; tensors are read by pointer.  What a
# call allocates, results and workspace, belongs to the stream it runs on: with
# `stream` given, a result that is used or dropped on another stream needs that
# stream to wait, and record_stream.  A step makes a call per layer and waits
# for none, so the checks are plain comparisons, and messages are made only
# where one fails.  None records a backward pass, so rows that require grad are
# refused while grad mode is on (a Function of one's own runs with it off:
# rope_rows with `inverse` is the gradient of rope_rows).
_t = None
_packed = None
_asked = _modes = _functions = _profiled = None


def _torch():
    global _t, _packed, _asked, _modes, _functions, _profiled
    if _t is None:
        import torch
        # torch.empty on the current device without its parsing and dispatch, where torch has it
        # (an attention call 16.6 -> 14.3 us of host time, kv_reserve 21 -> 15.6).  It skips what
        # torch.empty does for deterministic algorithms (a fill), dispatch and function modes and
        # profilers, so it is taken where torch can say that none of them is on.
        c = torch._C
        guards = getattr(getattr(c, "_dynamo", None), "guards", None)
        _asked = getattr(c, "_get_deterministic_algorithms", None)
        _modes = getattr(c, "_len_torch_dispatch_stack", None)
        _functions = getattr(c, "_len_torch_function_stack", None)
        _profiled = getattr(getattr(c, "_autograd", None), "_profiler_enabled", None)
        if _asked and _modes and _functions and _profiled:
            _packed = getattr(guards, "_empty_strided_cuda", None)
        _t = torch
    return _t


def _fast(dev):
    """The short allocation where it does what torch.empty on CUDA device `dev` does, else None."""
    if _packed is None or _t._C._cuda_getDevice() != dev or _asked() or _modes() or _functions() or _profiled():
        return None
    return _packed


def _empty(dev, shape, dtype, *fast):
    """A packed tensor on CUDA device `dev`; fast: what _fast gave for several."""
    packed = fast[0] if fast else _fast(dev)
    if packed is None:
        return _t.empty(shape, dtype=dtype, device=_t.device("cuda", dev))
    shape = tuple(shape)                     # (no torch.Size)
    n = len(shape)
    if n == 1:
        return packed(shape, (1,), dtype)
    if n == 2:
        return packed(shape, (max(shape[1], 1), 1), dtype)
    d = max(shape[2], 1)
    return packed(shape, (max(shape[1], 1) * d, d, 1), dtype)


def _refuse(msg):
    raise SpecError(-1, msg)


def _need(ok, msg):
    if not ok:
        _refuse(msg)


def _io_dtype(t):
    d = t.dtype
    if d is _t.bfloat16:
        return SPEC_DTYPE_BF16
    if d is _t.float32:
        return SPEC_DTYPE_F32
    _refuse(f"rows are fp32 or bf16, not {d}")


def _rows3(name, t):
    """Strides of a CUDA tensor [tokens, heads, head_dim]."""
    if t.requires_grad and _t.is_grad_enabled():
        _refuse(f"{name} requires grad, and the call has no backward pass: detach it, or call under torch.no_grad()")
    if not t.is_cuda or t.dim() != 3:
        _refuse(f"{name}: a CUDA tensor [tokens, heads, head_dim]")
    st = t.stride()
    if st[2] != 1 and t.shape[2] != 1 and t.numel():
        _refuse(f"{name}: the elements of a head must be adjacent")
    return st


def _index(name, t, n, dev):
    if t.dtype is not _t.int32 or t.shape != (n,) or t.get_device() != dev or not t.is_contiguous():
        _refuse(f"{name}: a contiguous int32 tensor of {n} on the rows' device")


def _alloc(stream, device, make):
    """make()'s tensors from the memory of the stream that the call runs on: the
    current stream's may still be in use by work queued there."""
    if stream is None or stream == _t._C._cuda_getCurrentRawStream(device.index):
        return make()
    # (handle 0 is the default stream, of which ExternalStream makes another)
    own = _t.cuda.ExternalStream(stream, device=device) if stream else _t.cuda.default_stream(device)
    with _t.cuda.stream(own):
        return make()


def _call(dev, stream, fn, *args):
    # the C calls behind torch.cuda.current_device and current_stream, whose
    # checks and objects cost more than the launch
    c = _t._C
    if c._cuda_getDevice() == dev:
        rc = fn(*args, c._cuda_getCurrentRawStream(dev) if stream is None else stream)
    else:
        with _t.cuda.device(dev):
            rc = fn(*args, c._cuda_getCurrentRawStream(dev) if stream is None else stream)
    if rc:
        _check(rc)


def _first_stride(name, t):
    """Elements between t[0] and t[1] as the C structure takes them, where 0
    stands for packed (of a single entry it is never used)."""
    if t.shape[0] == 1:
        return 0
    if t.stride(0) == 0:
        _refuse(f"{name}: a first stride of 0 (an expanded tensor); make it contiguous")
    return t.stride(0)


class KVCache:
    """A paged cache over caller-owned CUDA tensors: k, v [pages, n_kv_heads,
    page_size, head_dim] (bf16, or torch.float8_e4m3fn with uint8 k_scale,
    v_scale [pages, n_kv_heads, page_size]; pages may be strided, a page is
    contiguous) and the page table, int32 [seqs, max_pages].  Rows of the table
    may name the same pages (a shared prefix), but no tensor may be expanded
    along its first dimension.  The tensors are kept and read in place: write
    the table's rows as sequences grow."""

    def __init__(self, k, v, table, k_scale=None, v_scale=None):
        import torch
        _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype, "k and v: equal [pages, heads, page, dim]")
        _need(k.dtype in (torch.bfloat16, torch.float8_e4m3fn), f"the cache is bf16 or float8_e4m3fn, not {k.dtype}")
        f8 = k.dtype == torch.float8_e4m3fn
        _need(table.dtype == torch.int32 and table.dim() == 2 and table.stride(1) == 1, "table: int32 [seqs, max_pages]")
        pages, heads, ps, hd = k.shape
        for t in (k, v):
            _need(t.stride()[1:] == (ps * hd, hd, 1), "a page must be contiguous")
        stride, table_stride, scale_stride = _first_stride("k", k), _first_stride("table", table), 0
        _need(stride == _first_stride("v", v), "k and v must have one page stride")
        if f8:
            for t in (k_scale, v_scale):
                _need(t is not None and t.dtype == torch.uint8 and t.shape == (pages, heads, ps) and
                      t.stride()[1:] == (ps, 1), "an e4m3 cache needs uint8 scales [pages, heads, page]")
            scale_stride = _first_stride("k_scale", k_scale)
            _need(scale_stride == _first_stride("v_scale", v_scale), "the scales must have one page stride")
        else:
            _need(k_scale is None and v_scale is None, "a bf16 cache has no scales")
        for t in (k, v, table) + ((k_scale, v_scale) if f8 else ()):
            _need(t.is_cuda and t.device == k.device, "the cache's tensors must be on one CUDA device")
        self.k, self.v, self.k_scale, self.v_scale, self.table = k, v, k_scale, v_scale, table
        self.n_kv_heads, self.head_dim, self.page_size = heads, hd, ps
        self.seqs, self.max_pages = table.shape
        self.device = k.device
        self._dev = k.get_device()
        self._c = KVCacheDesc(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if f8 else None,
                              v_scale.data_ptr() if f8 else None, SPEC_DTYPE_E4M3 if f8 else SPEC_DTYPE_BF16,
                              pages, ps, heads, hd, stride, scale_stride, table.data_ptr(), table_stride,
                              self.seqs, self.max_pages)
        self._ref = ctypes.byref(self._c)
        self._ws = {}                        # workspace bytes of attn_paged calls by their sizes

    @classmethod
    def empty(cls, pages, page_size, n_kv_heads, head_dim, table, dtype="bf16"):
        """A zeroed pool of `pages` pages ('bf16' or 'e4m3') on the table's device."""
        import torch
        _need(dtype in ("bf16", "e4m3"), f"the cache is 'bf16' or 'e4m3', not {dtype!r}")
        shape = (pages, n_kv_heads, page_size, head_dim)
        if dtype == "bf16":
            k, v = (torch.zeros(shape, dtype=torch.bfloat16, device=table.device) for _ in range(2))
            return cls(k, v, table)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=table.device).view(torch.float8_e4m3fn)
                for _ in range(2))
        ks, vs = (torch.full(shape[:3], 127, dtype=torch.uint8, device=table.device) for _ in range(2))
        return cls(k, v, table, ks, vs)


def rope_plan(rot_dim, theta, interleaved=False, scaling="plain", factor=1.0, orig_ctx=0.0, low=1.0, high=4.0,
              mscale=1.0):
    """The rotation of rot_dim leading elements of a head, worked out once on
    the host: scaling 'plain', 'linear', 'ntk' or 'parts' (see spec_rope_desc)."""
    _need(scaling in _ROPE_SCALING, f"unknown scaling {scaling!r}")
    d = RopeDesc(rot_dim, int(bool(interleaved)), _ROPE_SCALING[scaling], theta, factor, orig_ctx, low, high, mscale)
    plan = RopePlan()
    _check(lib().spec_rope_plan(ctypes.byref(d), ctypes.byref(plan)))
    plan._ref = ctypes.byref(plan)
    return plan


def rope_rows(x, pos, plan, out=None, dtype=None, inverse=False, stream=None):
    """x [tokens, heads, head_dim] (fp32 or bf16, strided) rotated by the
    positions pos [tokens] int32; returns out (given, may be x itself, or new
    in `dtype`, by default x's).  inverse rotates back."""
    _torch()
    xs = _rows3("x", x)
    shape = x.shape
    n, h, d = shape
    dev = x.get_device()
    _index("pos", pos, n, dev)
    if out is None:
        out = _alloc(stream, x.device, lambda: _empty(dev, shape, x.dtype if dtype is None else dtype))
        ys = out.stride()
    else:
        if out.shape != shape or out.get_device() != dev or (dtype is not None and dtype is not out.dtype):
            _refuse("out: x's shape and device")
        ys = _rows3("out", out)
    _call(dev, stream, lib().spec_rope_rows, x.data_ptr(), _io_dtype(x), xs[0], xs[1], out.data_ptr(),
          _io_dtype(out), ys[0], ys[1], pos.data_ptr(), n, h, d, plan._ref, 1 if inverse else 0)
    return out


def kv_append(cache, k, v, seq, pos, plan=None, stream=None):
    """Write rows k (rotated by plan, if given) and v [tokens, n_kv_heads,
    head_dim] to positions pos of sequences seq (int32 [tokens]; a negative
    one skips the row).  Positions of one call must be distinct."""
    _torch()
    ks, vs = _rows3("k", k), _rows3("v", v)
    shape, dev = k.shape, cache._dev
    n, h, d = shape
    if v.shape != shape or k.dtype is not v.dtype or h != cache.n_kv_heads or d != cache.head_dim:
        _refuse("k and v: equal [tokens, n_kv_heads, head_dim] of the cache")
    if k.get_device() != dev or v.get_device() != dev:
        _refuse("k, v and the cache must be on one device")
    _index("seq", seq, n, dev)
    _index("pos", pos, n, dev)
    _call(dev, stream, lib().spec_kv_append, cache._ref, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
          _io_dtype(k), seq.data_ptr(), pos.data_ptr(), n, plan._ref if plan is not None else None)


def kv_gather(cache, seq, pos, dtype=None, stream=None):
    """(k, v) [tokens, n_kv_heads, head_dim] read back from positions pos of
    sequences seq, bf16 or fp32; rows that do not exist read as zeros."""
    _torch()
    n, dev = seq.shape[0], cache._dev
    _index("seq", seq, n, dev)
    _index("pos", pos, n, dev)
    shape = (n, cache.n_kv_heads, cache.head_dim)
    if dtype is None:
        dtype = _t.bfloat16
    k, v = _alloc(stream, cache.device, lambda: [_empty(dev, shape, dtype, f) for f in [_fast(dev)] * 2])
    _call(dev, stream, lib().spec_kv_gather, cache._ref, seq.data_ptr(), pos.data_ptr(), n, k.data_ptr(),
          v.data_ptr(), _io_dtype(k))
    return k, v


def _gain(name, t, shape, dev):
    if t.dtype is not _t.float32 or t.shape != shape or t.get_device() != dev or t.stride(-1) != 1:
        _refuse(f"{name}: fp32 {list(shape)} on the rows' device")
    if t.requires_grad and _t.is_grad_enabled():
        _refuse(f"{name} requires grad, and the call has no backward pass: detach it, or call under torch.no_grad()")


def rope_norm_rows(x, pos, plan, gain, eps=1e-5, out=None, dtype=None, stream=None):
    """rope_rows behind an RMS norm of each head: x * gain / sqrt(mean(x^2) +
    eps) over head_dim, then rotated.  gain: fp32 [head_dim], or [heads,
    head_dim] for a gain of each head (the q and k heads of one projection)."""
    _torch()
    xs = _rows3("x", x)
    shape = x.shape
    n, h, d = shape
    dev = x.get_device()
    _index("pos", pos, n, dev)
    _gain("gain", gain, shape[2:] if gain.dim() == 1 else shape[1:], dev)
    if out is None:
        out = _alloc(stream, x.device, lambda: _empty(dev, shape, x.dtype if dtype is None else dtype))
        ys = out.stride()
    else:
        if out.shape != shape or out.get_device() != dev or (dtype is not None and dtype is not out.dtype):
            _refuse("out: x's shape and device")
        ys = _rows3("out", out)
    _call(dev, stream, lib().spec_rope_norm_rows, x.data_ptr(), _io_dtype(x), xs[0], xs[1], out.data_ptr(),
          _io_dtype(out), ys[0], ys[1], pos.data_ptr(), n, h, d, gain.data_ptr(),
          gain.stride(0) if gain.dim() == 2 else 0, eps, plan._ref)
    return out


def qkv_append(cache, q, k, v, seq, pos, plan=None, q_norm=None, k_norm=None, eps=1e-5, out=None, stream=None):
    """A layer's rows behind its q/k/v projection in one launch: the heads of q
    [tokens, n_heads, head_dim] and k [tokens, n_kv_heads, head_dim] normed
    (fp32 gains [head_dim], if given) and rotated (plan, if given), q returned
    in bf16 (out, given or new; may be q itself), k and v written to positions
    pos of sequences seq as kv_append does."""
    _torch()
    qs, ks, vs = _rows3("q", q), _rows3("k", k), _rows3("v", v)
    qshape, shape, dev = q.shape, k.shape, cache._dev
    n, h, d = shape
    if v.shape != shape or k.dtype is not v.dtype or h != cache.n_kv_heads or d != cache.head_dim:
        _refuse("k and v: equal [tokens, n_kv_heads, head_dim] of the cache")
    if qshape[0] != n or qshape[2] != d or q.dtype is not k.dtype:
        _refuse("q: the tokens, head_dim and type of k")
    if q.get_device() != dev or k.get_device() != dev or v.get_device() != dev:
        _refuse("q, k, v and the cache must be on one device")
    _index("seq", seq, n, dev)
    _index("pos", pos, n, dev)
    for name, g in (("q_norm", q_norm), ("k_norm", k_norm)):
        if g is not None:
            _gain(name, g, shape[2:], dev)
    if out is None:
        out = _alloc(stream, cache.device, lambda: _empty(dev, qshape, _t.bfloat16))
        os_ = out.stride()
    else:
        if out.shape != qshape or out.dtype is not _t.bfloat16 or out.get_device() != dev:
            _refuse("out: bf16 of q's shape and device")
        os_ = _rows3("out", out)
    _call(dev, stream, lib().spec_qkv_append, cache._ref, q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1],
          v.data_ptr(), vs[0], vs[1], _io_dtype(k), seq.data_ptr(), pos.data_ptr(), n, qshape[1],
          plan._ref if plan is not None else None, q_norm.data_ptr() if q_norm is not None else None,
          k_norm.data_ptr() if k_norm is not None else None, eps, out.data_ptr(), os_[0], os_[1])
    return out


def _stack(cache, free, n_free):
    if free.dim() != 1:
        _refuse("free: a contiguous int32 tensor of page numbers")
    _index("free", free, free.shape[0], cache._dev)
    _index("n_free", n_free, 1, cache._dev)


def kv_reserve(cache, kv_lens, counts, free, n_free, tokens, stream=None):
    """Pages and index arrays of counts[b] new tokens of every sequence b
    (int32 [seqs]) behind its kv_lens[b] positions: takes the pages from the
    stack free[: n_free] (int32, n_free int32 [1]; both changed in place), writes
    them into the cache's table, and returns (cu_q [seqs + 1], kv_lens with the
    new tokens [seqs], seq [tokens], pos [tokens], lacking [1]), as the row and
    attention calls take them; `tokens` bounds the step's tokens, and entries
    past them are -1.  Requests are served in order and whole; one that does
    not fit gets nothing (its length is as before), and lacking counts the
    pages that were missing (want of room in the table or in `tokens` shows in
    the lengths alone)."""
    _torch()
    dev, seqs = cache._dev, cache.seqs
    _index("kv_lens", kv_lens, seqs, dev)
    _index("counts", counts, seqs, dev)
    _stack(cache, free, n_free)
    if not 0 <= tokens <= 0x7fffff00:
        _refuse("tokens: a bound on the step's tokens, up to 2^31 - 256")
    cu, lens, seq, pos, lacking = _alloc(stream, cache.device, lambda: [
        _empty(dev, (n,), _t.int32, f) for f in [_fast(dev)] for n in (seqs + 1, seqs, tokens, tokens, 1)])
    _call(dev, stream, lib().spec_kv_reserve, cache._ref, kv_lens.data_ptr(), counts.data_ptr(), free.data_ptr(),
          n_free.data_ptr(), free.shape[0], tokens, cu.data_ptr(), lens.data_ptr(), seq.data_ptr(), pos.data_ptr(),
          lacking.data_ptr())
    return cu, lens, seq, pos, lacking


def kv_release(cache, kv_lens, keep, free, n_free, stream=None):
    """The pages of positions keep[b] .. kv_lens[b] - 1 of every sequence b
    (int32 [seqs]: the lengths with the tokens that are dropped, and without)
    back to the stack free[: n_free]; their entries of the table become -1.
    Entries that are negative already (given back by the caller, as pages in
    front of a window) are left out.  A page that several sequences name must
    not be dropped by more than one."""
    _torch()
    dev = cache._dev
    _index("kv_lens", kv_lens, cache.seqs, dev)
    _index("keep", keep, cache.seqs, dev)
    _stack(cache, free, n_free)
    _call(dev, stream, lib().spec_kv_release, cache._ref, kv_lens.data_ptr(), keep.data_ptr(), free.data_ptr(),
          n_free.data_ptr(), free.shape[0])


def _attn_out(q, shape, dev, out, lse, need, stream):
    """The call's out, lse and workspace of `need` bytes, checked or new."""
    if q.dtype is not _t.bfloat16:
        _refuse(f"q is bf16, not {q.dtype}")
    if out is not None and (out.shape != shape or out.dtype is not _t.bfloat16 or out.get_device() != dev):
        _refuse("out: like q")
    if lse is not None and lse is not False and (lse.shape != shape[:2] or lse.dtype is not _t.float32 or lse.get_device() != dev or
                               not lse.is_contiguous()):
        _refuse("lse: contiguous fp32 [tokens, heads]")
    if out is not None and lse is not None and not need:
        return out, lse, None

    def make():
        f = _fast(dev)
        return (_empty(dev, shape, _t.bfloat16, f) if out is None else out,
                _empty(dev, shape[:2], _t.float32, f) if lse is None else lse,
                _empty(dev, (need,), _t.uint8, f) if need else None)
    return _alloc(stream, q.device, make)


def _window(window, sinks):
    if window < 0 or sinks < 0:
        _refuse("window and sinks must not be negative")
    return min(window, 0x7fffffff), min(sinks, 0x7fffffff)


def _paged_args(q, cache, cu_q, kv_lens):
    """(strides, shape, device) of an attention call over the cache."""
    qs = _rows3("q", q)
    shape, dev, seqs = q.shape, cache._dev, cache.seqs
    if shape[2] != cache.head_dim or q.get_device() != dev:
        _refuse("q must have the cache's head_dim and device")
    _index("cu_q", cu_q, seqs + 1, dev)
    _index("kv_lens", kv_lens, seqs, dev)
    return qs, shape, dev


def _ws_bytes(cache, key, dev, ask):
    """Workspace bytes of a call by its sizes (key), a function of them alone."""
    need = cache._ws.get(key)
    if need is None:
        with _t.cuda.device(dev):
            need = ask()
        if len(cache._ws) > 4096:
            cache._ws.clear()
        cache._ws[key] = need
    return need


def attn_paged(q, cache, cu_q, kv_lens, max_q=None, scale=0.0, out=None, lse=None, stream=None, window=0, sinks=0):
    """Causal attention of the sequences' newest tokens over the cache.  q
    [tokens, n_heads, head_dim] bf16; sequence b (row b of the cache's table)
    owns rows cu_q[b] .. cu_q[b+1]-1 and kv_lens[b] cached positions, its new
    ones included (int32 [seqs + 1], [seqs]); max_q bounds the rows of one
    sequence and goes into the choice of kernel (default: tokens; give the
    real bound for batches).  window > 0: the row at position p sees positions
    j <= p with j > p - window or j < sinks.  Returns (out, lse [tokens,
    n_heads] fp32, or None with lse=False); rows outside every sequence are
    not written."""
    _torch()
    qs, shape, dev = _paged_args(q, cache, cu_q, kv_lens)
    n, h, d = shape
    if max_q is None:
        max_q = n
    if window or sinks:
        window, sinks = _window(window, sinks)
        need = _ws_bytes(cache, (n, max_q, h, window, sinks), dev,
                         lambda: lib().spec_attn_paged_window_workspace(cache._ref, n, max_q, h, window, sinks))
        out, lse, ws = _attn_out(q, shape, dev, out, lse, need, stream)
        os_ = _rows3("out", out)
        _call(dev, stream, lib().spec_attn_paged_window, cache._ref, q.data_ptr(), qs[0], qs[1], cu_q.data_ptr(),
              kv_lens.data_ptr(), n, max_q, h, scale, window, sinks, out.data_ptr(), os_[0], os_[1],
              lse.data_ptr() if lse is not False else None, ws.data_ptr() if need else None, need)
        return out, (lse if lse is not False else None)
    need = _ws_bytes(cache, (n, max_q, h), dev, lambda: lib().spec_attn_paged_workspace(cache._ref, n, max_q, h))
    out, lse, ws = _attn_out(q, shape, dev, out, lse, need, stream)
    os_ = _rows3("out", out)
    _call(dev, stream, lib().spec_attn_paged, cache._ref, q.data_ptr(), qs[0], qs[1], cu_q.data_ptr(),
          kv_lens.data_ptr(), n, max_q, h, scale, out.data_ptr(), os_[0], os_[1],
          lse.data_ptr() if lse is not False else None, ws.data_ptr() if need else None, need)
    return out, (lse if lse is not False else None)


def attn_shared(q, cache, cu_q, kv_lens, shared, groups=None, max_q=None, scale=0.0, out=None, lse=None, stream=None):
    """attn_paged for sequences whose rows of the cache's table name the same
    pages at their beginning: the first shared[g] positions (int32 [groups]) of
    the sequences groups[g] .. groups[g+1]-1 (int32 [groups + 1]; default: one
    group of all) are read once for the group.  Any number of positions; it is
    cut to what every row of the group sees.  Whether sharing pays is judged by
    the sizes given and the table's width: for short contexts in a wide table
    attn_paged takes half the time."""
    _torch()
    qs, shape, dev = _paged_args(q, cache, cu_q, kv_lens)
    n, h, d = shape
    ng = 1 if groups is None else groups.shape[0] - 1 if groups.dim() == 1 else 0
    if ng < 1:
        _refuse("groups: int32 [groups + 1]")
    if groups is not None:
        _index("groups", groups, ng + 1, dev)
    _index("shared", shared, ng, dev)
    if max_q is None:
        max_q = n
    need = _ws_bytes(cache, (n, max_q, h, ng), dev,
                     lambda: lib().spec_attn_shared_workspace(cache._ref, ng, n, max_q, h))
    out, lse, ws = _attn_out(q, shape, dev, out, lse, need, stream)
    os_ = _rows3("out", out)
    _call(dev, stream, lib().spec_attn_shared, cache._ref, q.data_ptr(), qs[0], qs[1], cu_q.data_ptr(),
          kv_lens.data_ptr(), groups.data_ptr() if groups is not None else None, ng, shared.data_ptr(), n, max_q, h,
          scale, out.data_ptr(), os_[0], os_[1], lse.data_ptr() if lse is not False else None,
          ws.data_ptr() if need else None, need)
    return out, (lse if lse is not False else None)


def attn_prompt(q, k, v, cu, max_len=None, scale=0.0, out=None, lse=None, stream=None, window=0, sinks=0):
    """Causal attention within packed sequences: rows cu[b] .. cu[b+1]-1 of q
    [tokens, n_heads, head_dim] and k, v [tokens, n_kv_heads, head_dim] (bf16,
    may be slices of one projection) are sequence b; max_len bounds their
    lengths and sizes the grid (default: tokens; give the real bound for many);
    window and sinks as for attn_paged.  Returns (out, lse) as attn_paged."""
    _torch()
    qs, ks, vs = _rows3("q", q), _rows3("k", k), _rows3("v", v)
    shape, kshape, dev = q.shape, k.shape, q.get_device()
    n, h, d = shape
    if v.shape != kshape or kshape[0] != n or kshape[2] != d:
        _refuse("k and v: equal [tokens, n_kv_heads, head_dim]")
    if k.dtype is not _t.bfloat16 or v.dtype is not _t.bfloat16:
        _refuse("k and v are bf16")
    if k.get_device() != dev or v.get_device() != dev:
        _refuse("q, k and v must be on one device")
    seqs = cu.shape[0] - 1 if cu.dim() == 1 else 0
    if seqs < 1:
        _refuse("cu: int32 [sequences + 1]")
    _index("cu", cu, seqs + 1, dev)
    out, lse, _ = _attn_out(q, shape, dev, out, lse, 0, stream)
    os_ = _rows3("out", out)
    if window or sinks:
        window, sinks = _window(window, sinks)
        _call(dev, stream, lib().spec_attn_prompt_window, q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1],
              v.data_ptr(), vs[0], vs[1], cu.data_ptr(), seqs, n, n if max_len is None else max_len, h, kshape[1], d,
              scale, window, sinks, out.data_ptr(), os_[0], os_[1],
              lse.data_ptr() if lse is not False else None)
        return out, (lse if lse is not False else None)
    _call(dev, stream, lib().spec_attn_prompt, q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1],
          v.data_ptr(), vs[0], vs[1], cu.data_ptr(), seqs, n, n if max_len is None else max_len, h, kshape[1], d,
          scale, out.data_ptr(), os_[0], os_[1], lse.data_ptr() if lse is not False else None)
    return out, (lse if lse is not False else None)
