"""Python binding of libtq (TurboQuant hot path on B200), argument marshalling only.

Every computation runs in libtq.so's CUDA kernels; PyTorch provides device memory and
streams.  There is no fallback: if libtq.so has not been built this module raises on
first use (build it with ``python -m kv_cache_vector_08_b200.build``).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
from dataclasses import dataclass
from typing import Optional, Sequence

import numpy as np

__all__ = [
    "MODE_PROD", "MODE_MSE", "TQError", "Context", "Packed", "host_params", "alloc_packed",
    "quantize_kv", "quantize_workspace_size", "channel_perm_by_score", "dequantize", "prepare_queries", "attn_logits", "decode_attention",
    "decode_workspace_size", "search_topk", "launch_count", "lib_path", "lib",
    "rope", "rope_frequencies", "page_bounds", "alloc_page_bounds", "SparsePlan", "sparse_decode_attention",
    "sparse_workspace_size", "TreePlan", "tree_attention", "tree_workspace_size", "tree_mask",
]

MODE_PROD = 0
MODE_MSE = 1
DTYPE_F32, DTYPE_BF16, DTYPE_F16 = 0, 1, 2

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libtq.so")
_lib = None


class TQError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("libtq status %d: %s" % (status, msg))
        self.status = status


class _Packed(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("norm", ctypes.c_void_p), ("rnorm", ctypes.c_void_p),
                ("cap", ctypes.c_int64)]


class _DecodeOpts(ctypes.Structure):
    _fields_ = [("channel_perm", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("page_tokens", ctypes.c_int)]


class _RopeTensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int), ("x_token", ctypes.c_int64),
                ("x_head", ctypes.c_int64), ("out_token", ctypes.c_int64), ("out_head", ctypes.c_int64)]


class _RopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("factor", ctypes.c_double), ("original_len", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double)]


class _SparseOpts(ctypes.Structure):
    _fields_ = [("bounds", ctypes.c_void_p), ("bounds_dtype", ctypes.c_int), ("bounds_pages", ctypes.c_int64),
                ("select", ctypes.c_int), ("first", ctypes.c_int), ("last", ctypes.c_int), ("selected", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("page_tokens", ctypes.c_int), ("channel_perm", ctypes.c_void_p)]


class _Info(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int), ("bits", ctypes.c_int), ("k", ctypes.c_int), ("m", ctypes.c_int),
                ("mode", ctypes.c_int), ("planes", ctypes.c_int), ("d_pad", ctypes.c_int),
                ("code_bytes", ctypes.c_int), ("seed", ctypes.c_uint64)]


def lib_path() -> str:
    return _LIB_PATH


def lib():
    """Load libtq.so (raises if it is missing: there is no other implementation)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError("libtq.so not built at %s; run python -m kv_cache_vector_08_b200.build" % _LIB_PATH)
    L = ctypes.CDLL(_LIB_PATH)
    P, I, I64, U64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t
    F = ctypes.c_float
    PK = ctypes.POINTER(_Packed)
    sig = {
        "tq_init": (I, [ctypes.POINTER(P), I, I, U64, I]),
        "tq_host_params": (I, [I, I, U64, I, P, P, P, P]),
        "tq_free": (None, [P]),
        "tq_get_info": (I, [P, ctypes.POINTER(_Info)]),
        "tq_get_params": (I, [P, P, P, P, P]),
        "tq_quantize_workspace_size": (SZ, [P, I, I64, I64]),
        "tq_quantize_kv": (I, [P, P, I, I64, I64, PK, P, P, SZ, P]),
        "tq_dequantize": (I, [P, PK, P, I64, P, I64, P]),
        "tq_dequantize_qjl": (I, [P, PK, P, I64, P, I64, P]),
        "tq_prepare_queries": (I, [P, P, I64, I64, P, P]),
        "tq_attn_logits_workspace_size": (SZ, [P, I64]),
        "tq_attn_logits": (I, [P, P, I64, PK, I64, P, P, SZ, P]),
        "tq_decode_workspace_size": (SZ, [I, I, I, I, I, I64]),
        "tq_decode_attention": (I, [P, P, P, I, P, I, PK, PK, P, I, I, I, I, I64, F, P, P, SZ, P]),
        "tq_decode_attention_ex": (I, [P, P, P, I, P, I, PK, PK, P, I, I, I, I, I64, F, P, ctypes.POINTER(_DecodeOpts),
                                       P, SZ, P]),
        "tq_channel_perm_by_score": (I, [P, I, I, P]),
        "tq_quantize_cols_workspace_size": (SZ, [P, I64]),
        "tq_quantize_kv_cols": (I, [P, P, I, I64, I64, P, PK, P, P, SZ, P]),
        "tq_search_workspace_size": (SZ, [P, I64, I64, I]),
        "tq_search_topk": (I, [P, P, I64, PK, I64, I, P, P, P, SZ, P]),
        "tq_rope": (I, [P, I, I, I64, I, I, P, P, I, ctypes.c_double, I, P]),
        "tq_rope_frequencies": (I, [I, ctypes.c_double, ctypes.POINTER(_RopeScaling), P, ctypes.POINTER(ctypes.c_double)]),
        "tq_page_bounds": (I, [P, I64, I, I64, I64, P, P, I, I, I, I64, P, I, I, P, I64, P]),
        "tq_sparse_workspace_size": (SZ, [I, I, I, I, I, I64, I, I]),
        "tq_sparse_decode_attention": (I, [P, P, P, I, P, I, PK, PK, P, I, I, I, I, I64, F, P,
                                           ctypes.POINTER(_SparseOpts), P, SZ, P]),
        "tq_tree_workspace_size": (SZ, [I, I, I, I, I, I, I64]),
        "tq_tree_attention": (I, [P, P, P, I, P, I, PK, PK, P, P, P, I, I, I, I, I, I64, F, P,
                                  ctypes.POINTER(_DecodeOpts), P, SZ, P]),
        "tq_tree_mask": (I, [P, I, I, P]),
        "tq_last_error": (ctypes.c_char_p, []),
        "tq_kernel_launch_count": (U64, []),
        "tq_get_device_error": (I, [P, ctypes.POINTER(I)]),
        "tq_debug_set_wait_limit": (I, [U64]),
        "tq_debug_inject_stall": (I, [I]),
        "tq_debug_fail_alloc": (I, [I]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def _check(status: int):
    if status != 0:
        raise TQError(status, lib().tq_last_error().decode())


def launch_count() -> int:
    return int(lib().tq_kernel_launch_count())


def _torch():
    import torch
    return torch


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


_CODES = {}


def _dtype_code(t) -> int:
    if not _CODES:
        torch = _torch()
        _CODES.update({torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16})
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError("unsupported dtype %s" % t.dtype)
    return code


def _rows(t, d: int):
    """(pointer, n, ld) of a 2-D tensor whose rows are unit-stride with >= d elements."""
    if t.dim() != 2 or t.stride(1) != 1 or t.shape[1] < d:
        raise ValueError("expected a 2-D tensor [n, >=%d] with unit stride along rows" % d)
    return t.shape[0], max(t.stride(0), d)


def host_params(d: int, bits: int, seed: int, mode: int) -> dict:
    """The library's float64 parameters computed on the host (no GPU needed)."""
    k = bits - 1 if mode == MODE_PROD else bits
    Pi = np.zeros((d, d))
    S = np.zeros((d, d)) if mode == MODE_PROD else None
    c = np.zeros(2 ** k) if k >= 1 else np.zeros(1)
    t = np.zeros(max(2 ** k - 1, 1))
    p = lambda a: None if a is None else a.ctypes.data_as(ctypes.c_void_p)
    _check(lib().tq_host_params(d, bits, seed, mode, p(Pi), p(S), p(c), p(t)))
    return dict(Pi=Pi, S=S, centroids=c, boundaries=t[:2 ** k - 1])


class Context:
    """Owns one libtq context (Pi, S, codebook on the current CUDA device)."""

    def __init__(self, d: int, bits: int, seed: int, mode: int = MODE_PROD):
        h = ctypes.c_void_p()
        _check(lib().tq_init(ctypes.byref(h), d, bits, seed, mode))
        self._h = h
        info = _Info()
        _check(lib().tq_get_info(h, ctypes.byref(info)))
        self.d, self.bits, self.k, self.m, self.mode = info.d, info.bits, info.k, info.m, info.mode
        self.planes, self.d_pad, self.code_bytes, self.seed = info.planes, info.d_pad, info.code_bytes, info.seed

    @property
    def handle(self):
        return self._h

    def params(self) -> dict:
        d, K = self.d, 2 ** self.k
        Pi = np.zeros((d, d))
        S = np.zeros((d, d)) if self.mode == MODE_PROD else None
        c = np.zeros(K)
        t = np.zeros(max(K - 1, 1))
        p = lambda a: None if a is None else a.ctypes.data_as(ctypes.c_void_p)
        _check(lib().tq_get_params(self._h, p(Pi), p(S), p(c), p(t)))
        return dict(Pi=Pi, S=S, centroids=c, boundaries=t[:K - 1], mode=self.mode, k=self.k, m=self.m, d=d)

    def device_error(self) -> int:
        """Kernel-side failure code recorded for this context (0 = none); clears it."""
        v = ctypes.c_int(0)
        _check(lib().tq_get_device_error(self._h, ctypes.byref(v)))
        return v.value

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().tq_free(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


@dataclass
class Packed:
    """Caller-owned packed storage: codes [cap, code_bytes] uint8, norm [cap] fp16,
    rnorm [cap] fp16 (prod mode) -- all torch CUDA tensors."""
    codes: object
    norm: object
    rnorm: Optional[object]

    @property
    def cap(self) -> int:
        return self.codes.shape[0]

    def struct(self) -> _Packed:
        return _Packed(self.codes.data_ptr(), self.norm.data_ptr(),
                       0 if self.rnorm is None else self.rnorm.data_ptr(), self.codes.shape[0])


def alloc_packed(ctx: Context, cap: int, device=None) -> Packed:
    torch = _torch()
    device = device or torch.device("cuda", torch.cuda.current_device())
    codes = torch.zeros((cap, ctx.code_bytes), dtype=torch.uint8, device=device)
    norm = torch.zeros(cap, dtype=torch.float16, device=device)
    rnorm = torch.zeros(cap, dtype=torch.float16, device=device) if ctx.mode == MODE_PROD else None
    return Packed(codes, norm, rnorm)


def quantize_workspace_size(ctx: Context, x_dtype: int, n: int, ld: int) -> int:
    return int(lib().tq_quantize_workspace_size(ctx.handle, x_dtype, n, ld))


def quantize_kv(ctx: Context, x, dst: Packed, slots=None, stream=None, workspace=None, cols=None):
    """Quantize rows of x (CUDA tensor [n, >=d], fp32/bf16/fp16) into dst (slot v, or slots[v]).
    cols (CUDA int32 [d]): quantize the columns cols of each row of x instead of its first d.
    A workspace is allocated (torch caching allocator) when the call needs one and none is given."""
    torch = _torch()
    dt = _dtype_code(x)
    ps = dst.struct()
    if cols is not None:
        if x.dim() != 2 or x.stride(1) != 1:
            raise ValueError("expected a 2-D tensor with unit stride along rows")
        n, ld = x.shape[0], x.stride(0)
        need = int(lib().tq_quantize_cols_workspace_size(ctx.handle, n))
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        _check(lib().tq_quantize_kv_cols(ctx.handle, _ptr(x), dt, n, ld, _ptr(cols), ctypes.byref(ps), _ptr(slots),
                                         _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                         _stream(stream)))
        return
    n, ld = _rows(x, ctx.d)
    need = quantize_workspace_size(ctx, dt, n, ld)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    _check(lib().tq_quantize_kv(ctx.handle, _ptr(x), dt, n, ld, ctypes.byref(ps), _ptr(slots), _ptr(workspace),
                                0 if workspace is None else workspace.numel(), _stream(stream)))


def channel_perm_by_score(score, w0: int) -> np.ndarray:
    """Host permutation putting the w0 highest-scoring channels first (see tq.h)."""
    score = np.ascontiguousarray(score, dtype=np.float32)
    perm = np.zeros(score.shape[0], dtype=np.int32)
    _check(lib().tq_channel_perm_by_score(score.ctypes.data_as(ctypes.c_void_p), score.shape[0], int(w0),
                                          perm.ctypes.data_as(ctypes.c_void_p)))
    return perm


def dequantize(ctx: Context, src: Packed, n: int = None, slots=None, out=None, stream=None, qjl: bool = False):
    """x_hat = norm Pi^T c[idx] of stored vectors (qjl=True, prod mode: plus the QJL term
    norm sqrt(pi/2)/m rnorm S^T (2 s - 1))."""
    torch = _torch()
    if slots is not None:
        n = slots.shape[0]
    if out is None:
        out = torch.empty((n, ctx.d), dtype=torch.float32, device=src.codes.device)
    ps = src.struct()
    fn = lib().tq_dequantize_qjl if qjl else lib().tq_dequantize
    _check(fn(ctx.handle, ctypes.byref(ps), _ptr(slots), n, _ptr(out), out.stride(0), _stream(stream)))
    return out


def prepare_queries(ctx: Context, q, out=None, stream=None):
    torch = _torch()
    nq, ld = _rows(q, ctx.d)
    if out is None:
        out = torch.empty((nq, ctx.d + ctx.m), dtype=torch.float32, device=q.device)
    _check(lib().tq_prepare_queries(ctx.handle, _ptr(q), nq, ld, _ptr(out), _stream(stream)))
    return out


def attn_logits(ctx: Context, q, keys: Packed, n: int, out=None, workspace=None, stream=None):
    torch = _torch()
    q = q.contiguous()
    nq = q.shape[0]
    if out is None:
        out = torch.empty((nq, n), dtype=torch.float32, device=q.device)
    need = int(lib().tq_attn_logits_workspace_size(ctx.handle, nq))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    ps = keys.struct()
    _check(lib().tq_attn_logits(ctx.handle, _ptr(q), nq, ctypes.byref(ps), n, _ptr(out), _ptr(workspace),
                                workspace.numel(), _stream(stream)))
    return out


def decode_workspace_size(B, Hq, Hkv, D, ngroups, max_len) -> int:
    return int(lib().tq_decode_workspace_size(B, Hq, Hkv, D, ngroups, max_len))


class DecodePlan:
    """Pre-marshalled arguments of tq_decode_attention (avoids per-call ctypes setup)."""

    def __init__(self, kctx: Sequence[Context], vctx: Sequence[Context], group_off: Sequence[int],
                 kcache: Sequence[Packed], vcache: Sequence[Packed], B, Hq, Hkv, D, max_len, device=None,
                 channel_perm=None, block_table=None, page_tokens: int = 0):
        torch = _torch()
        # options: channel_perm CUDA int32 [Hkv, D]; block_table CUDA int32 [B, max_len / page_tokens]
        self._opts = None
        if channel_perm is not None or block_table is not None:
            self._opts = _DecodeOpts(0 if channel_perm is None else channel_perm.data_ptr(),
                                     0 if block_table is None else block_table.data_ptr(), int(page_tokens))
            self._keep_opts = (channel_perm, block_table)
        G = len(kctx)
        self.G, self.B, self.Hq, self.Hkv, self.D, self.max_len = G, B, Hq, Hkv, D, max_len
        self._k = (ctypes.c_void_p * G)(*[c.handle.value for c in kctx])
        self._v = (ctypes.c_void_p * G)(*[c.handle.value for c in vctx])
        self._off = (ctypes.c_int * (G + 1))(*list(group_off))
        self._kc = (_Packed * G)(*[p.struct() for p in kcache])
        self._vc = (_Packed * G)(*[p.struct() for p in vcache])
        self._keep = (kctx, vctx, kcache, vcache)
        need = decode_workspace_size(B, Hq, Hkv, D, G, max_len)
        device = device or kcache[0].codes.device
        self.workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)

    def __call__(self, q, seq_lens, scale: float, out, stream=None):
        if self._opts is not None:
            _check(lib().tq_decode_attention_ex(self._k, self._v, self._off, self.G, _ptr(q), _dtype_code(q), self._kc,
                                                self._vc, _ptr(seq_lens), self.B, self.Hq, self.Hkv, self.D,
                                                self.max_len, ctypes.c_float(scale), _ptr(out), ctypes.byref(self._opts),
                                                _ptr(self.workspace), self.workspace.numel(), _stream(stream)))
            return out
        _check(lib().tq_decode_attention(self._k, self._v, self._off, self.G, _ptr(q), _dtype_code(q), self._kc,
                                         self._vc, _ptr(seq_lens), self.B, self.Hq, self.Hkv, self.D,
                                         self.max_len, ctypes.c_float(scale), _ptr(out), _ptr(self.workspace),
                                         self.workspace.numel(), _stream(stream)))
        return out


def decode_attention(kctx, vctx, group_off, q, kcache, vcache, seq_lens, Hkv, max_len, scale, out=None,
                     stream=None, channel_perm=None, block_table=None, page_tokens=0):
    """One decode step; q [B, Hq, D] (fp32/bf16 CUDA), seq_lens int32 CUDA [B] -> out fp32 [B, Hq, D].
    Token t of sequence b, kv head h lives in slot (b*Hkv + h)*max_len + t of each cache."""
    torch = _torch()
    B, Hq, D = q.shape
    plan = DecodePlan(kctx, vctx, group_off, kcache, vcache, B, Hq, Hkv, D, max_len, device=q.device,
                      channel_perm=channel_perm, block_table=block_table, page_tokens=page_tokens)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    return plan(q.contiguous(), seq_lens, scale, out, stream)


def search_topk(ctx: Context, q, db: Packed, N: int, k: int, stream=None):
    torch = _torch()
    q = q.contiguous()
    nq = q.shape[0]
    scores = torch.empty((nq, k), dtype=torch.float32, device=q.device)
    ids = torch.empty((nq, k), dtype=torch.int64, device=q.device)
    need = int(lib().tq_search_workspace_size(ctx.handle, nq, N, k))
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    ps = db.struct()
    _check(lib().tq_search_topk(ctx.handle, _ptr(q), nq, ctypes.byref(ps), N, k, _ptr(scores), _ptr(ids),
                                _ptr(ws), ws.numel(), _stream(stream)))
    return scores, ids


# ------------------------------------------------------------------ around the cache
ROPE_SCALINGS = {None: 0, "none": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}


def _raw_stream(stream) -> int:
    """Address of the stream; the current one of the current device when None (without building a Stream object)."""
    if stream is not None:
        return stream.cuda_stream
    torch = _torch()
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _on_current_device(*tensors):
    """Every call launches on the current device: a tensor of another one (or of the host) is refused."""
    dev = _torch()._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != dev:      # (-1 for the host)
            raise ValueError("expected CUDA tensors on the current device (cuda:%d), got one on %s" % (dev, t.device))


def _int32(t, shape, name):
    if t.dtype is not _torch().int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of shape %s" % (name, tuple(shape)))


def rope_frequencies(rot: int, base: float = 10000.0, scaling=None, factor: float = 1.0, original_len: float = 0.0,
                     low: float = 1.0, high: float = 32.0):
    """(float64 numpy [rot/2] frequencies, factor on the rotated values) of rotary positions; scaling None,
    "linear", "ntk", "bands" or "yarn" (see tq_rope_frequencies in tq.h)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling must be one of %s" % sorted(k for k in ROPE_SCALINGS if k))
    freq = np.zeros(max(int(rot) // 2, 1))
    f = ctypes.c_double(0.0)
    s = _RopeScaling(ROPE_SCALINGS[scaling], factor, original_len, low, high)
    _check(lib().tq_rope_frequencies(int(rot), base, ctypes.byref(s), freq.ctypes.data_as(ctypes.c_void_p),
                                     ctypes.byref(f)))
    return freq, f.value


def rope(q, k, positions, freqs, *, interleaved: bool = False, factor: float = 1.0, transpose: bool = False,
         q_out=None, k_out=None, stream=None):
    """Rotary positions of q [n, Hq, D] and k [n, Hkv, D] (k may be None) in one launch -> (q_out, k_out).
    positions int32 / int64 CUDA [n]; freqs float64 CUDA [rot/2]; channels from rot on are copied.  The outputs may
    be q and k themselves.  transpose=True turns back: the gradient of the call without it, which autograd takes where
    q or k requires one (then without q_out and k_out; freqs get none)."""
    torch = _torch()
    if q.requires_grad or freqs.requires_grad or (k is not None and k.requires_grad):
        if torch.is_grad_enabled():
            return _rope_with_gradient(q, k, positions, freqs, interleaved, factor, transpose, q_out, k_out, stream)
    if freqs.dtype is not torch.float64 or freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError("freqs must be a contiguous float64 tensor [rot/2]")
    n, wide = q.shape[0], positions.dtype is torch.int64
    if not (wide or positions.dtype is torch.int32) or positions.shape != (n,) or not positions.is_contiguous():
        raise ValueError("positions must be a contiguous int32 or int64 tensor [n]")
    q_out, args = _rope_side(q, q_out, q, stream)
    count = 1
    if k is not None:
        k_out, more = _rope_side(k, k_out, q, stream)
        args += more
        count = 2
    _on_current_device(q, k, positions, freqs, q_out, k_out)
    _check(lib().tq_rope(_ROPE_SIDES[count].pack(*args), count, _dtype_code(q), n, q.shape[2], 2 * freqs.shape[0],
                         freqs.data_ptr(), positions.data_ptr(), 64 if wide else 32, factor,
                         (1 if interleaved else 0) | (2 if transpose else 0), _raw_stream(stream)))
    return q_out, k_out


def _rope_with_gradient(q, k, positions, freqs, interleaved, factor, transpose, q_out, k_out, stream):
    if q_out is not None or k_out is not None:
        raise ValueError("q_out and k_out cannot be given where q or k requires a gradient")
    if freqs.requires_grad:
        raise ValueError("freqs must not require a gradient: none is formed for them")
    with _on(stream):           # (autograd runs a backward pass on the stream that was current in the forward pass)
        y = _rope_function().apply(q, k, positions, freqs, interleaved, factor, transpose)
    return y if k is not None else (y, None)


def _rope_function():
    global _RopeFunction
    if _RopeFunction is None:
        torch = _torch()

        class _RopeFunction(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, positions, freqs, interleaved, factor, transpose):
                ctx.save_for_backward(positions, freqs)
                ctx.how = interleaved, factor, transpose
                ctx.set_materialize_grads(False)
                q_out, k_out = rope(q, k, positions, freqs, interleaved=interleaved, factor=factor, transpose=transpose)
                if k is None:
                    return q_out
                ctx.mark_non_differentiable(*(y for y, need in zip((q_out, k_out), ctx.needs_input_grad) if not need))
                return q_out, k_out

            @staticmethod
            def backward(ctx, gq, gk=None):
                # the transposed rotation of each gradient that is asked for, in one launch
                positions, freqs = ctx.saved_tensors
                interleaved, factor, transpose = ctx.how
                gq, gk = (g if need else None for g, need in zip((gq, gk), ctx.needs_input_grad))
                given = [g if g.stride(-1) == 1 else g.contiguous() for g in (gq, gk) if g is not None]
                back = iter(())
                if given:
                    back = iter(rope(given[0], given[1] if len(given) > 1 else None, positions, freqs,
                                     interleaved=interleaved, factor=factor, transpose=not transpose))
                return (*(None if g is None else next(back) for g in (gq, gk)), None, None, None, None, None)
    return _RopeFunction


_RopeFunction = None
_ROPE_SIDES = {n: struct.Struct("@" + n * "PPi4xqqqq") for n in (1, 2)}     # tq_rope_tensor, n times


def _rope_side(x, out, q, stream):
    """(output, fields of a tq_rope_tensor) of one tensor of the call."""
    if out is None:
        if stream is None:
            out = _torch().empty_like(x)
        else:
            with _on(stream):
                out = _torch().empty_like(x)
    shape = x.shape
    if len(shape) != 3 or shape[0] != q.shape[0] or shape[2] != q.shape[2] or out.shape != shape \
            or x.dtype is not q.dtype or out.dtype is not q.dtype:
        raise ValueError("q, k and their outputs must be [n, heads, D] of one dtype")
    xt, xh, xc = x.stride()
    ot, oh, oc = out.stride()
    if (xc != 1 or oc != 1) and shape.numel():
        raise ValueError("q, k and their outputs must have unit stride along channels")
    if ((ot == 0 and shape[0] > 1) or (oh == 0 and shape[1] > 1)) and shape.numel():
        raise ValueError("an output must not be expanded")
    return out, (x.data_ptr(), out.data_ptr(), shape[1], xt, xh, ot, oh)


def alloc_page_bounds(npages: int, Hkv: int, D: int, dtype, device=None):
    """Bounds of a paged cache's keys, [npages, Hkv, 2, D] (minimum, maximum): kept by page_bounds."""
    torch = _torch()
    return torch.zeros((npages, Hkv, 2, D), dtype=dtype, device=device or torch.device("cuda", torch.cuda.current_device()))


def page_bounds(k, cu_new, start, block_table, page_tokens: int, bounds, max_new: int, stream=None):
    """Fold the new keys k [rows, Hkv, D] into the bounds of their pages (in place) -> bounds.  Sequence b appends
    rows cu_new[b] .. cu_new[b+1]-1 as its tokens start[b], ...; max_new >= the largest number of new rows."""
    if k.dim() != 3 or k.stride(2) != 1 or bounds.dtype != k.dtype or not bounds.is_contiguous() \
            or bounds.dim() != 4 or bounds.shape[1:] != (k.shape[1], 2, k.shape[2]):
        raise ValueError("k must be [rows, Hkv, D] with unit stride along channels, bounds contiguous [pages, Hkv, 2, D] of its dtype")
    B = start.shape[0]
    _int32(start, (B,), "start")
    _int32(cu_new, (B + 1,), "cu_new")
    _int32(block_table, (B, block_table.shape[-1]), "block_table")
    _on_current_device(k, cu_new, start, block_table, bounds)
    _check(lib().tq_page_bounds(k.data_ptr(), k.shape[0], _dtype_code(k), k.stride(0), k.stride(1), cu_new.data_ptr(), start.data_ptr(),
                                B, k.shape[1], k.shape[2], int(max_new), block_table.data_ptr(), int(page_tokens),
                                block_table.shape[1], bounds.data_ptr(), bounds.shape[0], _raw_stream(stream)))
    return bounds


def _on(stream):
    """Allocations and copies of a call belong to the stream that it runs on."""
    return contextlib.nullcontext() if stream is None else _torch().cuda.stream(stream)


class _CachePlan:
    """Pre-marshalled caches of the calls below (as DecodePlan keeps them)."""

    def __init__(self, kctx, vctx, group_off, kcache, vcache, B, Hq, Hkv, D, max_len):
        G = len(kctx)
        self.G, self.B, self.Hq, self.Hkv, self.D, self.max_len = G, B, Hq, Hkv, D, max_len
        self._k = (ctypes.c_void_p * G)(*[c.handle.value for c in kctx])
        self._v = (ctypes.c_void_p * G)(*[c.handle.value for c in vctx])
        self._off = (ctypes.c_int * (G + 1))(*list(group_off))
        self._kc = (_Packed * G)(*[p.struct() for p in kcache])
        self._vc = (_Packed * G)(*[p.struct() for p in vcache])
        self._keep = (kctx, vctx, kcache, vcache)
        self.device = kcache[0].codes.device
        for p in (*kcache, *vcache):
            self._same_device(p.codes, p.norm, p.rnorm)
        self._streams = {_raw_stream(None)}          # where the plan's own tensors are at home, or recorded

    def _used_on(self, stream, *own):
        """The plan may be dropped while a call runs: its tensors' memory is then not to be used again before the call's
        stream, the given or the current one, is through with it."""
        raw = _raw_stream(stream)
        if raw not in self._streams:
            for t in own:
                t.record_stream(stream if stream is not None else _torch().cuda.current_stream())
            self._streams.add(raw)

    def _workspace(self, need):
        return _torch().empty(max(need, 1), dtype=_torch().uint8, device=self.device)

    def _same_device(self, *tensors):
        for t in tensors:
            if t is not None and t.device != self.device:
                raise ValueError("expected tensors on the caches' device (%s), got one on %s" % (self.device, t.device))

    def _query(self, q, shape, out, stream):
        if q.shape != shape:
            raise ValueError("q must be %s, got %s" % (shape, tuple(q.shape)))
        if out is None or not q.is_contiguous():
            with _on(stream):
                q = q.contiguous()
                if out is None:
                    return q, _torch().empty_like(q)
        if out.shape != shape or out.dtype is not q.dtype or not out.is_contiguous():
            raise ValueError("out must be contiguous, with the shape and dtype of q")
        return q, out


def sparse_workspace_size(B, Hq, Hkv, D, ngroups, max_len, page_tokens, select) -> int:
    return int(lib().tq_sparse_workspace_size(B, Hq, Hkv, D, ngroups, max_len, page_tokens, select))


class SparsePlan(_CachePlan):
    """Caches, block table and workspace of tq_sparse_decode_attention.  Calls that may overlap (on several streams,
    or captured into several graphs) need a plan each: they share its workspace and its `selected`."""

    def __init__(self, kctx: Sequence[Context], vctx: Sequence[Context], group_off: Sequence[int],
                 kcache: Sequence[Packed], vcache: Sequence[Packed], B, Hq, Hkv, D, max_len, *, block_table,
                 page_tokens: int, select: int, first: int = 1, last: int = 1, channel_perm=None):
        super().__init__(kctx, vctx, group_off, kcache, vcache, B, Hq, Hkv, D, max_len)
        torch = _torch()
        if page_tokens <= 0 or max_len % page_tokens != 0:
            raise ValueError("page_tokens must divide max_len")
        _int32(block_table, (B, max_len // page_tokens), "block_table")
        if channel_perm is not None:
            _int32(channel_perm, (Hkv, D), "channel_perm")
        self._same_device(block_table, channel_perm)
        self.select = int(select)
        self.selected = torch.empty((B, Hkv, max(self.select, 1)), dtype=torch.int32, device=self.device)
        self._opts = _SparseOpts(0, 0, 0, self.select, int(first), int(last), self.selected.data_ptr(),
                                 block_table.data_ptr(), int(page_tokens),
                                 0 if channel_perm is None else channel_perm.data_ptr())
        self._keep_opts = (block_table, channel_perm)
        self.workspace = self._workspace(sparse_workspace_size(B, Hq, Hkv, D, self.G, max_len, page_tokens, self.select))

    def __call__(self, q, bounds, seq_lens, scale: float, out=None, stream=None):
        """q [B, Hq, D] -> (out [B, Hq, D] of q's dtype, selected int32 [B, Hkv, select]: the plan's own tensor).
        No gradient is formed, as for decode_attention."""
        q, out = self._query(q, (self.B, self.Hq, self.D), out, stream)
        self._used_on(stream, self.workspace, self.selected)
        if bounds.dim() != 4 or bounds.shape[1:] != (self.Hkv, 2, self.D) or not bounds.is_contiguous():
            raise ValueError("bounds must be contiguous [pages, Hkv, 2, D]")
        _int32(seq_lens, (self.B,), "seq_lens")
        _on_current_device(q, bounds, seq_lens, out, self.workspace)      # (the caches are where the workspace is)
        o = self._opts
        o.bounds, o.bounds_dtype, o.bounds_pages = bounds.data_ptr(), _dtype_code(bounds), bounds.shape[0]
        _check(lib().tq_sparse_decode_attention(
            self._k, self._v, self._off, self.G, q.data_ptr(), _dtype_code(q), self._kc, self._vc, seq_lens.data_ptr(),
            self.B, self.Hq, self.Hkv, self.D, self.max_len, scale, out.data_ptr(), ctypes.byref(o),
            self.workspace.data_ptr(), self.workspace.numel(), _raw_stream(stream)))
        return out, self.selected


def sparse_decode_attention(kctx, vctx, group_off, q, bounds, kcache, vcache, seq_lens, Hkv, max_len, scale, *,
                            block_table, page_tokens, select, first=1, last=1, out=None, stream=None, channel_perm=None):
    """One decode step over the pages that their key bounds select -> (out, selected); see tq.h."""
    B, Hq, D = q.shape
    with _on(stream):
        plan = SparsePlan(kctx, vctx, group_off, kcache, vcache, B, Hq, Hkv, D, max_len, block_table=block_table,
                          page_tokens=page_tokens, select=select, first=first, last=last, channel_perm=channel_perm)
    return plan(q, bounds, seq_lens, scale, out, stream)


def tree_workspace_size(B, T, Hq, Hkv, D, ngroups, max_len) -> int:
    return int(lib().tq_tree_workspace_size(B, T, Hq, Hkv, D, ngroups, max_len))


def tree_mask(parents) -> np.ndarray:
    """Masks of drafted trees: parents int [B, T] (or [T]), each in [-1, j) -> int64 [B, T, ceil(T / 64)] with bit i of
    row j set where i is j or one of its ancestors (move it to the GPU with torch.from_numpy)."""
    p = np.ascontiguousarray(parents, dtype=np.int32)
    p = p[None] if p.ndim == 1 else p
    if p.ndim != 2:
        raise ValueError("parents must be [B, T] or [T]")
    B, T = p.shape
    m = np.zeros((B, T, (T + 63) // 64), dtype=np.int64)
    _check(lib().tq_tree_mask(p.ctypes.data_as(ctypes.c_void_p), B, T, m.ctypes.data_as(ctypes.c_void_p)))
    return m


class TreePlan(_CachePlan):
    """Caches, block table and workspace of tq_tree_attention.  Calls that may overlap (on several streams, or captured
    into several graphs) need a plan each: they share its workspace."""

    def __init__(self, kctx: Sequence[Context], vctx: Sequence[Context], group_off: Sequence[int],
                 kcache: Sequence[Packed], vcache: Sequence[Packed], B, T, Hq, Hkv, D, max_len, *, channel_perm=None,
                 block_table=None, page_tokens: int = 0):
        super().__init__(kctx, vctx, group_off, kcache, vcache, B, Hq, Hkv, D, max_len)
        self.T = int(T)
        if block_table is not None:
            if page_tokens <= 0 or max_len % page_tokens != 0:
                raise ValueError("page_tokens must divide max_len")
            _int32(block_table, (B, max_len // page_tokens), "block_table")
        if channel_perm is not None:
            _int32(channel_perm, (Hkv, D), "channel_perm")
        self._same_device(block_table, channel_perm)
        self._opts = _DecodeOpts(0 if channel_perm is None else channel_perm.data_ptr(),
                                 0 if block_table is None else block_table.data_ptr(), int(page_tokens))
        self._keep_opts = (channel_perm, block_table)
        self.workspace = self._workspace(tree_workspace_size(B, self.T, Hq, Hkv, D, self.G, max_len))

    def __call__(self, q, seq_lens, draft_lens, mask, scale: float, out=None, stream=None):
        """q [B, T, Hq, D] -> out of its shape and dtype.  draft_lens int32 [B] or None (T each); mask int64
        [B, T, ceil(T / 64)] (tree_mask) or None (a chain).  No gradient is formed, as for decode_attention."""
        torch = _torch()
        q, out = self._query(q, (self.B, self.T, self.Hq, self.D), out, stream)
        self._used_on(stream, self.workspace)
        _int32(seq_lens, (self.B,), "seq_lens")
        if draft_lens is not None:
            _int32(draft_lens, (self.B,), "draft_lens")
        if mask is not None and (mask.dtype is not torch.int64 or not mask.is_contiguous()
                                 or mask.shape != (self.B, self.T, (self.T + 63) // 64)):
            raise ValueError("mask must be a contiguous int64 tensor [B, T, ceil(T / 64)]")
        _on_current_device(q, seq_lens, draft_lens, mask, out, self.workspace)      # (the caches are where the workspace is)
        _check(lib().tq_tree_attention(
            self._k, self._v, self._off, self.G, q.data_ptr(), _dtype_code(q), self._kc, self._vc, seq_lens.data_ptr(),
            None if draft_lens is None else draft_lens.data_ptr(), None if mask is None else mask.data_ptr(), self.B, self.T, self.Hq, self.Hkv, self.D, self.max_len, scale, out.data_ptr(),
            ctypes.byref(self._opts), self.workspace.data_ptr(), self.workspace.numel(), _raw_stream(stream)))
        return out


def tree_attention(kctx, vctx, group_off, q, kcache, vcache, seq_lens, Hkv, max_len, scale, draft_lens=None, mask=None,
                   out=None, stream=None, channel_perm=None, block_table=None, page_tokens=0):
    """Attention of T drafted tokens per sequence, the last ones of its cache, under a tree mask; q [B, T, Hq, D] -> out
    of its shape and dtype (see tq.h)."""
    B, T, Hq, D = q.shape
    with _on(stream):
        plan = TreePlan(kctx, vctx, group_off, kcache, vcache, B, T, Hq, Hkv, D, max_len, channel_perm=channel_perm,
                        block_table=block_table, page_tokens=page_tokens)
    return plan(q, seq_lens, draft_lens, mask, scale, out, stream)
