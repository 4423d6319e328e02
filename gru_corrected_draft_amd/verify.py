"""Operators around the verification of a draft block: a paged key-value cache with the attention
that reads it, and the rules on the target's logits with the acceptance of the proposals.

Thin ctypes binding of ``include/domino_verify.h``; the mathematics of each operator stands there.
``PagedAttention`` and ``DraftVerifier`` marshal tensors: every argument is checked for type, shape,
device and layout, work goes to the current stream of the tensors' device, and the handle must not
be used by two threads at once, nor on two streams whose work is not ordered.  A handle belongs to the
GPU that is current where it is made, and takes tensors of that GPU alone.  Importing this module needs
the built library; there is no fallback.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import rollout as _rollout
from .rollout import DTYPE_BF16, DTYPE_FP32, DominoError

_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_FP32}
_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class AttentionConfig(ctypes.Structure):
    _fields_ = [(n, _i32) for n in
                ("q_heads", "kv_heads", "head_dim", "page_size", "max_requests", "dtype")]


class CacheArgs(ctypes.Structure):
    _fields_ = [("k_cache", _vp), ("v_cache", _vp), ("page_stride", _i64), ("head_stride", _i64),
                ("row_stride", _i64), ("num_pages", _i32), ("page_table", _vp), ("table_stride", _i64),
                ("table_width", _i32), ("kv_len", _vp), ("q_start", _vp), ("requests", _i32),
                ("tokens", _i32), ("max_new", _i32), ("max_kv", _i32)]


class VerifyConfig(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("vocab", "max_requests", "max_rows", "dtype")]


class LogitsArgs(ctypes.Structure):
    _fields_ = [("logits", _vp), ("request_stride", _i64), ("row_stride", _i64), ("requests", _i32),
                ("rows", _i32), ("draft", _vp), ("draft_stride", _i64), ("draft_len", _vp),
                ("history", _vp), ("history_stride", _i64), ("history_width", _i32),
                ("history_len", _vp), ("prompt_len", _vp), ("repetition", _vp), ("frequency", _vp),
                ("presence", _vp), ("bias_ids", _vp), ("bias_values", _vp), ("bias_stride", _i64),
                ("bias_width", _i32), ("bias_len", _vp), ("mask", _vp),
                ("mask_request_stride", _i64), ("mask_row_stride", _i64)]


_lib = None


def load_library():
    """The in-tree library with this module's functions declared (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    lib = _rollout.load_library()
    p = ctypes.POINTER
    lib.domino_attention_create.argtypes = [p(AttentionConfig), p(_vp)]
    lib.domino_attention_append.argtypes = [_vp, p(CacheArgs), _vp, _i64, _i64, _vp, _i64, _i64, _vp]
    lib.domino_attention_run.argtypes = [_vp, p(CacheArgs), _vp, _i64, _i64, _i32, _i32, _f32, _vp,
                                         _i64, _i64, _vp, _vp]
    lib.domino_verify_create.argtypes = [p(VerifyConfig), p(_vp)]
    lib.domino_verify_process.argtypes = [_vp, p(LogitsArgs), _vp, _i64, _i64, _vp]
    lib.domino_verify_run.argtypes = [_vp, p(LogitsArgs), _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp]
    for name in ("domino_attention_create", "domino_attention_append", "domino_attention_run",
                 "domino_verify_create", "domino_verify_process", "domino_verify_run"):
        getattr(lib, name).restype = ctypes.c_int
    for name in ("domino_attention_destroy", "domino_verify_destroy"):
        getattr(lib, name).argtypes = [_vp]
        getattr(lib, name).restype = None
    for name in ("domino_attention_last_error", "domino_verify_last_error"):
        getattr(lib, name).argtypes = [_vp]
        getattr(lib, name).restype = ctypes.c_char_p
    _lib = lib
    return lib


def _fits(t, dtype, shape, index):
    """The quick check of a call that is in order: type, shape and GPU of a tensor."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == index


def _want(name, t, dtype, shape, index):
    """Refuses a tensor that is not of this type and shape on GPU ``index``, its last dimension contiguous."""
    if t.dtype != dtype or tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if index < 0:
        raise ValueError("tensors must be on a GPU")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if shape and shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _int32(name, x):
    """Refuses what ctypes would cut to 32 bits without a word (2 ** 32 + 64 would become 64)."""
    if not -2147483648 <= x < 2147483648:
        raise ValueError(f"{name} must be a 32-bit number, got {x}")
    return x


# the current stream's address without a Stream object around it (a call's checks and arguments take
# about as long on the host as its kernel on the GPU, so each microsecond shows)
_stream = torch._C._cuda_getCurrentRawStream


class _Handle:
    def __init__(self, kind, cfg):
        self.lib = load_library()
        self._destroy = getattr(self.lib, f"domino_{kind}_destroy")
        self._error = getattr(self.lib, f"domino_{kind}_last_error")
        h = _vp()
        st = getattr(self.lib, f"domino_{kind}_create")(ctypes.byref(cfg), ctypes.byref(h))
        if st:
            raise DominoError(st, self._error(None).decode())
        self.handle = h
        self.index = torch.cuda.current_device()  # the GPU that the handle's workspace is on

    def _check(self, st):
        if st:
            raise DominoError(st, self._error(self.handle).decode())

    def _elsewhere(self, index):
        return ValueError(f"the handle is on cuda:{self.index}, the tensors on cuda:{index}")

    def close(self):
        if getattr(self, "handle", None):
            self._destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PagedAttention(_Handle):
    """Key-value cache in pages and the attention of new tokens over it.

    ``k_cache`` and ``v_cache`` are [pages, kv_heads, page_size, head_dim] tensors of the handle's
    dtype with the same strides and a contiguous last dimension; any order of the other three in
    memory will do (a permuted view of [pages, page_size, kv_heads, head_dim], a half of a tensor that
    holds both).  ``page_table`` is [requests, width], ``kv_len`` [requests] with the new tokens
    counted, ``q_start`` [requests + 1] the first token row of each request: int32 on the device,
    read by the kernels alone.  ``max_new`` and ``max_kv`` bound the new tokens and the cache length of
    a request; they default to what the arguments allow, and kernels are faster with tighter ones.
    """

    def __init__(self, q_heads, kv_heads, head_dim, page_size, dtype=torch.bfloat16, max_requests=64):
        if dtype not in _DTYPES:
            raise TypeError("dtype must be torch.bfloat16 or torch.float32")
        sizes = dict(q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page_size=page_size, max_requests=max_requests)
        super().__init__("attention", AttentionConfig(*(_int32(n, x) for n, x in sizes.items()), _DTYPES[dtype]))
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.page_size, self.dtype = page_size, dtype
        self._scale = 1.0 / math.sqrt(head_dim)

    def _cache(self, k_cache, v_cache, page_table, kv_len, q_start, tokens, max_new, max_kv, index):
        shape = (k_cache.shape[0] if k_cache.dim() else 0, self.kv_heads, self.page_size, self.head_dim)
        strides = k_cache.stride()
        b, width = page_table.shape if page_table.dim() == 2 else (-1, -1)
        if not (_fits(k_cache, self.dtype, shape, index) and _fits(v_cache, self.dtype, shape, index)
                and v_cache.stride() == strides and strides[3] == 1 and index == self.index
                and _fits(page_table, torch.int32, (b, width), index) and _fits(kv_len, torch.int32, (b,), index)
                and _fits(q_start, torch.int32, (b + 1,), index) and page_table.stride(1) == 1
                and kv_len.stride(0) == 1 and q_start.stride(0) == 1):
            _want("k_cache", k_cache, self.dtype, shape, index)
            _want("v_cache", v_cache, self.dtype, shape, index)
            if v_cache.stride() != strides:
                raise ValueError("k_cache and v_cache must have the same strides")
            _want("page_table", page_table, torch.int32, (b, width), index)
            _want("kv_len", kv_len, torch.int32, (b,), index)
            _want("q_start", q_start, torch.int32, (b + 1,), index)
            if index != self.index:
                raise self._elsewhere(index)
        if max_new is None:
            max_new = tokens
        if max_kv is None:
            max_kv = min(width * self.page_size, 2 ** 31 - 1)
        if (max_new | max_kv) >> 31:  # negative ones are the library's to refuse
            _int32("max_new", max_new)
            _int32("max_kv", max_kv)
        return CacheArgs(k_cache.data_ptr(), v_cache.data_ptr(), strides[0], strides[1], strides[2], shape[0],
                         page_table.data_ptr(), page_table.stride(0), width, kv_len.data_ptr(),
                         q_start.data_ptr(), b, tokens, max_new, max_kv)

    def append(self, k, v, k_cache, v_cache, page_table, kv_len, q_start, max_new=None, max_kv=None):
        """Write the new tokens' ``k`` and ``v`` ([tokens, kv_heads, head_dim]) into the cache."""
        tokens, index = k.shape[0], k.get_device()
        shape = (tokens, self.kv_heads, self.head_dim)
        ks, vs = k.stride(), v.stride()
        if not (_fits(k, self.dtype, shape, index) and _fits(v, self.dtype, shape, index)
                and ks[2] == 1 and vs[2] == 1):
            _want("k", k, self.dtype, shape, index)
            _want("v", v, self.dtype, shape, index)
        c = self._cache(k_cache, v_cache, page_table, kv_len, q_start, tokens, max_new, max_kv, index)
        st = self.lib.domino_attention_append(self.handle, ctypes.byref(c), k.data_ptr(), ks[0], ks[1],
                                              v.data_ptr(), vs[0], vs[1], _stream(index))
        if st:
            self._check(st)

    def run(self, q, k_cache, v_cache, page_table, kv_len, q_start, max_new=None, max_kv=None, window=0,
            sinks=0, scale=None, out=None, return_lse=False):
        """Attention of the new tokens' ``q`` ([tokens, q_heads, head_dim]); returns ``out`` of the
        same shape, or (out, lse) with lse [tokens, q_heads] fp32.  ``window`` = 0 sees the whole
        cache; otherwise a token sees the last ``window`` positions up to its own and the first
        ``sinks``.  ``scale`` defaults to head_dim ** -0.5.  Rows of ``out`` that belong to no request
        are left as they are."""
        tokens, index = q.shape[0], q.get_device()
        shape = (tokens, self.q_heads, self.head_dim)
        qs = q.stride()
        if not (_fits(q, self.dtype, shape, index) and qs[2] == 1):
            _want("q", q, self.dtype, shape, index)
        c = self._cache(k_cache, v_cache, page_table, kv_len, q_start, tokens, max_new, max_kv, index)
        if (window | sinks) >> 31:
            _int32("window", window)
            _int32("sinks", sinks)
        if out is None:
            out = torch.empty(shape, dtype=self.dtype, device=q.device)
        else:
            _want("out", out, self.dtype, shape, index)
        lse = torch.empty(shape[:2], dtype=torch.float32, device=q.device) if return_lse else None
        os = out.stride()
        st = self.lib.domino_attention_run(
            self.handle, ctypes.byref(c), q.data_ptr(), qs[0], qs[1], window, sinks,
            self._scale if scale is None else scale, out.data_ptr(), os[0], os[1],
            lse.data_ptr() if return_lse else None, _stream(index))
        if st:
            self._check(st)
        return (out, lse) if return_lse else out


class DraftVerifier(_Handle):
    """Rules on the target's logits and the acceptance of a draft block.

    ``logits`` is [requests, rows, vocab] in the handle's dtype, rows and requests at any stride, row
    t scoring what follows the request's text and its first t proposals; ``draft`` [requests, rows - 1]
    int32 (or None: no proposals), of which ``draft_len`` [requests] int32 gives those in use.  Rules,
    each optional: ``history`` [requests, width] int32 with ``history_len`` and ``prompt_len``
    [requests] int32 (the first prompt_len entries are the prompt); ``repetition``, ``frequency``,
    ``presence`` [requests] fp32; ``bias_ids`` and ``bias_values`` [requests, n] with ``bias_len``;
    ``mask`` [requests, rows, ceil(vocab / 32)] int32 whose bit v % 32 of word v / 32 allows id v
    (expanded views share a mask between rows or requests).
    """

    def __init__(self, vocab, dtype=torch.bfloat16, max_requests=64, max_rows=16):
        if dtype not in _DTYPES:
            raise TypeError("dtype must be torch.bfloat16 or torch.float32")
        sizes = dict(vocab=vocab, max_requests=max_requests, max_rows=max_rows)
        super().__init__("verify", VerifyConfig(*(_int32(n, x) for n, x in sizes.items()), _DTYPES[dtype]))
        self.vocab, self.dtype = vocab, dtype

    def _args(self, logits, draft, draft_len, history, history_len, prompt_len, repetition, frequency,
              presence, bias_ids, bias_values, bias_len, mask):
        if logits.dim() != 3:
            raise ValueError("logits must be [requests, rows, vocab]")
        b, rows, _ = logits.shape
        ls, index, i32, f32 = logits.stride(), logits.get_device(), torch.int32, torch.float32

        def take(name, t, dtype, shape):
            if not (_fits(t, dtype, shape, index) and t.stride(-1) == 1):
                _want(name, t, dtype, shape, index)
            return t.data_ptr()

        take("logits", logits, self.dtype, (b, rows, self.vocab))
        a = LogitsArgs(logits.data_ptr(), ls[0], ls[1], b, rows)
        if index != self.index:
            raise self._elsewhere(index) if index >= 0 else ValueError("tensors must be on a GPU")
        if draft is not None and rows > 1:
            a.draft, a.draft_stride = take("draft", draft, i32, (b, rows - 1)), draft.stride(0)
        if history is not None:
            width = history.shape[1] if history.dim() == 2 else -1
            a.history, a.history_stride = take("history", history, i32, (b, width)), history.stride(0)
            a.history_width = width
        if (bias_ids is None) != (bias_values is None):
            raise ValueError("bias_ids and bias_values must be given together")
        if bias_ids is not None:
            width = bias_ids.shape[1] if bias_ids.dim() == 2 else -1
            a.bias_ids = take("bias_ids", bias_ids, i32, (b, width))
            a.bias_values = take("bias_values", bias_values, f32, (b, width))
            if b > 1 and bias_ids.stride(0) != bias_values.stride(0):
                raise ValueError("bias_ids and bias_values must have the same strides")
            a.bias_stride, a.bias_width = bias_ids.stride(0), width
        per_request = (b,)
        if draft_len is not None:
            a.draft_len = take("draft_len", draft_len, i32, per_request)
        if history_len is not None:
            a.history_len = take("history_len", history_len, i32, per_request)
        if prompt_len is not None:
            a.prompt_len = take("prompt_len", prompt_len, i32, per_request)
        if bias_len is not None:
            a.bias_len = take("bias_len", bias_len, i32, per_request)
        if repetition is not None:
            a.repetition = take("repetition", repetition, f32, per_request)
        if frequency is not None:
            a.frequency = take("frequency", frequency, f32, per_request)
        if presence is not None:
            a.presence = take("presence", presence, f32, per_request)
        if mask is not None:
            a.mask = take("mask", mask, i32, (b, rows, (self.vocab + 31) // 32))
            a.mask_request_stride, a.mask_row_stride = mask.stride(0), mask.stride(1)
        return a

    def process(self, logits, draft=None, draft_len=None, history=None, history_len=None, prompt_len=None,
                repetition=None, frequency=None, presence=None, bias_ids=None, bias_values=None,
                bias_len=None, mask=None, out=None):
        """The processed logits, rounded once to the handle's dtype.  ``out`` may be ``logits``."""
        a = self._args(logits, draft, draft_len, history, history_len, prompt_len, repetition, frequency,
                       presence, bias_ids, bias_values, bias_len, mask)
        index = logits.get_device()
        if out is None:
            out = torch.empty(logits.shape, dtype=self.dtype, device=logits.device)
        else:
            _want("out", out, self.dtype, tuple(logits.shape), index)
            if out.data_ptr() == logits.data_ptr() and out.stride() != logits.stride():
                raise ValueError("out over the logits must have their strides")
        os = out.stride()
        st = self.lib.domino_verify_process(self.handle, ctypes.byref(a), out.data_ptr(), os[0], os[1],
                                            _stream(index))
        if st:
            self._check(st)
        return out

    def run(self, logits, draft=None, draft_len=None, temperature=None, accept_u=None, noise=None,
            history=None, history_len=None, prompt_len=None, repetition=None, frequency=None,
            presence=None, bias_ids=None, bias_values=None, bias_len=None, mask=None,
            return_logprob=False):
        """Accept proposals and choose the token after them; returns (tokens [requests, rows] int32,
        accepted [requests] int32), and logprob [requests, rows] fp32 if asked for.  ``temperature``
        [requests] fp32 (None: greedy) needs ``noise`` [requests, vocab] fp32 drawn from the unit
        exponential and, with proposals, ``accept_u`` [requests, rows - 1] fp32 uniform in [0, 1)."""
        a = self._args(logits, draft, draft_len, history, history_len, prompt_len, repetition, frequency,
                       presence, bias_ids, bias_values, bias_len, mask)
        b, rows, index, dev = a.requests, a.rows, logits.get_device(), logits.device
        temp = u = n = None
        u_stride = n_stride = 0
        if temperature is not None:
            _want("temperature", temperature, torch.float32, (b,), index)
            temp = temperature.data_ptr()
            if noise is None or (accept_u is None and a.draft):
                raise ValueError("temperature needs noise, and accept_u where there are proposals")
            _want("noise", noise, torch.float32, (b, self.vocab), index)
            n, n_stride = noise.data_ptr(), noise.stride(0)
            if a.draft:
                _want("accept_u", accept_u, torch.float32, (b, rows - 1), index)
                u, u_stride = accept_u.data_ptr(), accept_u.stride(0)
        tokens = torch.empty((b, rows), dtype=torch.int32, device=dev)
        accepted = torch.empty((b,), dtype=torch.int32, device=dev)
        logprob = torch.empty((b, rows), dtype=torch.float32, device=dev) if return_logprob else None
        st = self.lib.domino_verify_run(self.handle, ctypes.byref(a), temp, u, u_stride, n, n_stride,
                                        tokens.data_ptr(), accepted.data_ptr(),
                                        logprob.data_ptr() if return_logprob else None, _stream(index))
        if st:
            self._check(st)
        return (tokens, accepted, logprob) if return_logprob else (tokens, accepted)
