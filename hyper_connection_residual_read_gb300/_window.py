"""Binding of the verify-window operators: the C ABI of include/hc_window.h, same names.

Argument marshalling only, as in ``_lib``: sizes, types and strides are read off the
tensors, whose shapes must agree; everything else is checked by the library. Shapes
that disagree, tensors that are not laid out as the header says and unsupported types
raise ``HcReadError`` with ``HC_ERR_ARG``, as the library's own refusals do.

The calls go through a small CPython module (``_hcpywindow``, built with the library) that
reads the tensors in C: the same work in Python took 13 us a call, three times the launch
itself. Where that module was not built, they go through ctypes.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._lib import HC_ERR_ARG, HC_OK, HcReadError
from ._lib import _stream as _any_stream

HC_DTYPE_BF16 = 0
HC_DTYPE_FP16 = 1
HC_DTYPE_FP32 = 2

HC_PLAN_MAX_REQUESTS = 8192
HC_KV4_MAX_BLOCK = 256
HC_KV4_MAX_GROUP = 128
HC_KV4_MAX_MASKED = 64
HC_LOGPROBS_MAX_TOP = 32

# every symbol include/hc_window.h declares
WINDOW_EXPORTS = ("hc_window_plan", "hc_kv4_append", "hc_kv4_load", "hc_kv4_attention",
                  "hc_token_logprobs")

_DTYPES = {torch.bfloat16: HC_DTYPE_BF16, torch.float16: HC_DTYPE_FP16, torch.float32: HC_DTYPE_FP32}
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32


class hc_kv4_cache(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("blocks", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("block_size", ctypes.c_int), ("head_dim", ctypes.c_int)]


_bound = None
_call = None         # the _hcpywindow module, bound to the library's entry points


def _stream(stream):
    """As ``_lib``'s, with the current stream's handle read directly (torch's stream object
    costs 3 us)."""
    if stream is None and torch.cuda.is_initialized():
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return _any_stream(stream)


def _bind_call(lib) -> None:
    global _call
    try:
        from . import _hcpywindow
    except ImportError:
        return
    addr = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    _hcpywindow.bind(*[addr(getattr(lib, name)) for name in WINDOW_EXPORTS], torch.bfloat16,
                     torch.float16, torch.float32, torch.int32, torch.int64, torch.uint8)
    _call = _hcpywindow


def _load():
    global _bound
    if _bound is not None:
        return _bound
    lib = _lib.load()
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    cache = ctypes.POINTER(hc_kv4_cache)
    lib.hc_window_plan.argtypes = [i32] * 5 + [vp] * 12
    lib.hc_kv4_append.argtypes = [cache, i32, i32, vp, i64, i64, vp, i64, i64, vp, vp]
    lib.hc_kv4_load.argtypes = [cache, i32, vp, i32, vp, vp, vp]
    lib.hc_kv4_attention.argtypes = [cache] + [i32] * 5 + [ctypes.c_float, i32, vp, i64, i64] + [vp] * 7
    lib.hc_token_logprobs.argtypes = [i32] * 4 + [vp, i64] + [vp] * 8
    for name in WINDOW_EXPORTS:
        getattr(lib, name).restype = i32
    _bound = lib
    _bind_call(lib)
    return lib


def _raise(fn: str, code: int) -> None:
    if code != HC_OK:
        raise HcReadError(fn, code)


def _need(fn: str, ok: bool) -> None:
    if not ok:
        raise HcReadError(fn, HC_ERR_ARG)


def _flat(t, dtype, shape) -> bool:
    return t.dtype is dtype and t.shape == shape and t.is_contiguous()


def _cache(fn: str, codes, scales) -> hc_kv4_cache:
    _need(fn, codes.dtype is torch.uint8 and codes.dim() == 5 and codes.is_contiguous())
    blocks, two, heads, size, half = codes.shape
    _need(fn, two == 2 and _flat(scales, torch.bfloat16, (blocks, 2, heads, size, 2)))
    return hc_kv4_cache(codes.data_ptr(), scales.data_ptr(), blocks, heads, size, 2 * half)


def hc_window_plan(cached_lens, new_lens, free_blocks, free_count, block_size, block_table, slots,
                   request_of, positions, cu_lens, kv_lens, free_left, stream=None) -> None:
    """Cache blocks, slots and positions of a step's new tokens from the requests' lengths.
    All int32, but ``slots`` (int64); ``block_table`` [requests][width] is updated."""
    lib, fn = _bound or _load(), "hc_window_plan"
    if _call is not None:
        return _raise(fn, _call.plan(cached_lens, new_lens, free_blocks, free_count, block_size, block_table,
                                slots, request_of, positions, cu_lens, kv_lens, free_left, _stream(stream)))
    n, cap = cached_lens.numel(), slots.numel()
    _need(fn, block_table.dim() == 2 and _flat(block_table, _I32, (n, block_table.shape[1])) and
          _flat(cached_lens, _I32, (n,)) and _flat(new_lens, _I32, (n,)) and
          _flat(free_blocks, _I32, (free_blocks.numel(),)) and _flat(free_count, _I32, (1,)) and
          _flat(slots, _I64, (cap,)) and _flat(request_of, _I32, (cap,)) and
          _flat(positions, _I32, (cap,)) and _flat(cu_lens, _I32, (n + 1,)) and
          _flat(kv_lens, _I32, (n,)) and _flat(free_left, _I32, (1,)))
    code = lib.hc_window_plan(n, block_table.shape[1], block_size, cap, free_blocks.numel(),
                              cached_lens.data_ptr(), new_lens.data_ptr(), free_blocks.data_ptr(),
                              free_count.data_ptr(), block_table.data_ptr(), slots.data_ptr(),
                              request_of.data_ptr(), positions.data_ptr(), cu_lens.data_ptr(),
                              kv_lens.data_ptr(), free_left.data_ptr(), _stream(stream))
    _raise(fn, code)


def hc_kv4_append(k, v, slots, codes, scales, stream=None) -> None:
    """Rounds the keys and values ``k``, ``v`` [tokens][kv heads][head dim] (any strides of
    the first two axes) to 4 bits and writes them to their ``slots`` (int64)."""
    lib, fn = _bound or _load(), "hc_kv4_append"
    if _call is not None:
        return _raise(fn, _call.append(k, v, slots, codes, scales, _stream(stream)))
    cache = _cache(fn, codes, scales)
    shape = k.shape
    _need(fn, k.dtype in _DTYPES and v.dtype is k.dtype and v.shape == shape and len(shape) == 3 and
          shape[1] == cache.kv_heads and shape[2] == cache.head_dim and
          _flat(slots, _I64, (shape[0],)))
    ks, vs = k.stride(), v.stride()
    _need(fn, ks[2] == 1 and vs[2] == 1)
    code = lib.hc_kv4_append(cache, shape[0], _DTYPES[k.dtype], k.data_ptr(), ks[0], ks[1], v.data_ptr(),
                             vs[0], vs[1], slots.data_ptr(), _stream(stream))
    _raise(fn, code)


def hc_kv4_load(slots, codes, scales, k_out, v_out, stream=None) -> None:
    """Reads ``slots`` (int64) back into ``k_out``, ``v_out`` [tokens][kv heads][head dim]."""
    lib, fn = _bound or _load(), "hc_kv4_load"
    if _call is not None:
        return _raise(fn, _call.load(slots, codes, scales, k_out, v_out, _stream(stream)))
    cache = _cache(fn, codes, scales)
    shape = (slots.numel(), cache.kv_heads, cache.head_dim)
    _need(fn, k_out.dtype in _DTYPES and _flat(k_out, k_out.dtype, shape) and
          _flat(v_out, k_out.dtype, shape) and _flat(slots, _I64, (shape[0],)))
    code = lib.hc_kv4_load(cache, shape[0], slots.data_ptr(), _DTYPES[k_out.dtype], k_out.data_ptr(),
                           v_out.data_ptr(), _stream(stream))
    _raise(fn, code)


def hc_kv4_attention(q, codes, scales, block_table, cu_lens, kv_lens, max_new, out, lse=None,
                     mask=None, scale=None, stream=None) -> None:
    """Attention of each request's new tokens ``q`` [tokens][q heads][head dim] (any strides
    of the first two axes) against its cache, into ``out`` (and ``lse``, fp32). ``mask``
    (int64 bits, one word a token) replaces the causal order within the new tokens;
    ``scale`` defaults to 1 / sqrt(head dim)."""
    lib, fn = _bound or _load(), "hc_kv4_attention"
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    if _call is not None:
        return _raise(fn, _call.attention(q, codes, scales, block_table, cu_lens, kv_lens, max_new, out, lse,
                                          mask, scale, _stream(stream)))
    cache = _cache(fn, codes, scales)
    shape = q.shape
    n = kv_lens.numel()
    _need(fn, len(shape) == 3 and shape[2] == cache.head_dim and q.stride(2) == 1 and
          q.dtype in _DTYPES and _flat(out, q.dtype, shape) and
          (lse is None or _flat(lse, _F32, shape[:2])) and
          (mask is None or _flat(mask, _I64, shape[:1])) and block_table.dim() == 2 and
          _flat(block_table, _I32, (n, block_table.shape[1])) and _flat(cu_lens, _I32, (n + 1,)) and
          _flat(kv_lens, _I32, (n,)))
    code = lib.hc_kv4_attention(
        cache, n, shape[0], shape[1], max_new, block_table.shape[1],
        scale, _DTYPES[q.dtype], q.data_ptr(),
        q.stride(0), q.stride(1), cu_lens.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr(),
        None if mask is None else mask.data_ptr(), out.data_ptr(),
        None if lse is None else lse.data_ptr(), _stream(stream))
    _raise(fn, code)


def hc_token_logprobs(logits, tokens, logprob, entropy, lse, rank, top_ids, top_logprobs,
                      stream=None) -> None:
    """Log probabilities of ``tokens`` (int32) under ``logits`` [tokens][vocabulary] (any row
    stride), with the entropy, log-sum-exp, rank, and the ``top_ids.shape[1]`` most likely
    tokens with theirs."""
    lib, fn = _bound or _load(), "hc_token_logprobs"
    if _call is not None:
        return _raise(fn, _call.logprobs(logits, tokens, logprob, entropy, lse, rank, top_ids, top_logprobs,
                                    _stream(stream)))
    _need(fn, logits.dim() == 2 and top_ids.dim() == 2 and logits.dtype in _DTYPES)
    t, vocab = logits.shape
    top = top_ids.shape[1]
    _need(fn, (vocab == 1 or logits.stride(1) == 1) and _flat(tokens, _I32, (t,)) and
          _flat(logprob, _F32, (t,)) and _flat(entropy, _F32, (t,)) and _flat(lse, _F32, (t,)) and
          _flat(rank, _I32, (t,)) and _flat(top_ids, _I32, (t, top)) and
          _flat(top_logprobs, _F32, (t, top)))
    code = lib.hc_token_logprobs(t, vocab, top, _DTYPES[logits.dtype], logits.data_ptr(), logits.stride(0),
                                 tokens.data_ptr(), logprob.data_ptr(), entropy.data_ptr(),
                                 lse.data_ptr(), rank.data_ptr(), top_ids.data_ptr(),
                                 top_logprobs.data_ptr(), _stream(stream))
    _raise(fn, code)
