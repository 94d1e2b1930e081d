"""Binding of the operators of include/hc_serve.h, same names: argument marshalling only, as in
``_window``. Shapes that disagree, tensors that are not laid out as the header says and
unsupported types raise ``HcReadError`` with ``HC_ERR_ARG``, as the library's own refusals do.

The calls go through a small CPython module (``_hcpyserve``, built with the library) that
reads the tensors in C; where it was not built, through ctypes.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._window import _DTYPES, _F32, _I32, _I64, _cache, _flat, _need, _raise, _stream, hc_kv4_cache

HC_ROTARY_MAX_AXES = 4
HC_SAMPLE_MAX_VOCAB = 262144

# every symbol include/hc_serve.h declares
SERVE_EXPORTS = ("hc_kv4_append_rotary", "hc_kv4_attention_shared", "hc_sample_tokens")


class hc_rotary(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("axis_of", ctypes.c_void_p), ("q_norm", ctypes.c_void_p),
                ("k_norm", ctypes.c_void_p), ("eps", ctypes.c_float), ("length", ctypes.c_int),
                ("dim", ctypes.c_int), ("axes", ctypes.c_int), ("interleaved", ctypes.c_int)]


_bound = None
_call = None         # the _hcpyserve module, bound to the library's entry points


def _bind_call(lib) -> None:
    global _call
    try:
        from . import _hcpyserve
    except ImportError:
        return
    addr = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    _hcpyserve.bind(*[addr(getattr(lib, name)) for name in SERVE_EXPORTS], torch.bfloat16, torch.float16,
                    torch.float32, torch.int32, torch.int64, torch.uint8)
    _call = _hcpyserve


def _load():
    global _bound
    if _bound is not None:
        return _bound
    lib = _lib.load()
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    cache, rotary = ctypes.POINTER(hc_kv4_cache), ctypes.POINTER(hc_rotary)
    lib.hc_kv4_append_rotary.argtypes = [cache, rotary, i32, i32, i32] + [vp, i64, i64] * 3 + [vp] * 4
    lib.hc_kv4_attention_shared.argtypes = [cache] + [i32] * 8 + [f32, i32, vp, i64, i64] + [vp] * 11
    lib.hc_sample_tokens.argtypes = [i32] * 3 + [vp, i64] + [vp] * 8
    for name in SERVE_EXPORTS:
        getattr(lib, name).restype = i32
    _bound = lib
    _bind_call(lib)
    return lib


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rows(t, dtype, shape) -> bool:
    return t.dtype is dtype and t.shape == shape and t.stride(2) == 1


def hc_kv4_append_rotary(q, k, v, cos_sin, positions, slots, codes, scales, q_out, q_norm=None, k_norm=None,
                         eps=1e-6, axis_of=None, interleaved=False, stream=None) -> None:
    """Norms (where weights are given) and rotates the queries ``q`` [tokens][q heads][head dim]
    and keys ``k`` [tokens][kv heads][head dim] (any strides of the first two axes), writes the
    queries to ``q_out``, and rounds the keys and the values ``v`` to 4 bits into their ``slots``
    (int64). ``positions`` (int32) [tokens] or [axes][tokens] are rows of ``cos_sin`` [length][2]
    [dims / 2] (fp32), ``axis_of`` (int32) [dims / 2] the axis of each frequency. ``q`` and
    ``q_out`` may be None (keys and values alone), and ``cos_sin`` with ``positions`` (no
    rotation)."""
    lib, fn = _bound or _load(), "hc_kv4_append_rotary"
    if _call is not None:
        return _raise(fn, _call.rotary(q, k, v, cos_sin, positions, slots, codes, scales, q_out, q_norm, k_norm, eps,
                                       axis_of, interleaved, _stream(stream)))
    cache = _cache(fn, codes, scales)
    _need(fn, k.dim() == 3 and k.dtype in _DTYPES)
    t, dt, heads, d = k.shape[0], k.dtype, 0 if q is None else q.shape[1], cache.head_dim
    _need(fn, _rows(k, dt, (t, cache.kv_heads, d)) and _rows(v, dt, (t, cache.kv_heads, d)) and
          _flat(slots, _I64, (t,)) and (q is None) == (q_out is None) and
          (cos_sin is None) == (positions is None) and (axis_of is None or cos_sin is not None))
    if q is not None:
        _need(fn, q.dim() == 3 and _rows(q, dt, (t, heads, d)) and _flat(q_out, dt, (t, heads, d)))
    r = hc_rotary(_ptr(cos_sin), _ptr(axis_of), _ptr(q_norm), _ptr(k_norm), eps, 0, 0, 0, bool(interleaved))
    if cos_sin is not None:
        _need(fn, cos_sin.dim() == 3 and _flat(cos_sin, _F32, (cos_sin.shape[0], 2, cos_sin.shape[2])) and
              positions.dim() in (1, 2) and positions.dtype is _I32 and positions.is_contiguous() and
              positions.shape[-1] == t and (axis_of is None or _flat(axis_of, _I32, (cos_sin.shape[2],))))
        r.length, r.dim = cos_sin.shape[0], 2 * cos_sin.shape[2]
        r.axes = positions.shape[0] if positions.dim() == 2 else 1
    _need(fn, (q_norm is None or _flat(q_norm, dt, (d,))) and (k_norm is None or _flat(k_norm, dt, (d,))))
    strides = lambda x: (0, 0) if x is None else (x.stride(0), x.stride(1))  # noqa: E731
    code = lib.hc_kv4_append_rotary(cache, r, t, heads, _DTYPES[dt], _ptr(q), *strides(q), k.data_ptr(), *strides(k),
                                    v.data_ptr(), *strides(v), _ptr(positions), slots.data_ptr(), _ptr(q_out),
                                    _stream(stream))
    _raise(fn, code)


def hc_kv4_attention_shared(q, codes, scales, prefix_table, prefix_lens, cu_groups, max_shared, block_table, cu_lens,
                            kv_lens, max_new, workspace, out, lse=None, mask=None, scale=None, stream=None) -> None:
    """``hc_kv4_attention`` of requests in groups, each group behind a prefix that its requests
    share: ``prefix_table`` [groups][width], ``prefix_lens`` [groups] and the groups' first
    requests ``cu_groups`` [groups + 1], all int32. ``max_shared`` bounds the new tokens of a
    group, ``workspace`` has q heads * (head dim + 2) floats a token."""
    lib, fn = _bound or _load(), "hc_kv4_attention_shared"
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    if _call is not None:
        return _raise(fn, _call.shared(q, codes, scales, prefix_table, prefix_lens, cu_groups, max_shared, block_table,
                                       cu_lens, kv_lens, max_new, workspace, out, lse, mask, scale, _stream(stream)))
    cache = _cache(fn, codes, scales)
    shape, n, groups = q.shape, kv_lens.numel(), prefix_lens.numel()
    _need(fn, len(shape) == 3 and shape[2] == cache.head_dim and q.stride(2) == 1 and q.dtype in _DTYPES and
          _flat(out, q.dtype, shape) and (lse is None or _flat(lse, _F32, shape[:2])) and
          (mask is None or _flat(mask, _I64, shape[:1])) and block_table.dim() == 2 and prefix_table.dim() == 2 and
          _flat(block_table, _I32, (n, block_table.shape[1])) and
          _flat(prefix_table, _I32, (groups, prefix_table.shape[1])) and _flat(prefix_lens, _I32, (groups,)) and
          _flat(cu_groups, _I32, (groups + 1,)) and _flat(cu_lens, _I32, (n + 1,)) and _flat(kv_lens, _I32, (n,)) and
          _flat(workspace, _F32, (workspace.numel(),)) and
          workspace.numel() >= shape[0] * shape[1] * (shape[2] + 2))
    code = lib.hc_kv4_attention_shared(
        cache, n, groups, shape[0], shape[1], max_new, max_shared, block_table.shape[1], prefix_table.shape[1], scale,
        _DTYPES[q.dtype], q.data_ptr(), q.stride(0), q.stride(1), cu_lens.data_ptr(), kv_lens.data_ptr(),
        block_table.data_ptr(), cu_groups.data_ptr(), prefix_lens.data_ptr(), prefix_table.data_ptr(), _ptr(mask),
        workspace.data_ptr(), out.data_ptr(), _ptr(lse), _stream(stream))
    _raise(fn, code)


def hc_sample_tokens(logits, uniform, tokens, logprobs, temperature=None, top_k=None, top_p=None, min_p=None,
                     stream=None) -> None:
    """Draws a token of each row of ``logits`` [tokens][vocabulary] (any row stride) by the numbers
    ``uniform`` in [0, 1), into ``tokens`` (int32), with its log probability under what it was
    drawn from. ``temperature``, ``top_p``, ``min_p`` (fp32) and ``top_k`` (int32) have a value a
    row; None: 1, all, none, all."""
    lib, fn = _bound or _load(), "hc_sample_tokens"
    if _call is not None:
        return _raise(fn, _call.sample(logits, uniform, tokens, logprobs, temperature, top_k, top_p, min_p,
                                       _stream(stream)))
    _need(fn, logits.dim() == 2 and logits.dtype in _DTYPES)
    t, vocab = logits.shape
    _need(fn, (vocab == 1 or logits.stride(1) == 1) and _flat(uniform, _F32, (t,)) and _flat(tokens, _I32, (t,)) and
          _flat(logprobs, _F32, (t,)) and (top_k is None or _flat(top_k, _I32, (t,))) and
          all(x is None or _flat(x, _F32, (t,)) for x in (temperature, top_p, min_p)))
    code = lib.hc_sample_tokens(t, vocab, _DTYPES[logits.dtype], logits.data_ptr(), logits.stride(0),
                                uniform.data_ptr(), _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p),
                                tokens.data_ptr(), logprobs.data_ptr(), _stream(stream))
    _raise(fn, code)
