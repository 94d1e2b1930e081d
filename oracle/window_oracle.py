"""Plain CPU implementations of the verify-window operators (include/hc_window.h) in
numpy: whole numbers exactly, everything else in float64. Test infrastructure only; no
code is shared with the CUDA path.

16-bit formats travel as raw ``uint16`` bits, as in ``hc_oracle``.
"""
from __future__ import annotations

import numpy as np

from .hc_oracle import bf16_bits_to_f64


def plan(cached, new, free, count, block, table, capacity):
    """Request by request. Returns (table, slots, request_of, positions, cu, kv, left)."""
    table = np.array(table, dtype=np.int64)
    width = table.shape[1]
    count = min(max(int(count), 0), len(free))
    slots = np.full(capacity, -1, dtype=np.int64)
    request_of, positions = np.full(capacity, -1), np.full(capacity, -1)
    cu, kv, wanted, taken = [0], [], 0, 0
    for b, (c, n) in enumerate(zip(cached, new)):
        c, n = max(int(c), 0), max(int(n), 0)
        have, total = -(-c // block), -(-(c + n) // block)
        want = total - have if total <= width else 0
        granted = total <= width and (want == 0 or wanted + want <= count)
        if granted:
            for j in range(want):
                table[b, have + j] = free[count - 1 - (wanted + j)]
            taken += want
        wanted += want
        for i in range(n):
            t = cu[-1] + i
            if t < capacity:
                request_of[t], positions[t] = b, c + i
                if granted:
                    slots[t] = table[b, (c + i) // block] * block + (c + i) % block
        cu.append(cu[-1] + n)
        kv.append(c + n if granted else c)
    return table, slots, request_of, positions, np.array(cu), np.array(kv), count - taken


def _bf16_towards(x, up: bool) -> np.ndarray:
    """The nearest bf16 on one side of finite float64 values, in integer steps of the
    format: unit = the spacing of bf16 at |x| (normal and subnormal)."""
    _, e = np.frexp(x)
    unit = np.exp2(np.maximum(e.astype(np.float64), -125.0) - 8.0)
    return (np.ceil(x / unit) if up else np.floor(x / unit)) * unit


def round_group(x):
    """Codes (last axis), step and minimum of groups along the last axis. x: float64
    holding fp32 (or narrower) values."""
    x = np.asarray(x, dtype=np.float64)
    f32 = lambda a: np.asarray(a, dtype=np.float64).astype(np.float32).astype(np.float64)  # noqa: E731
    with np.errstate(all="ignore"):
        low, high = x.min(-1), x.max(-1)
        fine = np.isfinite(low) & np.isfinite(high)
        lo, hi = np.where(fine, low, 0.0), np.where(fine, high, 0.0)
        m = _bf16_towards(lo, False)
        m = np.where(np.abs(m) > 3.3895313892515355e38, -np.inf, m)
        width = f32(hi - m)
        step = _bf16_towards(np.where(np.isfinite(width), f32(width * np.float64(np.float32(1.0 / 15.0))), 0.0), True)
        fine &= np.isfinite(width)
        step = np.where((step > 0) & (step < 2.0 ** -126), 2.0 ** -126, step)
        r = np.where(step > 0, f32(1.0 / np.where(step > 0, step, 1.0)), 0.0)
        codes = np.clip(np.rint(f32(f32(x - m[..., None]) * r[..., None])), 0, 15)
    codes = np.where(fine[..., None], codes, 0).astype(np.uint8)
    return codes, np.where(fine, step, np.nan), np.where(fine, m, np.nan)


def pack(codes) -> np.ndarray:
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed) -> np.ndarray:
    return np.stack([packed & 15, packed >> 4], axis=-1).reshape(*packed.shape[:-1], -1)


def attention(q, codes, scales, table, cu, kv, mask=None, scale=1.0):
    """Token by token and head by head. q: float64 [tokens][q heads][dim]; codes: packed;
    scales: bf16 bits. Returns (out, lse, size): size is sum p (|s (c - 8)| + |m + 8 s|),
    the magnitude of the terms that the sums of `out` add up."""
    tokens, hq, d = q.shape
    h, block = codes.shape[2], codes.shape[3]
    out = np.zeros((tokens, hq, d))
    size = np.zeros((tokens, hq, d))
    lse = np.full((tokens, hq), -np.inf)
    for b in range(len(kv)):
        n, length = cu[b + 1] - cu[b], max(int(kv[b]), 0)
        if n <= 0 or length == 0:
            continue
        at = np.arange(length)
        pages = np.asarray(table[b])[at // block]
        c = unpack(codes[pages, :, :, at % block]).astype(np.float64)     # [length][2][h][d]
        sm = bf16_bits_to_f64(scales[pages, :, :, at % block])            # [length][2][h][2]
        s, m = sm[..., 0:1], sm[..., 1:2]
        value = m + s * c
        terms = np.abs(s * (c - 8)) + np.abs(m + 8 * s)
        for i in range(n):
            t = cu[b] + i
            first = length - n
            if mask is None:
                sees = at <= first + i
            else:
                sees = np.array([j < first or bool((int(mask[t]) >> int(j - first)) & 1) for j in at])
            if not sees.any():
                continue
            for head in range(hq):
                g = head // (hq // h)
                x = scale * (value[sees, 0, g] @ q[t, head])
                top = x.max()
                p = np.exp(x - top)
                lse[t, head] = top + np.log(p.sum())
                p = p / p.sum()
                out[t, head] = p @ value[sees, 1, g]
                size[t, head] = p @ terms[sees, 1, g]
    return out, lse, size


def logprobs(x, ids, top):
    """x: float64 logits. Returns dict of float64 and whole-number arrays."""
    rows, vocab = x.shape
    with np.errstate(all="ignore"):
        peak = x.max(-1)
        ref = np.where(np.isfinite(peak), peak, 0.0)
        total = np.exp(x - ref[:, None]).sum(-1)
        lse = np.where(total > 0, ref + np.log(total), -np.inf)
        # x - lse without a sum of both: at 1e30, 64 bits do not hold the logarithm beside it
        lp = np.where(np.isneginf(x), -np.inf, x - ref[:, None] - np.where(total > 0, np.log(total), 0)[:, None])
        p = np.exp(lp)
        entropy = -np.where(p > 0, p * lp, 0.0).sum(-1) + 0.0
    known = (ids >= 0) & (ids < vocab)
    mine = np.where(known, x[np.arange(rows), np.where(known, ids, 0)], -np.inf)
    order = np.argsort(-x, axis=-1, kind="stable")[:, :top]
    return dict(logprob=np.where(known, lp[np.arange(rows), np.where(known, ids, 0)], -np.inf),
                entropy=entropy, lse=lse,
                rank=np.where(known, (x > mine[:, None]).sum(-1), vocab),
                top_ids=order, top_logprobs=np.take_along_axis(lp, order, -1))
