"""Plain CPU implementations of the operators of include/hc_serve.h in numpy: what is stated as
single fp32 operations in numpy's fp32, whole numbers exactly, everything else in float64. Test
infrastructure only; no code is shared with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

from .hc_oracle import bf16_bits_to_f64
from .window_oracle import unpack

F = np.float32


def norm_rotate(x, weight, eps, cos, sin, interleaved, wide=False):
    """Heads x [tokens][heads][dim] normed by `weight` (None: not) and rotated: cos, sin [tokens]
    [dims / 2]. In fp32 steps, or (wide) by the formula in float64."""
    kind = np.float64 if wide else F
    x = np.asarray(x, dtype=kind)
    with np.errstate(all="ignore"):
        if weight is not None:
            y, d = x * x, x.shape[-1]
            while y.shape[-1] > 1:
                y = y[..., 0::2] + y[..., 1::2]
            r = kind(1) / np.sqrt(y * kind(1 / d) + kind(F(eps)))
            x = (x * r) * np.asarray(weight, dtype=kind)
        half = cos.shape[-1]
        a, b = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
        c, s = (np.asarray(t, dtype=kind)[:, None] for t in (cos, sin))
        out = x.copy()
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def table_rows(cos_sin, positions, axis_of):
    """The cosines and sines [tokens][dims / 2] of tokens at positions [axes][tokens]."""
    half = cos_sin.shape[2]
    axis = np.zeros(half, dtype=int) if axis_of is None else np.asarray(axis_of)
    row = np.asarray(positions)[axis].T
    return cos_sin[row, 0, np.arange(half)], cos_sin[row, 1, np.arange(half)]


def cached(codes, scales, pages, length):
    """Keys and values [2][length][kv heads][dim] of the first `length` tokens in `pages`, and the
    sizes |s (c - 8)| + |m + 8 s| of their parts. scales: bf16 bits."""
    block = codes.shape[3]
    if length == 0:
        return (np.zeros((2, 0, codes.shape[2], 2 * codes.shape[4])),) * 2
    at = np.arange(length)
    pages = np.asarray(pages)[at // block]
    c = unpack(codes[pages, :, :, at % block]).astype(np.float64)          # [length][2][h][d]
    sm = bf16_bits_to_f64(scales[pages, :, :, at % block])
    s, m = sm[..., 0:1], sm[..., 1:2]
    return (m + s * c).swapaxes(0, 1), (np.abs(s * (c - 8)) + np.abs(m + 8 * s)).swapaxes(0, 1)


def attention_shared(q, codes, scales, prefix_table, prefix_lens, cu_groups, table, cu, kv, mask=None, scale=1.0):
    """Token by token and head by head over the prefix and the own tokens as one sequence. Returns
    (out, lse, size) as window_oracle.attention."""
    tokens, hq, d = q.shape
    h = codes.shape[2]
    out, size = np.zeros((tokens, hq, d)), np.zeros((tokens, hq, d))
    lse = np.full((tokens, hq), -np.inf)
    for group in range(len(prefix_lens)):
        before = max(int(prefix_lens[group]), 0)
        common, common_size = cached(codes, scales, prefix_table[group], before)
        for b in range(cu_groups[group], cu_groups[group + 1]):
            n, length = int(cu[b + 1] - cu[b]), max(int(kv[b]), 0)
            mine, mine_size = cached(codes, scales, table[b], length)
            value, terms = np.concatenate([common, mine], 1), np.concatenate([common_size, mine_size], 1)
            back = np.arange(before + length) - before - (length - n)      # of the prefix: below 0, or hidden by no rule
            back[:before] = -1
            for i in range(n):
                t = cu[b] + i
                if mask is None:
                    sees = back <= i
                else:
                    sees = np.array([j < 0 or bool((int(mask[t]) >> int(j)) & 1) for j in back], dtype=bool)
                if not sees.any():
                    continue
                for head in range(hq):
                    g = head // (hq // h)
                    x = scale * (value[0, sees, g] @ q[t, head])
                    top = x.max()
                    p = np.exp(x - top)
                    lse[t, head] = top + np.log(p.sum())
                    p = p / p.sum()
                    out[t, head] = p @ value[1, sees, g]
                    size[t, head] = p @ terms[1, sees, g]
    return out, lse, size


def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row. Returns (token, logprob, near): near is how close a decision was, the smallest
    distance of the uniform number to a border or of a sum or weight to a filter's, relative to
    what it is compared with (1 where all weights are 0 or 1, whose sums are exact, as their products
    with fp32 numbers are in 64 bits)."""
    x = np.asarray(x, dtype=np.float64)
    settings = (u, temperature, top_p, min_p)
    if np.isnan(x).any() or np.isposinf(x).any() or np.isneginf(x).all() or np.isnan(settings).any() or math.isinf(temperature):
        return -1, math.nan, 1.0
    if temperature < 2.0 ** -64:
        return int(np.argmax(x)), 0.0, 1.0
    with np.errstate(over="ignore"):
        w = np.exp((x - x.max()) / temperature)
    order = np.argsort(-x, kind="stable")
    near = 1.0
    if 1 <= top_k < len(order):
        order = order[:top_k]
    exact = np.isin(w[order], (0.0, 1.0)).all()
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w[order])])
        goal = max(top_p, 0.0) * before[-1]
        stays = before[:-1] < goal
        stays[0] = True
        near = min(near, np.abs(before[1:-1] - goal).min(initial=np.inf) / before[-1])
        order = order[stays]
    least = min(max(min_p, 0.0), 1.0)
    if least > 0:
        near = min(near, np.abs(w[order] / least - 1)[w[order] != 1].min(initial=np.inf))
        order = order[w[order] >= least]
    order = np.sort(order)
    upto = np.cumsum(w[order])
    goal = min(max(u, 0.0), 1 - 2.0 ** -53) * upto[-1]
    some = w[order] > 0
    i = int(np.argmax((upto > goal) & some)) if ((upto > goal) & some).any() else int(np.nonzero(some)[0][-1])
    if goal > 0:
        near = min(near, np.abs(upto - goal).min() / upto[-1])
    if exact:
        near = 1.0
    return int(order[i]), math.log(w[order[i]] / upto[-1]), near
