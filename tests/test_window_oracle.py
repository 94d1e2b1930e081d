"""Pins of the verify-window oracle on the CPU: hand-worked cases, closed forms, torch's
routines, and exact rational arithmetic for the 4-bit rounding."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import window_oracle as W
from oracle.hc_oracle import bf16_bits_to_f64


def test_plan_by_hand():
    """Block 4, a table of 3 blocks a row, free stack [9, 8, 7] (7 on top).

    request 0: 3 cached + 2 new: blocks 1 -> 2, takes 7
    request 1: 4 cached + 4 new: blocks 1 -> 2, takes 8
    request 2: 1 cached + 8 new: blocks 1 -> 3, wants 2 where 1 is left: refused
    request 3: 5 cached + 1 new: blocks 2 -> 2, wants none: granted
    request 4: 0 cached + 1 new: wants 1, but 2's wants come first: refused
    request 5: 9 cached + 4 new: 4 blocks, more than a row: refused
    """
    table = [[1, -1, -1], [2, -1, -1], [3, -1, -1], [4, 5, -1], [-1, -1, -1], [6, 10, 11]]
    got = W.plan([3, 4, 1, 5, 0, 9], [2, 4, 8, 1, 1, 4], [9, 8, 7], 3, 4, table, 22)
    t, slots, of, pos, cu, kv, left = got
    assert t.tolist() == [[1, 7, -1], [2, 8, -1], [3, -1, -1], [4, 5, -1], [-1, -1, -1], [6, 10, 11]]
    assert slots.tolist() == [7, 28, 32, 33, 34, 35] + [-1] * 8 + [21] + [-1] * 7
    assert of.tolist() == [0] * 2 + [1] * 4 + [2] * 8 + [3] + [4] + [5] * 4 + [-1] * 2
    assert pos[:6].tolist() == [3, 4, 4, 5, 6, 7] and pos[14] == 5 and pos[16] == 9
    assert cu.tolist() == [0, 2, 6, 14, 15, 16, 20] and kv.tolist() == [5, 8, 1, 6, 0, 9] and left == 1


def _fl(x: Fraction, bits: int, low: int, mode: str) -> Fraction:
    """x rounded to `bits` significant bits with least exponent `low`: 'near', 'down', 'up'."""
    if x == 0:
        return x
    e = 0
    while Fraction(2) ** e > abs(x):
        e -= 1
    while Fraction(2) ** (e + 1) <= abs(x):
        e += 1
    unit = Fraction(2) ** (max(e, low) - bits + 1)
    n = x / unit
    down = n.numerator // n.denominator
    if mode == "down":
        return down * unit
    if mode == "up":
        return -((-n.numerator) // n.denominator) * unit
    rest = n - down
    if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and down % 2):
        down += 1
    return down * unit


@pytest.mark.parametrize("seed", range(6))
def test_rounding_in_rational_arithmetic(seed):
    g = np.random.default_rng(seed)
    x = g.standard_normal((12, 16)) * np.exp2(g.integers(-20, 20, (12, 1)))
    x += g.standard_normal((12, 1)) * np.exp2(g.integers(-4, 8, (12, 1)))
    if seed == 0:
        x[0], x[1], x[2, 1:] = 0.0, 1.5, -x[2, 0]
        x[3] = np.arange(16) / 8                        # exact codes and ties
        x[4] = np.arange(16) * 2.0 ** -133              # subnormal steps
    x = x.astype(np.float32).astype(np.float64)
    codes, step, low = W.round_group(x)
    fifteenth = _fl(Fraction(1, 15), 24, -126, "near")
    for row, c, s, m in zip(x, codes, step, low):
        f = [Fraction(v) for v in row]
        em = _fl(min(f), 8, -126, "down")
        es = _fl(_fl(_fl(max(f) - em, 24, -126, "near") * fifteenth, 24, -126, "near"), 8, -126, "up")
        if 0 < es < Fraction(2) ** -126:
            es = Fraction(2) ** -126
        assert Fraction(float(m)) == em and Fraction(float(s)) == es
        r = _fl(1 / es, 24, -126, "near") if es else Fraction(0)
        for v, code in zip(f, c):
            z = _fl(_fl(v - em, 24, -126, "near") * r, 24, -126, "near")
            want = z.numerator // z.denominator
            rest = z - want
            if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and want % 2):
                want += 1
            assert min(max(want, 0), 15) == code


def test_rounding_error_is_half_a_step():
    g = np.random.default_rng(9)
    x = (g.standard_normal((200, 64)) * 3 + 40).astype(np.float32).astype(np.float64)
    codes, s, m = W.round_group(x)
    err = np.abs(m[:, None] + s[:, None] * codes - x)
    assert (err <= s[:, None] * (0.5 + 1e-5)).all()
    assert (codes.min(-1) == 0).any() and codes.max() <= 15


def test_groups_that_are_not_finite_are_nan():
    x = np.ones((5, 16))
    x[0, 3], x[1, 3], x[2, 3] = np.nan, np.inf, -np.inf
    x[3, 3], x[3, 4] = 3e38, -3e38                        # finite, but too wide for fp32
    codes, s, m = W.round_group(x)
    assert np.isnan(s[:4]).all() and np.isnan(m[:4]).all() and (codes[:4] == 0).all()
    assert s[4] == 0 and m[4] == 1 and (codes[4] == 0).all()


def test_pack_is_low_half_first():
    c = np.arange(16, dtype=np.uint8)[None]
    assert W.pack(c)[0, :2].tolist() == [0x10, 0x32] and (W.unpack(W.pack(c)) == c).all()


def test_attention_equals_softmax_of_the_dequantised_cache():
    g = np.random.default_rng(1)
    h, hq, d, block, length, n = 2, 4, 16, 4, 13, 3
    codes = g.integers(0, 256, (6, 2, h, block, d // 2)).astype(np.uint8)
    bits = torch.from_numpy(g.uniform(0.1, 0.4, (6, 2, h, block, 2))).bfloat16().view(torch.int16).numpy().view(np.uint16)
    table = np.array([[3, 1, 5, 0]])
    q = g.standard_normal((n, hq, d))
    out, lse, _ = W.attention(q, codes, bits, table, [0, n], [length], scale=0.25)
    sm = bf16_bits_to_f64(bits)
    full = sm[..., 1:] + sm[..., :1] * W.unpack(codes)
    kv = np.concatenate([full[p].transpose(0, 1, 2, 3) for p in table[0]], axis=2)[:, :, :length]
    for head in range(hq):
        k, v = torch.from_numpy(kv[0, head // 2]), torch.from_numpy(kv[1, head // 2])
        a = torch.from_numpy(q[:, head]) @ k.T * 0.25
        a = a.masked_fill(torch.arange(length)[None] > (length - n + torch.arange(n))[:, None], float("-inf"))
        assert np.allclose(out[:, head], (torch.softmax(a, -1) @ v).numpy(), rtol=1e-12, atol=1e-14)
        assert np.allclose(lse[:, head], torch.logsumexp(a, -1).numpy(), rtol=1e-12)
    # a mask of the causal order is the causal order; an empty one sees the cached part
    m = [1, 3, 7]
    assert np.array_equal(W.attention(q, codes, bits, table, [0, n], [length], m, 0.25)[0], out)
    alone = W.attention(q, codes, bits, table, [0, n], [n], [0, 1, 0], 0.25)
    assert (alone[0][0] == 0).all() and np.isneginf(alone[1][[0, 2]]).all() and (alone[0][1] != 0).any()


def test_logprobs_against_torch():
    g = np.random.default_rng(2)
    x = g.standard_normal((5, 37)) * 3
    x[0, 5] = -np.inf
    x[2, 3] = x[2, 30] = 50.0
    ids = np.array([1, 36, 30, -1, 37])
    r = W.logprobs(x, ids, 4)
    lp = torch.log_softmax(torch.from_numpy(x), -1)
    ent = torch.distributions.Categorical(logits=torch.from_numpy(np.where(np.isneginf(x), -1e9, x))).entropy()
    assert np.allclose(r["logprob"][:3], lp[[0, 1, 2], [1, 36, 30]].numpy(), rtol=1e-13)
    assert np.isneginf(r["logprob"][3:]).all() and (r["rank"][3:] == 37).all()
    assert np.allclose(r["entropy"], ent.numpy(), rtol=1e-12)
    assert r["top_ids"][2, :2].tolist() == [3, 30] and r["rank"][2] == 0
    r = W.logprobs(np.full((1, 6), -np.inf), np.array([2]), 3)
    assert r["lse"][0] == r["logprob"][0] == -np.inf and r["entropy"][0] == 0 and r["rank"][0] == 0
    assert r["top_ids"].tolist() == [[0, 1, 2]] and np.isneginf(r["top_logprobs"]).all()
