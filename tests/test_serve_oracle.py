"""The oracle of the operators of include/hc_serve.h against brute force and hand values."""
import math

import numpy as np
import pytest

from oracle import serve_oracle as S
from oracle import window_oracle as W


def test_rotation_is_a_rotation():
    g = np.random.default_rng(0)
    x, angle = g.standard_normal((5, 3, 64)), g.random((5, 24)) * 7
    for inter in (False, True):
        y = S.norm_rotate(x, None, 0, np.cos(angle), np.sin(angle), inter, wide=True)
        assert np.array_equal(y[..., 48:], x[..., 48:])
        z = x[..., 0:48:2] + 1j * x[..., 1:48:2] if inter else x[..., :24] + 1j * x[..., 24:48]
        z = z * np.exp(1j * angle)[:, None]
        got = y[..., 0:48:2] + 1j * y[..., 1:48:2] if inter else y[..., :24] + 1j * y[..., 24:48]
        assert np.allclose(got, z, atol=1e-12)
        steps = S.norm_rotate(x, None, 0, np.cos(angle), np.sin(angle), inter)
        assert steps.dtype == np.float32 and np.abs(steps - S.norm_rotate(x.astype(np.float32), None, 0, np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32), inter, True)).max() < 1e-6


def test_norm():
    g = np.random.default_rng(1)
    x, w, none = g.standard_normal((4, 2, 64)) * 3, g.random(64), np.zeros((4, 0))
    y = S.norm_rotate(x, w, 0.25, none, none, False, wide=True)
    for t in range(4):
        for h in range(2):
            assert np.allclose(y[t, h], x[t, h] / math.sqrt((x[t, h] ** 2).sum() / 64 + 0.25) * w)
    assert np.abs(S.norm_rotate(x, w, 0.25, none, none, False) - y).max() < 1e-6


def test_axes():
    table = np.arange(7 * 2 * 4).reshape(7, 2, 4)
    c, s = S.table_rows(table, [[1, 2], [6, 0]], [0, 1, 1, 0])
    assert c.tolist() == [[8, 49, 50, 11], [16, 1, 2, 19]] and (s - c == 4).all()
    assert (S.table_rows(table, [[3, 5]], None)[0] == table[[3, 5], 0]).all()


def test_shared_attention_is_attention_over_both():
    """With prefixes of whole blocks: hc_kv4_attention's oracle over the joined tables."""
    g = np.random.default_rng(2)
    codes = g.integers(0, 256, (20, 2, 2, 16, 32)).astype(np.uint8)
    scales = (g.random((20, 2, 2, 16, 2)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    order = g.permutation(20)
    prefix_table, table = order[:4].reshape(2, 2), order[4:13].reshape(3, 3)
    lens, cg, cu, kv = [32, 16], [0, 2, 3], [0, 2, 5, 6], [40, 20, 1]
    q = g.standard_normal((6, 4, 64))
    mask = [1, 3, 1, 2, 5, 1]
    for m in (None, mask):
        out, lse, size = S.attention_shared(q, codes, scales, prefix_table, lens, cg, table, cu, kv, m, 0.1)
        joined = [[*prefix_table[0], *table[0]], [*prefix_table[0], *table[1]], [prefix_table[1][0], *table[2], 0]]
        want = W.attention(q, codes, scales, joined, cu, [72, 52, 17], m, 0.1)
        for a, b in zip((out, lse, size), want):
            assert np.allclose(a, b, atol=1e-12)


def test_attention_of_an_empty_prefix_and_of_nothing():
    codes, scales = np.zeros((2, 2, 1, 16, 32), dtype=np.uint8), np.zeros((2, 2, 1, 16, 2), dtype=np.uint16)
    q = np.ones((2, 1, 64))
    out, lse, _ = S.attention_shared(q, codes, scales, [[0]], [0], [0, 2], [[0], [1]], [0, 1, 2], [0, 3])
    assert np.isneginf(lse[0, 0]) and lse[1, 0] == pytest.approx(math.log(3)) and (out == 0).all()


def test_sample_by_hand():
    x = [1.0, 3.0, 2.0, 3.0]
    e = np.exp(np.array(x) - 3)
    draw = lambda u, **kw: S.sample(x, u, **kw)[0]  # noqa: E731
    assert [draw(u) for u in (0.0, e[0] / e.sum() - 1e-9, e[0] / e.sum() + 1e-9, 0.999)] == [0, 0, 1, 3]
    assert S.sample(x, 0.7, temperature=0.0)[:2] == (1, 0.0)
    assert [draw(u, top_k=1) for u in (0, 0.99)] == [1, 1] and [draw(u, top_k=2) for u in (0, 0.49, 0.51, 0.99)] == [1, 1, 3, 3]
    assert [draw(u, top_k=3) for u in (0, 0.99)] == [1, 3] and draw(0.5, top_k=3, top_p=0.0) == 1
    p = 1 / e.sum()
    assert draw(0.99, top_p=p - 1e-6) == 1 and draw(0.99, top_p=p + 1e-6) == 3 and draw(0.0, top_p=0.9) == 1
    assert draw(0.0, min_p=math.exp(-1) - 1e-6) == 1 and draw(0.0, min_p=0.1) == 0 and draw(0.99, min_p=1.0) == 3
    assert S.sample(x, 0.6, top_k=2)[1] == pytest.approx(math.log(0.5))
    token, lp, _ = S.sample(x, 0.0, temperature=2.0)
    assert token == 0 and lp == pytest.approx(math.log(math.exp(-1) / (1 + 2 * 1 + math.exp(-1) + math.exp(-0.5) - 1)))


def test_sample_rows_that_are_none():
    for x, kw in (([1, math.nan], {}), ([1, math.inf], {}), ([-math.inf] * 2, {}), ([1, 2], dict(temperature=math.nan)),
                  ([1, 2], dict(temperature=math.inf)), ([1, 2], dict(top_p=math.nan)), ([1, 2], dict(min_p=math.nan))):
        token, lp, _ = S.sample(x, 0.5, **kw)
        assert token == -1 and math.isnan(lp)


def test_sample_draws_each_token_as_often_as_its_weight():
    g = np.random.default_rng(3)
    x = g.standard_normal(9)
    n = 4000
    got = np.bincount([S.sample(x, (i + 0.5) / n, top_p=0.9, temperature=0.7)[0] for i in range(n)], minlength=9)
    w = np.exp((x - x.max()) / 0.7)
    order = np.argsort(-w)
    w[order[np.cumsum(w[order]) - w[order] >= 0.9 * w.sum()]] = 0
    assert (np.abs(got - n * w / w.sum()) <= 1).all()
