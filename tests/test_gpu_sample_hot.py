"""hc_sample_tokens at temperatures next to fp32's largest, on both sides of where the kernel weighs
them in another way (2^64), with logits of -inf and logits as large as the type holds.

Tolerances: a weight is within 2^-27 of the formula's, so that two sums that are compared differ by
at most 2^-26 of the larger; nearer decisions are not compared. logprob within 2^-20 of 1 + its
size, as the header says.
"""
import numpy as np
import pytest
import torch

import hyper_connection_residual_read_gb300 as hc

from oracle import serve_oracle as S
from test_gpu_serve import DT, f64, run_sample

pytestmark = pytest.mark.gpu

NEAR = 2.0 ** -26
NEARLY_ONE = float(np.float32(1 - 2.0 ** -24))


@pytest.fixture(scope="module", autouse=True)
def context():
    hc.hc_read_init(0, 64, 1e-6)
    yield
    assert hc.hc_read_status() == hc.HC_OK


def check(x, u, **settings):
    got, lp = run_sample(x, u, **settings)
    x64, skipped = f64(x), 0
    for t in range(len(x64)):
        each = {k: float(np.float32(v[t])) if k != "top_k" else int(v[t]) for k, v in settings.items()}
        token, want, close = S.sample(x64[t], float(np.float32(u[t])), **each)
        # whatever the borders: the row is written, with a token that has weight
        assert 0 <= got[t] < x64.shape[1] and np.isfinite(x64[t, got[t]]) and np.isfinite(lp[t]), (t, got[t], lp[t], each)
        if close < NEAR:
            skipped += 1
            continue
        assert got[t] == token, (t, got[t], token, u[t], each, close)
        assert abs(lp[t] - want) <= 2.0 ** -20 * (1 + abs(want)), (t, lp[t], want, each)
    assert skipped <= 1 + len(x64) // 10


def filters(rows):
    full = lambda v: np.full(rows, v)  # noqa: E731
    return [{}, dict(top_p=full(0.9)), dict(top_p=full(0.3)), dict(top_k=full(7)), dict(top_k=full(300)),
            dict(top_k=full(300), top_p=full(0.5)), dict(min_p=full(0.2)), dict(min_p=full(1.0), top_p=full(0.99))]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab,first", [(7, 0), (1003, 0), (1003, 1), (1001, 3), (70001, 1)])
@pytest.mark.parametrize("size", ["small", "as large"])
def test_sample_of_hot_rows(dtype, vocab, first, size):
    """-inf among the logits, and rows that begin and end inside a vector (what lies around them
    counts as -inf too)."""
    g = np.random.default_rng(vocab + first)
    t = np.array([1.8e19, 1.9e19, 1e25, 2e37, 1e38, 3e38, np.finfo(np.float32).max], dtype=np.float32)
    x = g.standard_normal((len(t), first + vocab + 2)) * (3.0 if size == "small" else t[:, None].astype(np.float64) * 0.3)
    x = np.clip(x, -3.3e38, 3.3e38)
    x[:, 1:][g.random((len(t), first + vocab + 1)) < 0.4] = -np.inf
    x[:, first] = np.where(np.isfinite(x[:, first]), x[:, first], 0.5)
    x = torch.from_numpy(x).to(DT[dtype]).cuda()[:, first:first + vocab]
    for settings in filters(len(t)):
        for u in (np.full(len(t), NEARLY_ONE), np.zeros(len(t)), g.random(len(t))):
            check(x, u, temperature=t, **settings)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sample_between_the_ends_of_the_type(dtype):
    """Logits at both ends of what the type holds: their difference is beyond fp32."""
    g = np.random.default_rng(3)
    most = torch.finfo(DT[dtype]).max
    x = torch.from_numpy(np.where(g.random((6, 2003)) < 0.5, -1.0, 1.0)).to(DT[dtype]).cuda() * most
    x[:, 5], x[0, 7], x[3, 9] = most, float("-inf"), 0.0
    t = np.array([3.4e38, 2e38, 1e38, 3.4e38, 1e30, 1e20], dtype=np.float32)
    for settings in filters(6):
        for u in (np.full(6, NEARLY_ONE), g.random(6)):
            check(x, u, temperature=t, **settings)
