"""Log probabilities against 64 bits with tolerances from what a row is made of, so that rows
with a logit far from the others are held as closely as any.

With T the row's largest logit (finite) and V the vocabulary:

* lse: T and T log2(e) are rounded to fp32 (2^-24 of |T| each, and once more in the sum), and
  s carries the error of its exponentials (2^-22) and of its partial sums, which add at most
  2^7 terms one after the other here: 2^-22 |T| + 2^-17;
* a log probability (x - r) - ln s, r a reference near T: the errors of s, to which r log2(e) in
  fp32 belongs where |r| is at most 1024 (beyond, differences from r are taken first), and
  the difference's rounding: 2^-17 + 2^-22 min(|T|, 1100) + 2^-23 |x - T|;
* the entropy ln s - b / s: both are at most ln V + 28 (the sums' reference is within 27.7 of
  the largest logit) and as exact as s: 2^-17 + 2^-20 (ln V + 28).
"""
import numpy as np
import pytest
import torch

import hyper_connection_residual_read_gb300 as hc

from oracle import window_oracle as W

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def context():
    hc.hc_read_init(0, 64, 1e-6)
    yield
    assert hc.hc_read_status() == hc.HC_OK


def score(x, ids, top, stream=None):
    t = x.shape[0]
    f = lambda *s: torch.full(s, 77.0, device="cuda")  # noqa: E731
    i = lambda *s: torch.full(s, -77, dtype=torch.int32, device="cuda")  # noqa: E731
    out = dict(logprob=f(t), entropy=f(t), lse=f(t), rank=i(t), top_ids=i(t, top), top_logprobs=f(t, top))
    ids = torch.as_tensor(np.asarray(ids), dtype=torch.int32).cuda()
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    hc.hc_token_logprobs(x, ids, *out.values(), stream=stream)
    if stream is not None:
        stream.synchronize()                                # its results are copied on another one
    return {k: v.cpu().numpy() for k, v in out.items()}


def check(x, ids, top, **kw):
    got, x64, ids = score(x, ids, top, **kw), x.double().cpu().numpy(), np.asarray(ids)
    want = W.logprobs(x64, ids, top)
    for name in ("rank", "top_ids"):
        assert np.array_equal(got[name], want[name]), name
    peak, size = x64.max(-1), np.log(x64.shape[1])
    peak = np.where(np.isfinite(peak), peak, 0)
    known = (ids >= 0) & (ids < x64.shape[1])
    mine = x64[np.arange(len(ids)), np.where(known, ids, 0)]
    tops = np.take_along_axis(x64, want["top_ids"], -1)
    near = 2.0 ** -17 + 2.0 ** -22 * np.minimum(np.abs(peak), 1100)
    away = lambda y, t: 2.0 ** -23 * np.where(np.isfinite(y), np.abs(y - t), 0)  # noqa: E731
    with np.errstate(invalid="ignore"):
        tol = dict(lse=2.0 ** -17 + 2.0 ** -22 * np.abs(peak), logprob=near + away(mine, peak),
                   entropy=np.full(len(ids), 2.0 ** -17 + 2.0 ** -20 * (size + 28)),
                   top_logprobs=near[:, None] + away(tops, peak[:, None]))
        for name, t in tol.items():
            g, w = got[name].astype(np.float64), want[name]
            off = np.where(g == w, 0, np.abs(g - w))
            assert (off <= t).all(), (name, np.argwhere(~(off <= t))[:4], g[~(off <= t)][:4], w[~(off <= t)][:4])


def hard_rows(vocab, dtype):
    """One far logit above the others, all the same far from 0, the type's lowest value beside
    an ordinary one and alone, -inf around a few, ramps, and ordinary rows moved away from 0."""
    low, g = torch.finfo(dtype).min, torch.Generator().manual_seed(vocab)
    far = 3e4 if dtype is torch.float16 else 1e30
    x = torch.zeros(14, vocab, dtype=torch.float64)
    x[0, vocab // 2] = far
    x[1] = -far
    x[2], x[2, 1] = low, 3.0
    x[3] = low
    x[4] = float("-inf")
    x[4, ::5] = torch.arange(len(x[4, ::5]), dtype=torch.float64) * -0.25
    x[5] = torch.arange(vocab, dtype=torch.float64) * 1e-3
    x[6] = -x[5]
    x[7] = torch.randn(vocab, generator=g, dtype=torch.float64) * 3 + 1000
    x[8] = torch.randn(vocab, generator=g, dtype=torch.float64) * 3 - 900
    x[9] = torch.randn(vocab, generator=g, dtype=torch.float64) * 3 - 5000
    x[10] = torch.randn(vocab, generator=g, dtype=torch.float64) * 40
    x[11] = -200.0
    x[11, vocab - 1] = 0.0
    x[12] = torch.linspace(-80, 80, vocab, dtype=torch.float64)[torch.randperm(vocab, generator=g)]
    x[13] = torch.where(torch.arange(vocab) % 97 == 5, 12.0, -30.0)
    return x.to(dtype)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("vocab", [8, 257, 1003, 32000])
def test_rows_far_from_ordinary(dtype, vocab):
    x = hard_rows(vocab, DT[dtype]).cuda()
    g = np.random.default_rng(vocab)
    ids = g.integers(0, vocab, len(x))
    ids[[0, 2, 11]] = vocab // 2, 1, vocab - 1
    check(x, ids, min(8, vocab))
    check(x, np.where(np.arange(len(x)) % 2, x.float().argmax(-1).cpu().numpy(), 0), 1)


@pytest.mark.parametrize("dtype", list(DT))
def test_ordinary_rows_on_another_stream(dtype):
    g = np.random.default_rng(4)
    x = torch.from_numpy(g.standard_normal((9, 32000)) * 4).to(DT[dtype]).cuda()
    check(x, g.integers(0, 32000, 9), 20, stream=torch.cuda.Stream())
    check(x[:, 3:20000], g.integers(0, 19997, 9), 20, stream=torch.cuda.Stream())
