"""The verify-window operators on the GPU against the 64-bit oracle
(oracle/window_oracle.py), at the sizes, masks and values where they can go wrong.

Tolerances (derived, per element):

* whole numbers, codes, steps and minima: equal.
* load: the oracle's value rounded to the output type: equal (one fp32 rounding first:
  within one ulp of the type where that rounding falls on a tie).
* attention out: half an ulp of the output type (8 significant bits for bf16, 11 for
  fp16: 2^-8 and 2^-11 of |o|), plus the weights: each p_j s_j is rounded once to 11 bits
  (2^-11 relative) and carries the error of its exponent, fp32 sums of |q||k| terms, for
  which as much again is allowed while logits stay below 2^8: 2^-10 of sum p (|s (c - 8)|
  + |m + 8 s|); plus 2^-24 of the largest step times the number of keys, for weights
  below the range of 16 bits.
* lse: fp32 sums of head_dim products and of the exponentials: 2^-19 of 1 + the largest
  sum of |terms| of a logit.
* log probabilities: |x| and the logarithm rounded to fp32 a few times, the sum over the
  vocabulary in fp32 partial sums: 2^-20 of 1 + the largest finite |x| of the row + ln V.
"""
import numpy as np
import pytest
import torch

import hyper_connection_residual_read_gb300 as hc

from oracle import window_oracle as W
from oracle.hc_oracle import bf16_bits_to_f64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def context():
    hc.hc_read_init(0, 64, 1e-6)
    yield
    assert hc.hc_read_status() == hc.HC_OK


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def f64(t):
    return t.double().cpu().numpy()


def bits16(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------

def run_plan(cached, new, free, count, block, table, capacity):
    n = len(cached)
    z = lambda k, dt=torch.int32: torch.full((k,), -77, dtype=dt, device="cuda")  # noqa: E731
    t = i32(table)
    out = [z(capacity, torch.int64), z(capacity), z(capacity), z(n + 1), z(n), z(1)]
    hc.hc_window_plan(i32(cached), i32(new), i32(free), i32([count]), block, t, *out)
    return [t.cpu().numpy()] + [x.cpu().numpy() for x in out[:5]] + [int(out[5])]


def check_plan(cached, new, free, count, block, table, capacity):
    got = run_plan(cached, new, free, count, block, table, capacity)
    want = W.plan(cached, new, free, count, block, table, capacity)
    for name, x, y in zip(("table", "slots", "request_of", "positions", "cu", "kv", "left"), got, want):
        assert np.array_equal(x, y), name


@pytest.mark.parametrize("requests,new,cached,block,pool", [
    (1, 1, 0, 16, 1.0), (1, 5000, 0, 32, 1.0), (1, 1, 16, 16, 1.0), (3, 8, 100, 16, 0.0),
    (31, 8, 500, 16, 0.5), (33, 4, 3000, 64, 1.0), (511, 9, 64, 128, 0.6), (513, 3, 64, 256, 0.9),
    (1500, 40, 200, 16, 0.7), (4097, 2, 40, 16, 0.8), (8192, 3, 20, 16, 0.3)])
def test_plan(requests, new, cached, block, pool):
    g = np.random.default_rng(requests * 7 + new)
    c, n = g.integers(0, cached + 1, requests), g.integers(0, new + 1, requests)
    have, total = -(-c // block), -(-(c + n) // block)
    width = max(1, int(total.max()) - (1 if requests > 100 else 0))     # some rows too long
    count = int(pool * (total - have).sum())
    ids = g.permutation(int(have.sum()) + count + 5)
    table = g.integers(0, 1 << 20, (requests, width))
    check_plan(c, n, ids[: count + 5], count, block, table, int(n.sum()) + 37)


def test_plan_odd_lengths_and_counts():
    # negative lengths count as 0, a count beyond the list is cut, a short capacity cuts
    check_plan([-5, 3, 16], [4, -1, 20], [3, 1, 4], 99, 16, [[7, 8], [9, 10], [11, 12]], 9)
    check_plan([0, 0], [0, 0], [3], -4, 16, [[7], [8]], 0)
    check_plan([0], [40], [], 0, 16, [[1, 2, 3]], 40)
    big = 2 ** 31 - 8
    check_plan([big, 5], [3, 3], [1, 2], 2, 256, [[0] * 4, [6] * 4], 8)


# ---------------------------------------------------------------------------
# cache
# ---------------------------------------------------------------------------

def blank_cache(blocks, heads, block, dim, poison=True):
    codes = torch.full((blocks, 2, heads, block, dim // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((blocks, 2, heads, block, 2), float("nan") if poison else 1.0,
                        dtype=torch.bfloat16, device="cuda")
    return codes, scales


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("tokens,heads,dim,block", [
    (1, 1, 64, 16), (1, 8, 128, 16), (17, 3, 128, 32), (33, 5, 64, 256), (200, 2, 128, 64)])
def test_append_and_load(dtype, tokens, heads, dim, block):
    g = np.random.default_rng(tokens + dim)
    fused = torch.from_numpy(g.standard_normal((tokens, 3 * heads * dim)) *
                             np.exp2(g.integers(-6, 6, (tokens, 1)))).to(DT[dtype]).cuda()
    k = fused[:, heads * dim:2 * heads * dim].view(tokens, heads, dim)
    # values: another layout (heads outermost), with an offset
    v = (torch.from_numpy(g.standard_normal((heads, tokens, dim)) + 5).to(DT[dtype]).cuda()).transpose(0, 1)
    blocks = tokens // block + 3
    codes, scales = blank_cache(blocks, heads, block, dim)
    before = codes.clone(), bits16(scales)
    slots = torch.from_numpy(g.permutation(blocks * block)[:tokens].astype(np.int64)).cuda()
    if tokens > 20:
        slots[[2, 7]] = torch.tensor([-1, -100]).cuda()
    hc.hc_kv4_append(k, v, slots, codes, scales)
    put = slots.cpu().numpy()
    keep = put >= 0
    wc, ws = before[0].cpu().numpy(), before[1].copy()
    for kv, x in enumerate((k, v)):
        c, s, m = W.round_group(f64(x))
        as_bits = lambda a: (a.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)  # noqa: E731
        wc[put[keep] // block, kv, :, put[keep] % block] = W.pack(c[keep])
        ws[put[keep] // block, kv, :, put[keep] % block] = np.stack([as_bits(s[keep]), as_bits(m[keep])], -1)
    assert np.array_equal(codes.cpu().numpy(), wc)
    assert np.array_equal(bits16(scales), ws)
    for out in DT.values():
        ko, vo = (torch.full((tokens, heads, dim), 9.0, dtype=out, device="cuda") for _ in range(2))
        hc.hc_kv4_load(slots, codes, scales, ko, vo)
        for kv, o in enumerate((ko, vo)):
            sm = bf16_bits_to_f64(ws[np.maximum(put, 0) // block, kv, :, np.maximum(put, 0) % block])
            c = W.unpack(wc[np.maximum(put, 0) // block, kv, :, np.maximum(put, 0) % block])
            want = np.where(keep[:, None, None], sm[..., 1:] + sm[..., :1] * c, 0.0)
            want = torch.from_numpy(want.astype(np.float32)).to(out)
            assert torch.equal(o.cpu(), want)


def test_append_of_difficult_groups():
    """Constants, zeros, ties, subnormals, the largest values, NaN and infinities."""
    d = 64
    x = np.zeros((12, d))
    x[1] = -3.25
    x[2] = np.arange(d) % 16 / 8
    x[3] = (np.arange(d) % 31) / 4 - 1                      # many ties
    x[4] = np.arange(d) * 2.0 ** -140
    x[5] = np.where(np.arange(d) % 2, 1.5 * 2.0 ** 127, 0)
    x[6] = np.where(np.arange(d) % 2, 1.5 * 2.0 ** 127, -1.5 * 2.0 ** 127)
    x[7, 5] = np.nan
    x[8, 63] = np.inf
    x[9, 0] = -np.inf
    x[10] = 1000 + np.arange(d) * 2.0 ** -12
    x[11] = -1e-30 * np.arange(d)
    x = x.astype(np.float32)
    t = torch.from_numpy(x).cuda().view(12, 1, d)
    codes, scales = blank_cache(1, 1, 16, d)
    slots = torch.arange(12).cuda()
    hc.hc_kv4_append(t, t, slots, codes, scales)
    c, s, m = W.round_group(x.astype(np.float64))
    got = scales.double().cpu().numpy()[0, :, 0, :12]
    for kv in range(2):
        assert np.array_equal(codes.cpu().numpy()[0, kv, 0, :12], W.pack(c))
        assert np.array_equal(got[kv, :, 0], s, equal_nan=True) and np.array_equal(got[kv, :, 1], m, equal_nan=True)
    assert np.isnan(s).tolist() == [False] * 6 + [True] * 4 + [False] * 2


def test_slots_outside_the_cache_are_skipped_and_reported():
    codes, scales = blank_cache(2, 1, 16, 64)
    before = codes.clone()
    k = torch.ones(3, 1, 64, device="cuda")
    slots = torch.tensor([32, 1 << 40, 5]).cuda()
    hc.hc_kv4_append(k, k, slots, codes, scales)
    assert hc.hc_read_status() == hc.HC_ERR_BOUNDS and hc.hc_read_status() == hc.HC_OK
    changed = (codes != before).flatten(3).any(-1).nonzero().cpu().tolist()
    assert changed == [[0, 0, 0], [0, 1, 0]]
    o = torch.ones(3, 1, 64, device="cuda")
    p = torch.ones(3, 1, 64, device="cuda")
    hc.hc_kv4_load(slots, codes, scales, o, p)
    assert hc.hc_read_status() == hc.HC_ERR_BOUNDS
    assert (o[:2] == 0).all() and (o[2] == 1).all() and (p[2] == 1).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

class Case:
    """A cache of random codes with unused slots poisoned, and windows of queries."""

    def __init__(self, seed, lens, q_heads, kv_heads, dim, block, dtype, mask=None, offset=0.0,
                 spread=0.3, q_size=1.0, blocks=0):
        g = np.random.default_rng(seed)
        self.lens, self.block, self.dtype = lens, block, dtype
        n = len(lens)
        kv, new = np.array([x for x, _ in lens]), np.array([y for _, y in lens])
        have = -(-kv // block)
        total = max(int(have.sum()) + 2, blocks)
        order = g.permutation(total)
        width = max(1, int(have.max())) + 1
        self.table = np.full((n, width), -1)
        at = 0
        for b in range(n):
            self.table[b, : have[b]] = order[at:at + have[b]]
            at += have[b]
        self.codes = g.integers(0, 256, (total, 2, kv_heads, block, dim // 2)).astype(np.uint8)
        step = 0.25 * np.exp(spread * g.standard_normal((total, 2, kv_heads, block)))
        low = -7.5 * step + 0.2 * g.standard_normal(step.shape) + offset
        sm = np.stack([step, low], -1)
        used = np.zeros((total, block), dtype=bool)
        for b in range(n):
            for p in range(have[b]):
                used[self.table[b, p], : min(block, kv[b] - p * block)] = True
        poison = np.where(g.random(used.shape) < 0.5, np.nan, np.inf)
        sm = np.where(used[:, None, None, :, None], sm, poison[:, None, None, :, None])
        self.scales = torch.from_numpy(sm).bfloat16()
        self.cu = np.concatenate([[0], np.cumsum(new)])
        self.kv, self.max_new = kv, max(1, int(new.max()))
        tokens = int(new.sum())
        self.q = torch.from_numpy(g.standard_normal((tokens, q_heads, dim)) * q_size).to(DT[dtype])
        self.mask = None
        if mask is not None:
            self.mask = np.array([mask(int(i), int(m), g) for m in new for i in range(m)], dtype=np.uint64)

    def run(self, scale=None, stream=None, max_new=None, q=None):
        q = self.q.cuda() if q is None else q
        out = torch.full(q.shape, 55.0, dtype=q.dtype, device="cuda")
        lse = torch.full(q.shape[:2], 55.0, device="cuda")
        mask = None if self.mask is None else torch.from_numpy(self.mask.view(np.int64)).cuda()
        hc.hc_kv4_attention(q, torch.from_numpy(self.codes).cuda(), self.scales.cuda(), i32(self.table),
                            i32(self.cu), i32(self.kv), max_new or self.max_new, out, lse=lse, mask=mask,
                            scale=scale, stream=stream)
        return out, lse

    def check(self, out, lse, scale=None, tokens=None):
        d = self.q.shape[2]
        scale = 1 / np.sqrt(d) if scale is None else scale
        q, bits = f64(self.q), bits16(self.scales)
        cu, kv, mask, table = self.cu, self.kv, self.mask, self.table
        want, wl, size = W.attention(q, self.codes, bits, table, cu, kv, mask, scale)
        got, gl = f64(out), f64(lse)
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isneginf(gl), np.isneginf(wl))
        sm = bf16_bits_to_f64(bits)
        fine = np.where(np.isfinite(sm), sm, 0)
        step, base = np.abs(fine[..., 0]), np.abs(fine[..., 1] + 8 * fine[..., 0])
        half = 2.0 ** (-8 if self.dtype == "bf16" else -11)
        tol = half * np.abs(want) + 2.0 ** -10 * size + 2.0 ** -24 * 8 * step.max() * max(kv) + 1e-7
        ok = np.isnan(want) | (np.abs(got - want) <= tol)
        assert ok.all(), (np.argwhere(~ok)[:5], got[~ok][:5], want[~ok][:5], tol[~ok][:5])
        terms = abs(scale) * np.abs(q).sum(-1) * (8 * step[:, 0].max() + base[:, 0].max())
        fin = np.isfinite(wl)
        assert (np.abs(gl - wl)[fin] <= (2.0 ** -19 * (1 + terms))[fin]).all()


def causal(i, n, g):
    return (1 << (i + 1)) - 1


def tree(i, n, g):
    return int(g.integers(0, 1 << n)) | (1 << i)


def holes(i, n, g):
    return 0 if i % 3 == 0 else int(g.integers(0, 1 << n))


HEADS = [(8, 8, 64), (8, 2, 128), (20, 4, 128), (7, 1, 64), (32, 4, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("block", [16, 64, 256])
def test_attention_of_single_tokens(heads, dtype, block):
    lens = [(1, 1), (2, 1), (15, 1), (16, 1), (17, 1), (0, 1), (31, 1), (33, 1), (127, 1), (129, 1), (300, 1), (1025, 1)]
    c = Case(1, lens, *heads, block, dtype)
    c.check(*c.run())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("mask", [None, causal, tree, holes], ids=["none", "causal", "tree", "holes"])
def test_attention_of_verify_windows(heads, dtype, mask):
    """Windows of 0 to 8 tokens; lengths that end inside pages and tiles; a request that
    is all window, one shorter than its window (its first tokens see nothing)."""
    lens = [(8, 8), (5, 8), (0, 3), (64, 1), (65, 5), (70, 0), (130, 7), (513, 8), (1000, 2), (0, 0), (1, 1)]
    c = Case(2, lens, *heads, 16, dtype, mask=mask)
    c.check(*c.run())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [(8, 8, 64), (8, 2, 128), (5, 1, 128), (14, 2, 64)], ids=str)
@pytest.mark.parametrize("lens", [[(33, 33)], [(64, 64), (100, 40), (40, 100), (0, 0), (300, 1)],
                                  [(129, 127), (257, 200), (640, 9)], [(700, 300)]], ids=str)
def test_attention_of_chunks(heads, dtype, lens):
    c = Case(3, lens, *heads, 32, dtype)
    c.check(*c.run())


@pytest.mark.parametrize("heads", [(8, 2, 128), (16, 1, 64)], ids=str)
def test_attention_with_masks_of_64_tokens(heads):
    def m(i, n, g):
        return (int(g.integers(0, 1 << 62)) & ((1 << i) - 1)) | (1 << i) if i else 1
    c = Case(4, [(64, 64), (200, 64), (90, 33), (1000, 64)], *heads, 16, "bf16", mask=m)
    c.check(*c.run())


@pytest.mark.parametrize("length", [4096, 20011])
@pytest.mark.parametrize("new", [1, 6, 40])
def test_attention_over_long_caches(length, new):
    """One long request split over many blocks of the launch, beside short ones."""
    c = Case(5, [(length, new), (3, 1), (length // 2, 1)], 8, 2, 128, 64, "bf16")
    c.check(*c.run())


def test_attention_of_many_short_requests():
    g = np.random.default_rng(6)
    lens = [(int(g.integers(0, 90)), int(g.integers(0, 3))) for _ in range(700)]
    c = Case(6, lens, 4, 2, 64, 16, "fp16")
    c.check(*c.run())


@pytest.mark.parametrize("heads", [(8, 8, 64), (8, 4, 128)], ids=str)
def test_attention_of_many_chunks(heads):
    """Chunks of all sizes in one call: blocks of the launch that go through pieces of one
    and of two row tiles, whole and shared, in every order."""
    g = np.random.default_rng(7)
    lens = []
    for _ in range(60):
        new = int(g.integers(0, 300))
        lens.append((new + int(g.integers(0, 700)), new))
    c = Case(7, lens, *heads, 16, "fp16")
    c.check(*c.run())


def test_attention_of_chunks_that_see_no_cache():
    """Requests whose tokens are not in the cache at all: their table rows hold nothing."""
    c = Case(9, [(0, 40), (30, 30), (0, 200), (17, 90)], 8, 2, 128, 16, "bf16")
    c.check(*c.run())


@pytest.mark.parametrize("new", [5, 7, 9, 17, 32])
def test_attention_of_one_window_split_over_the_launch(new):
    c = Case(8, [(16001, new)], 8, 2, 128, 32, "bf16", mask=tree)
    c.check(*c.run())


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kind", ["large q", "small q", "offset", "spread", "zero scale", "negative scale"])
def test_attention_values(kind, dtype, new):
    """Peaked and flat softmaxes, keys and values far from zero, steps over many orders."""
    kw = {"large q": dict(q_size=20.0), "small q": dict(q_size=1e-3), "offset": dict(offset=6.0),
          "spread": dict(spread=2.5)}.get(kind, {})
    scale = {"zero scale": 0.0, "negative scale": -0.05}.get(kind)
    c = Case(7, [(400, new), (90, new)], 8, 2, 64, 16, dtype, **kw)
    c.check(*c.run(scale), scale)


@pytest.mark.parametrize("new", [4, 80])
def test_attention_wide_range_of_bf16_queries(new):
    """bf16 queries far beyond fp16's range, with a scale that brings the logits back."""
    c = Case(8, [(200, new)], 4, 1, 128, 16, "bf16", q_size=1.0)
    for size in (2.0 ** 60, 2.0 ** -60):
        big = Case(8, [(200, new)], 4, 1, 128, 16, "bf16", q_size=1.0)
        big.q = (c.q.double() * size).bfloat16()
        out, lse = big.run(scale=0.09 / size)
        big.check(out, lse, 0.09 / size)


@pytest.mark.parametrize("new", [3, 50])
def test_attention_sees_nan_only_where_it_looks(new):
    """A key group held as NaN makes every row that sees it NaN, a value group too, and
    no other row: those before it in the window, or whose mask hides it."""
    c = Case(9, [(200, new), (60, new)], 4, 2, 64, 16, "bf16")
    at = 200 - 2                                       # the last two tokens of request 0 see it
    page, off = c.table[0][at // 16], at % 16
    c.scales[page, 0, 0, off] = float("nan")           # key of kv head 0
    c.scales[page, 1, 1, off] = float("nan")           # value of kv head 1
    out, lse = c.run()
    rows = out.float().isnan().all(-1).cpu().numpy()
    some = out.float().isnan().any(-1).cpu().numpy()
    assert np.array_equal(rows, some)
    want = np.zeros_like(rows)
    want[new - 2:new] = True
    assert np.array_equal(rows, want)
    assert lse.isnan().cpu().numpy()[:, :2].any() and not lse.isnan().cpu().numpy()[:, 2:].any()


def test_attention_strides_streams_and_repeats():
    """Queries as a slice of fused rows, heads outermost, another stream, and the same
    bits again."""
    c = Case(10, [(300, 5), (77, 3), (1200, 1)], 8, 2, 128, 16, "bf16")
    base = c.run()
    c.check(*base)
    t, h, d = c.q.shape
    fused = torch.full((t, 3 * h * d), 7.0, dtype=c.q.dtype, device="cuda")
    fused[:, h * d:2 * h * d] = c.q.cuda().reshape(t, -1)
    outer = torch.empty(h, t, d, dtype=c.q.dtype, device="cuda")
    outer.copy_(c.q.cuda().transpose(0, 1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for q in (fused[:, h * d:2 * h * d].view(t, h, d), outer.transpose(0, 1)):
        for stream in (None, side):
            out, lse = c.run(q=q, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(out, base[0]) and torch.equal(lse, base[1])


def test_attention_in_a_graph():
    c = Case(11, [(300, 4), (77, 4)], 8, 2, 128, 16, "bf16")
    base = c.run()
    q, codes, scales = c.q.cuda(), torch.from_numpy(c.codes).cuda(), c.scales.cuda()
    table, cu, kv = i32(c.table), i32(c.cu), i32(c.kv)
    out, lse = torch.zeros_like(base[0]), torch.zeros_like(base[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hc.hc_kv4_attention(q, codes, scales, table, cu, kv, 4, out, lse=lse)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, base[0]) and torch.equal(lse, base[1])


def test_attention_of_bad_entries_is_reported():
    c = Case(12, [(100, 2), (50, 2)], 4, 2, 64, 16, "bf16")
    c.table[0, 3] = 1 << 20
    out, lse = c.run()
    assert hc.hc_read_status() == hc.HC_ERR_BOUNDS
    want = Case(12, [(100, 2), (50, 2)], 4, 2, 64, 16, "bf16")
    w = W.attention(f64(want.q)[2:], want.codes, bits16(want.scales), want.table[1:], [0, 2], [50], None, 1 / 8)
    assert np.allclose(f64(out)[2:], w[0], atol=2e-2)
    # more new tokens than max_new says
    c = Case(13, [(100, 5)], 4, 2, 64, 16, "bf16")
    c.run(max_new=3)
    assert hc.hc_read_status() == hc.HC_ERR_BOUNDS
    # a cache longer than its table's row
    c = Case(14, [(64, 1)], 4, 2, 64, 16, "bf16")
    c.kv = np.array([1000])
    c.run()
    assert hc.hc_read_status() == hc.HC_ERR_BOUNDS and hc.hc_read_status() == hc.HC_OK


def test_cache_beyond_32_bits():
    """A pool of 4.6 GB of codes: written, read back and attended at its far end."""
    blocks, h, block, d = 70001, 8, 64, 128
    codes = torch.zeros((blocks, 2, h, block, d // 2), dtype=torch.uint8, device="cuda")
    assert codes.numel() > 1 << 32
    scales = torch.full((blocks, 2, h, block, 2), float("nan"), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(3)
    n = 150
    k, v = (torch.randn(n, h, d, generator=g).bfloat16().cuda() for _ in range(2))
    pages = np.array([blocks - 1, 3, blocks - 2])
    slots = torch.from_numpy(pages[np.arange(n) // block] * block + np.arange(n) % block).cuda()
    hc.hc_kv4_append(k, v, slots, codes, scales)
    ko, vo = torch.empty_like(k, dtype=torch.float32), torch.empty_like(v, dtype=torch.float32)
    hc.hc_kv4_load(slots, codes, scales, ko, vo)
    for x, y in ((k, ko), (v, vo)):
        c, s, m = W.round_group(f64(x))
        assert np.array_equal(f64(y).astype(np.float32), (m[..., None] + s[..., None] * c).astype(np.float32))
    for new in (2, n):
        q = torch.randn(new, 16, d, generator=g).bfloat16().cuda()
        out = torch.empty_like(q)
        hc.hc_kv4_attention(q, codes, scales, i32([pages]), i32([0, new]), i32([n]), new, out)
        a = torch.einsum("thd,jhd->htj", q.double(), ko.double().repeat_interleave(2, 1)) / np.sqrt(d)
        seen = torch.arange(n).cuda()[None] <= (n - new + torch.arange(new).cuda())[:, None]
        p = torch.softmax(a.masked_fill(~seen, float("-inf")), -1)
        want = torch.einsum("htj,jhd->thd", p, vo.double().repeat_interleave(2, 1))
        assert (out.double() - want).abs().max() <= 2.0 ** -8 * want.abs().max()


# ---------------------------------------------------------------------------
# log probabilities
# ---------------------------------------------------------------------------

def run_logprobs(x, ids, top, stream=None):
    t = x.shape[0]
    f = lambda *s: torch.full(s, 77.0, device="cuda")  # noqa: E731
    i = lambda *s: torch.full(s, -77, dtype=torch.int32, device="cuda")  # noqa: E731
    out = dict(logprob=f(t), entropy=f(t), lse=f(t), rank=i(t), top_ids=i(t, top), top_logprobs=f(t, top))
    hc.hc_token_logprobs(x, i32(ids), *out.values(), stream=stream)
    return {k: v.cpu().numpy() for k, v in out.items()}


def check_logprobs(x, ids, top, **kw):
    got, x64 = run_logprobs(x, ids, top, **kw), f64(x)
    want = W.logprobs(x64, np.asarray(ids), top)
    for name in ("rank", "top_ids"):
        assert np.array_equal(got[name], want[name]), (name, got[name][:3], want[name][:3])
    peak = np.abs(np.where(np.isfinite(x64), x64, 0)).max(-1)
    tol = 2.0 ** -20 * (1 + peak + np.log(x.shape[1]))
    for name in ("logprob", "entropy", "lse", "top_logprobs"):
        g, w = got[name].astype(np.float64), want[name]
        t = tol if g.ndim == 1 else tol[:, None]
        same = (g == w) | (np.abs(np.where(np.isfinite(g), g, 0) - np.where(np.isfinite(w), w, 0)) <= t)
        assert (same & (np.isfinite(g) == np.isfinite(w))).all(), name


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab,top", [
    (1, 1, 1), (1, 7, 7), (3, 33, 0), (2, 1000, 32), (1, 32000, 8), (5, 50257, 5), (40, 4099, 20),
    (300, 2048, 1), (1, 200003, 32), (9, 131072, 10)])
def test_logprobs(dtype, rows, vocab, top):
    g = np.random.default_rng(rows + vocab)
    x = torch.from_numpy(g.standard_normal((rows, vocab)) * 3).to(DT[dtype]).cuda()
    ids = g.integers(0, vocab, rows)
    ids[0] = int(x[0].float().argmax())
    check_logprobs(x, ids, top)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab", [8, 1003, 70001])
def test_logprobs_of_difficult_rows(dtype, vocab):
    """All equal; all -inf; one finite; -inf but for a few; a huge peak; very negative;
    the type's lowest value; ascending and descending (every element beats the last)."""
    low = torch.finfo(DT[dtype]).min
    x = torch.zeros(11, vocab, dtype=torch.float64)
    x[1] = float("-inf")
    x[2] = float("-inf")
    x[2, vocab - 1] = -4.5
    x[3] = float("-inf")
    x[3, ::5] = torch.arange(len(x[3, ::5]), dtype=torch.float64) * -0.25
    x[4, vocab // 2] = 1e30
    x[5] = -1e30
    x[6] = low
    x[6, 1] = 3.0
    x[7] = low
    x[8] = torch.arange(vocab, dtype=torch.float64) * 1e-3
    x[9] = -x[8]
    x[10, 1::2] = -0.0
    x = x.to(DT[dtype]).cuda()
    ids = np.array([0, 3, vocab - 1, 1, vocab // 2, 2, 1, 0, 0, vocab - 1, 5])
    check_logprobs(x, ids, min(8, vocab))
    check_logprobs(x, np.array([-1, vocab, 1 << 30, -(1 << 31)] + [0] * 7), 3)


def test_logprobs_strides_ties_and_streams():
    g = np.random.default_rng(5)
    wide = torch.from_numpy(np.round(g.standard_normal((6, 3001)) * 2)).bfloat16().cuda()   # many ties
    ids = g.integers(0, 900, 6)
    for lo in range(4):
        check_logprobs(wide[:, lo:lo + 900 + lo], ids, 32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check_logprobs(wide[::2], ids[::2], 5, stream=side)
    side.synchronize()
    one = torch.from_numpy(g.standard_normal((1, 700))).bfloat16().cuda().expand(4, 700)     # row stride 0
    check_logprobs(one, ids[:4] % 700, 4)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_logprobs_of_rows_that_are_not_finite(bad):
    x = torch.randn(3, 5000, device="cuda")
    x[1, 1234] = bad
    r = run_logprobs(x, [1, 2, 3], 4)
    for name in ("logprob", "entropy", "top_logprobs"):
        assert np.isnan(r[name][1]).all() and np.isfinite(r[name][[0, 2]]).all(), name
    assert not np.isfinite(r["lse"][1])


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def refuses(f, *args, **kw):
    with pytest.raises(hc.HcReadError) as e:
        f(*args, **kw)
    assert e.value.code == hc.HC_ERR_ARG


def test_refusals_of_the_cache_operators():
    codes, scales = blank_cache(2, 2, 16, 64)
    k = torch.ones(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    slots = torch.arange(4).cuda()
    for dim, block in ((96, 16), (64, 24), (64, 512), (32, 16)):
        c, s = blank_cache(1, 2, block, dim)
        refuses(hc.hc_kv4_append, torch.ones(4, 2, dim, device="cuda"), torch.ones(4, 2, dim, device="cuda"), slots, c, s)
    refuses(hc.hc_kv4_append, k.cpu(), k, slots, codes, scales)                 # host memory
    refuses(hc.hc_kv4_append, k, k, slots.cpu(), codes, scales)
    odd = torch.ones(4, 2 * 64 + 4, device="cuda", dtype=torch.bfloat16)
    refuses(hc.hc_kv4_append, odd[:, :128].view(4, 2, 64), k, slots, codes, scales)   # stride not 16 bytes
    off = torch.ones(4 * 128 + 8, device="cuda", dtype=torch.bfloat16)[1:513].view(4, 2, 64)
    refuses(hc.hc_kv4_append, off, k, slots, codes, scales)                     # base not 16 bytes
    refuses(hc.hc_kv4_load, slots, codes, scales, k, k)                         # outputs overlap
    refuses(hc.hc_kv4_load, slots, codes, scales, k, k.float())
    refuses(hc.hc_kv4_append, codes.view(torch.bfloat16)[:1, 0, 0, :4].reshape(4, 1, -1).expand(4, 2, 16), k, slots, codes, scales)


def test_refusals_of_attention():
    c = Case(20, [(40, 2)], 4, 2, 64, 16, "bf16")
    q, codes, scales = c.q.cuda(), torch.from_numpy(c.codes).cuda(), c.scales.cuda()
    table, cu, kv, out = i32(c.table), i32(c.cu), i32(c.kv), torch.zeros_like(c.q).cuda()
    lse = torch.zeros(2, 4, device="cuda")
    ok = dict(q=q, codes=codes, scales=scales, block_table=table, cu_lens=cu, kv_lens=kv, max_new=2, out=out)
    hc.hc_kv4_attention(**ok)
    hc.hc_kv4_attention(**dict(ok, max_new=0))                                   # nothing to do
    mask = torch.ones(2, dtype=torch.int64, device="cuda")
    for bad in (dict(max_new=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(out=q),
                dict(q=q.float(), out=out.float()), dict(q=q[:, :3], out=out[:, :3].contiguous()),
                dict(lse=lse.half()), dict(lse=lse[:1]), dict(mask=mask, max_new=65), dict(mask=mask[:1]),
                dict(cu_lens=cu.cpu()), dict(kv_lens=kv.long()), dict(out=out.half()),
                dict(block_table=table[0])):
        refuses(hc.hc_kv4_attention, **dict(ok, **bad))
    many = torch.zeros(1, 2 * 129, 64, dtype=torch.bfloat16, device="cuda")
    refuses(hc.hc_kv4_attention, **dict(ok, q=many, out=torch.zeros_like(many)))


def test_refusals_of_plan_and_logprobs():
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    slots = torch.zeros(8, dtype=torch.int64, device="cuda")
    good = dict(cached_lens=z(2), new_lens=z(2), free_blocks=z(4), free_count=z(1), block_size=16,
                block_table=z(2, 4), slots=slots, request_of=z(8), positions=z(8), cu_lens=z(3),
                kv_lens=z(2), free_left=z(1))
    hc.hc_window_plan(**good)
    for bad in (dict(block_size=20), dict(block_size=8), dict(block_size=0), dict(free_left=good["free_count"]),
                dict(kv_lens=good["cached_lens"]), dict(cached_lens=z(2).cpu()), dict(slots=slots.int())):
        refuses(hc.hc_window_plan, **dict(good, **bad))
    n = hc.HC_PLAN_MAX_REQUESTS + 1
    refuses(hc.hc_window_plan, **dict(good, cached_lens=z(n), new_lens=z(n), block_table=z(n, 4), cu_lens=z(n + 1),
                                      kv_lens=z(n)))
    x, ids = torch.zeros(2, 40, device="cuda"), z(2)
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    out = [f(2), f(2), f(2), z(2), z(2, 4), f(2, 4)]
    hc.hc_token_logprobs(x, ids, *out)
    refuses(hc.hc_token_logprobs, x, ids, *out[:4], z(2, 33), f(2, 33))           # more than 32
    refuses(hc.hc_token_logprobs, x[:, :3], ids, *out)                            # more than the vocabulary
    refuses(hc.hc_token_logprobs, x.double(), ids, *out)
    refuses(hc.hc_token_logprobs, x.t().contiguous().t(), ids, *out)              # columns strided
    refuses(hc.hc_token_logprobs, x, ids, out[0], out[0], *out[2:])               # outputs overlap
    refuses(hc.hc_token_logprobs, x, ids.long(), *out)


def test_calls_of_nothing():
    codes, scales = blank_cache(1, 1, 16, 64)
    e = torch.empty(0, 1, 64, device="cuda")
    s = torch.empty(0, dtype=torch.int64, device="cuda")
    hc.hc_kv4_append(e, e, s, codes, scales)
    hc.hc_kv4_load(s, codes, scales, e, e.clone())
    f = torch.empty(0, device="cuda")
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    hc.hc_token_logprobs(torch.empty(0, 5, device="cuda"), i, f, f, f, i, i.view(0, 2), f.view(0, 2))
    hc.hc_kv4_attention(e.bfloat16(), codes, scales, i.view(0, 3), i32([0]), i, 1, e.bfloat16())
    hc.hc_kv4_attention(e.bfloat16(), codes, scales, i32([[0]]), i32([0, 0]), i32([5]), 1, e.bfloat16())
