"""The verify-window operators at the edges of what their header allows: lengths next to
2^31, values of very different sizes in one call, NaN, and entries that are not valid.
Against the 64-bit oracle (oracle/window_oracle.py) or exact expectations."""
import numpy as np
import pytest
import torch

import hyper_connection_residual_read_gb300 as hc

from oracle import window_oracle as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def context():
    hc.hc_read_init(0, 64, 1e-6)
    yield
    assert hc.hc_read_status() == hc.HC_OK


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


# ---------------------------------------------------------------------------
# lengths next to 2^31
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("cached,new", [(2 ** 31 - 300, 200), (2 ** 31 - 200, 150), (2 ** 31 - 2, 1), (2 ** 31 - 256, 9)])
def test_plan_of_lengths_next_to_the_largest(cached, new):
    """A table row that covers 2^31 tokens: blocks held are told from new ones in every
    token's slot and in the table."""
    block, width = 256, 1 << 23
    table = np.full((1, width), 5)
    have = -(-cached // block)
    table[0, have - 1] = 77
    free = np.arange(100, 107)
    out = [torch.full((new + 3,), -9, dtype=torch.int64, device="cuda"), i32([-9] * (new + 3)), i32([-9] * (new + 3)),
           i32([0, 0]), i32([0]), i32([0])]
    t = i32(table)
    hc.hc_window_plan(i32([cached]), i32([new]), i32(free), i32([len(free)]), block, t, *out)
    want = W.plan([cached], [new], free, len(free), block, table, new + 3)
    got = [t.cpu().numpy(), *[x.cpu().numpy() for x in out[:5]], int(out[5])]
    for name, x, y in zip(("table", "slots", "request_of", "positions", "cu", "kv", "left"), got, want):
        assert np.array_equal(x, y), name
    assert got[5].tolist() == [cached + new]


def test_calls_of_the_most_tokens():
    """2^31 - 1 tokens: a plan whose arrays have room for as many, and a write of one key and
    value (strides of 0) to as many slots, of which two are."""
    n = 2 ** 31 - 1
    slots = torch.full((n,), -9, dtype=torch.int64, device="cuda")
    of, at = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    cu, kv, left, table = i32([0] * 3), i32([0] * 2), i32([0]), i32([[0, 0], [0, 0]])
    hc.hc_window_plan(i32([0, 5]), i32([20, 3]), i32([7, 8, 9]), i32([3]), 16, table, slots, of, at, cu, kv, left)
    assert cu.tolist() == [0, 20, 23] and kv.tolist() == [20, 8] and int(left) == 1
    assert slots[:24].tolist() == [9 * 16 + i for i in range(16)] + [8 * 16 + i for i in range(4)] + [5, 6, 7, -1]
    for x in (slots, of, at):
        assert bool((x[23:24] == -1).all()) and bool((x[-5000:] == -1).all()) and int((x[:: 2 ** 20] == -9).sum()) == 0
    del of, at
    slots[:23] = -1
    slots[1], slots[-1] = 3, 17
    codes = torch.zeros((2, 2, 1, 16, 32), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((2, 2, 1, 16, 2), dtype=torch.bfloat16, device="cuda")
    one = torch.ones(64, device="cuda").bfloat16().expand(n, 1, 64)
    hc.hc_kv4_append(one, one, slots, codes, scales)
    want = torch.zeros_like(scales)
    want[0, :, 0, 3, 1] = want[1, :, 0, 1, 1] = 1.0
    assert torch.equal(scales, want) and not codes.any()
    assert hc.hc_read_status() == hc.HC_OK


@pytest.mark.parametrize("q_heads,new", [(8, 1), (4, 3), (1, 40)])
def test_attention_over_lengths_next_to_the_largest(q_heads, new):
    """2^31 - 1 tokens: all pages but the last are one block, and the last one's keys have
    logits that make up for their number; the slot behind the end is NaN. A lane sums up to
    2^17 terms or tiles in fp32, 2^-8 relative at worst: so much of lse, and of values 4
    apart twice that, and half an ulp of bf16 below 8."""
    d, block, width, kv = 64, 256, 1 << 23, 2 ** 31 - 1
    g = np.random.default_rng(3)
    codes = g.integers(0, 256, (2, 2, 1, block, d // 2)).astype(np.uint8)
    step = np.full((2, 2, 1, block), 0.125)
    low = np.full(step.shape, -0.9375)
    low[1, 0] += 2.0                                    # sum(q) is near 64: exp(16) times as much weight a key
    low[1, 1] += 4.0
    q = torch.from_numpy(1 + 0.15 * g.standard_normal((new, q_heads, d))).bfloat16()
    scales = torch.from_numpy(np.stack([step, low], -1)).bfloat16().cuda()
    scales[1, :, :, 255] = float("nan")
    table = torch.zeros((1, width), dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    out = torch.zeros_like(q).cuda()
    lse = torch.zeros((new, q_heads), device="cuda")
    hc.hc_kv4_attention(q.cuda(), torch.from_numpy(codes).cuda(), scales, table, i32([0, new]), i32([kv]), new, out, lse=lse)
    assert hc.hc_read_status() == hc.HC_OK
    value = low[..., None] + step[..., None] * W.unpack(codes)              # [block][kv][1][token][d]
    x = np.einsum("nhd,btd->nhbt", q.double().numpy(), value[:, 0, 0]) / 8
    times = np.ones((new, 2, block))
    times[:, 0] = width - 1
    for i in range(new):
        times[i, 1, 255 - new + i + 1:] = 0
    p = np.exp(x) * times[:, None]
    part = p[:, :, 1].sum(-1) / p.sum((-1, -2))
    assert 0.05 < part.min() and part.max() < 0.95, "the last page matters, and not alone"
    want_lse = np.log(p.sum((-1, -2)))
    want = np.einsum("nhbt,btd->nhd", p, value[:, 1, 0]) / p.sum((-1, -2))[..., None]
    assert np.abs(lse.double().cpu().numpy() - want_lse).max() <= 2.0 ** -8
    assert np.abs(out.double().cpu().numpy() - want).max() <= 2 * 4 * 2.0 ** -8 + 2.0 ** -6


# ---------------------------------------------------------------------------
# attention: values
# ---------------------------------------------------------------------------

class Cache:
    """Requests of (cached + new, new) tokens in a shuffled pool, from given steps and minima."""

    def __init__(self, seed, lens, kv_heads, dim, block=16, spread=0.3):
        g = np.random.default_rng(seed)
        self.lens, self.block, self.dim = lens, block, dim
        have = [-(-kv // block) for kv, _ in lens]
        order, at = g.permutation(sum(have) + 1), 0
        self.table = np.full((len(lens), max(1, max(have))), -1)
        for b, n in enumerate(have):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (sum(have) + 1, 2, kv_heads, block)
        self.codes = g.integers(0, 256, (*shape, dim // 2)).astype(np.uint8)
        step = 0.25 * np.exp(spread * g.standard_normal(shape))
        self.scales = np.stack([step, -7.5 * step + 0.2 * g.standard_normal(shape)], -1)
        self.cu = np.concatenate([[0], np.cumsum([n for _, n in lens])])
        self.kv = np.array([kv for kv, _ in lens])

    def set(self, request, position, kind, head, step, low):
        """The group of a token: kind 0 its key, 1 its value."""
        at = self.table[request, position // self.block], kind, head, position % self.block
        self.scales[at] = step, low

    def run(self, q, mask=None, scale=None):
        """out and lse in float64."""
        out = torch.full(q.shape, 55.0, dtype=q.dtype, device="cuda")
        lse = torch.full(q.shape[:2], 55.0, device="cuda")
        bits = None if mask is None else torch.from_numpy(np.array(mask, dtype=np.uint64).view(np.int64)).cuda()
        hc.hc_kv4_attention(q.cuda(), torch.from_numpy(self.codes).cuda(), torch.from_numpy(self.scales).bfloat16().cuda(),
                            i32(self.table), i32(self.cu), i32(self.kv), max(n for _, n in self.lens), out, lse=lse, mask=bits,
                            scale=scale)
        assert hc.hc_read_status() == hc.HC_OK
        return out.double().cpu().numpy(), lse.double().cpu().numpy()

    def queries(self, heads, dtype=torch.bfloat16, seed=0):
        g = torch.Generator().manual_seed(seed)
        return torch.randn(int(self.cu[-1]), heads, self.dim, generator=g).to(dtype)


def expect(c, q, mask=None, scale=None):
    """In 64 bits, request by request: out, lse, and what each may be off by. out: half an
    ulp of its type; 2^-10 of sum p (|s (c - 8)| + |m + 8 s|), as each weight is rounded to
    11 bits and carries its exponent's error; and for weights below 16 bits' range, of
    every key, 2^-22 of the largest p s. lse: 2^-19 of 1 + the largest sum of a logit's
    terms. All of it of the keys that the row sees, and of no others."""
    scale = c.dim ** -0.5 if scale is None else scale
    bits = torch.from_numpy(c.scales).bfloat16().double().numpy()
    half = 2.0 ** (-8 if q.dtype == torch.bfloat16 else -11)
    heads, x = q.shape[1], q.double().numpy()
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    lse, lse_tol = np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2])
    for b, (kv, new) in enumerate(c.lens):
        if not kv:
            continue
        at = np.arange(kv)
        page, off = c.table[b][at // c.block], at % c.block
        code = W.unpack(c.codes[page, :, :, off]).astype(np.float64)                 # [kv][2][h][d]
        s, m = (bits[page, :, :, off][..., i:i + 1] for i in (0, 1))
        value, terms = m + s * code, np.abs(s * (code - 8)) + np.abs(m + 8 * s)
        rows = slice(c.cu[b], c.cu[b + 1])
        if mask is None:
            sees = at[None] <= (kv - new + np.arange(new))[:, None]
        else:
            back = at - (kv - new)
            sees = (back < 0)[None] | (((np.array(mask[rows], dtype=object)[:, None] >> np.maximum(back, 0)[None]) & 1) == 1)
        for h in range(heads):
            g = h // (heads // value.shape[2])
            z = np.where(sees, scale * (x[rows, h] @ value[:, 0, g].T), -np.inf)
            size = np.where(sees, abs(scale) * (np.abs(x[rows, h]) @ terms[:, 0, g].T), 0.0)
            top = z.max(-1, keepdims=True)
            p = np.where(sees, np.exp(z - np.where(np.isfinite(top), top, 0)), 0.0)
            total = p.sum(-1, keepdims=True)
            with np.errstate(divide="ignore", invalid="ignore"):
                lse[rows, h] = (top + np.log(total))[:, 0]
                p = p / np.where(total > 0, total, 1)
            out[rows, h] = np.where(p > 0, p, 0) @ value[:, 1, g]
            tol[rows, h] = half * np.abs(out[rows, h]) + 2.0 ** -10 * (p @ terms[:, 1, g]) + \
                2.0 ** -22 * kv * (p * s[:, 1, g, 0]).max(-1, keepdims=True) + 1e-30
            lse_tol[rows, h] = 2.0 ** -19 * (1 + size.max(-1))
            if kv > 1:
                second = np.partition(z, -2, axis=-1)[:, -2]
                with np.errstate(invalid="ignore"):
                    gap = np.where(np.isfinite(second), top[:, 0] - second, np.inf)
                    other = np.minimum(1.0, kv * np.exp(np.minimum(2 * lse_tol[rows, h] - gap, 0)))
                tol[rows, h] += np.where(lse_tol[rows, h] > 2.0 ** -9, other * 2 * np.abs(value[:, 1, g]).max(), 0)[:, None]
    return out, lse, tol, lse_tol


def agrees(c, q, mask=None, scale=None, rows=None):
    """The rows (all of them) of a call with what `expect` says."""
    out, lse = c.run(q, mask, scale)
    want, want_lse, tol, lse_tol = expect(c, q, mask, scale)
    rows = np.ones(lse.shape, dtype=bool) if rows is None else rows
    # what q's type cannot hold is an infinity of the same sign
    with np.errstate(invalid="ignore"):
        beyond = (np.abs(want) + tol >= torch.finfo(q.dtype).max) & (out == np.sign(want) * np.inf)
        off, lse_off = np.where(beyond, 0, np.abs(out - want))[rows], np.abs(lse - want_lse)[rows & np.isfinite(want_lse)]
    assert np.array_equal(np.isneginf(lse[rows]), np.isneginf(want_lse[rows]))
    assert (off <= tol[rows]).all(), ("out", (off / tol[rows]).max())
    assert (lse_off <= lse_tol[rows & np.isfinite(want_lse)]).all(), ("lse", (lse_off / lse_tol[rows & np.isfinite(want_lse)]).max())


# query heads on one kv head, new tokens: each form of the two kernels (8 and 16 rows; 128
# rows, and more)
FORMS = [(4, 1), (3, 2), (5, 3), (4, 4), (10, 4), (2, 150)]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,new", FORMS)
@pytest.mark.parametrize("kv", [1, 33, 700, 20000])
def test_attention_that_sees_nothing_but_nan_is_nan(q_heads, new, dim, kv):
    """Keys held as NaN alone; and queries that are NaN, beside rows that are not."""
    new = min(new, kv)
    c = Cache(1, [(kv, new), (50, new)], 1, dim)
    c.set(0, np.arange(kv), 0, 0, np.nan, np.nan)
    out, lse = c.run(c.queries(q_heads))
    assert np.isnan(out[:new]).all() and np.isnan(lse[:new]).all()
    assert not np.isnan(out[new:]).any() and not np.isnan(lse[new:]).any()
    c = Cache(2, [(kv, new), (50, new)], 1, dim)
    q = c.queries(q_heads)
    q[0, 0, 3] = q[-1, q_heads - 1, 0] = float("nan")
    out, lse = c.run(q)
    bad = np.zeros(lse.shape, dtype=bool)
    bad[0, 0] = bad[-1, q_heads - 1] = True
    assert np.isnan(out[bad]).all() and np.isnan(lse[bad]).all()
    agrees(c, q, rows=~bad)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,new", FORMS)
@pytest.mark.parametrize("size", [2.0 ** 14, 2.0 ** 100, 3e38])
def test_values_of_keys_that_weigh_nothing_cost_no_bits(q_heads, new, dim, dtype, size):
    """Values far larger than the others, of the window's last token, which only its own row
    sees (their first dimension aside they are 0: not to be seen is not to matter), and of
    keys whose weight is next to nothing."""
    c = Cache(3, [(300, new), (2000, new), (37, new)], 1, dim)
    q = c.queries(q_heads, dtype) * 0.5 + 1
    for b, (kv, _) in enumerate(c.lens):
        if new > 1:
            c.set(b, kv - 1, 1, 0, size / 20, -size / 3)
        for position in (0, 18, kv // 2):
            c.set(b, position, 0, 0, 0.01, -20.0)       # a logit below -150 where sum(q) is near dim
            c.set(b, position, 1, 0, min(size, 2.0 ** 60), 0.0)
    rows = np.ones((int(c.cu[-1]), q_heads), dtype=bool)
    if new > 1:
        rows[c.cu[1:] - 1] = False                      # the rows that see the large one
    agrees(c, q, rows=rows)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,new", FORMS)
def test_queries_of_different_sizes_in_one_call(q_heads, new, dim):
    """Rows 2^24 apart, and rows beyond fp16's range beside one with an infinity: each row
    has the bits of its own size."""
    c = Cache(4, [(300, new), (2000, new), (37, min(new, 37))], 1, dim)
    q = c.queries(q_heads)
    i = torch.arange(q.shape[0])[:, None] + torch.arange(q_heads)[None]
    agrees(c, q * torch.exp2(-24.0 * (i % 3 == 0) + 24.0 * (i % 3 == 1))[..., None].bfloat16())
    big = q * 2.0 ** 20
    big[0, 0, 5] = float("inf")
    rows = np.ones(q.shape[:2], dtype=bool)
    rows[0, 0] = False
    agrees(c, big, scale=2.0 ** -23, rows=rows)


@pytest.mark.parametrize("q_heads,new", FORMS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("up", [7, 8, 9, 12, 30, 100, 125])
def test_keys_and_values_below_one_that_is_not_seen(q_heads, new, dim, up):
    """The window's last token, which its own row alone sees, has a key and a value 2^up above
    the others, whose steps have odd significands (all 8 bits are needed): it costs the
    other rows nothing. With a mask too, where a token in the middle of the window is hidden."""
    c = Cache(5, [(300, new), (2000, new), (140, min(new, 140))], 2, dim, spread=0)
    g = np.random.default_rng(up)
    c.scales[..., 0] = (129 + 2 * g.integers(0, 63, c.scales.shape[:-1])) / 1024.0
    c.scales[..., 1] = -7.5 * c.scales[..., 0] + 0.2 * g.standard_normal(c.scales.shape[:-1])
    q = c.queries(2 * q_heads, torch.float16)
    if new == 1:
        return agrees(c, q)
    size = 2.0 ** min(up, 124)
    hidden = [kv - 1 for kv, _ in c.lens]
    for b, at in enumerate(hidden):
        for kind in (0, 1):
            for head in (0, 1):
                c.set(b, at, kind, head, size / 8, -size)
    rows = np.ones((int(c.cu[-1]), 2 * q_heads), dtype=bool)
    rows[c.cu[1:] - 1] = False
    agrees(c, q, rows=rows)
    if new <= 64:
        mask = [((1 << (i + 1)) - 1) & ~1 for _, n in c.lens for i in range(n)]      # nobody sees the window's first
        for b, at in enumerate(hidden):
            first = c.lens[b][0] - c.lens[b][1]
            old = c.table[b, at // 16], at % 16
            put = c.table[b, first // 16], first % 16
            c.scales[put[0], :, :, put[1]], c.scales[old[0], :, :, old[1]] = \
                c.scales[old[0], :, :, old[1]].copy(), c.scales[put[0], :, :, put[1]].copy()
        agrees(c, q, mask=mask)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q_heads,new", FORMS)
@pytest.mark.parametrize("spread", [1.0, 2.5, 8.0])
def test_steps_over_many_orders(q_heads, new, spread, dtype):
    """Steps of keys and values spread over up to 2^70, all of them seen by some row."""
    c = Cache(6, [(400, new), (1100, new), (90, min(new, 90))], 2, 64, spread=spread)
    q = c.queries(2 * q_heads, dtype)
    agrees(c, q * (0.25 ** 4 if spread == 8.0 else 1.0), scale=2.0 ** -12 if spread == 8.0 else None)


@pytest.mark.parametrize("q_heads,new", FORMS)
def test_values_that_fall_and_rise_by_tiles(q_heads, new):
    """Values whose size changes from one stretch of 128 tokens to the next, by more than a
    tile's range, up and down; constants and zeros among them."""
    c = Cache(7, [(1500, new), (1030, new)], 1, 128)
    for b, (kv, _) in enumerate(c.lens):
        for tile in range(-(-kv // 128)):
            at = np.arange(tile * 128, min(kv, tile * 128 + 128))
            size = 2.0 ** [0, 12, -14, -13, 40, 39, -70, 3, 0, 0, 30, -30][tile]
            index = c.table[b, at // 16], 1, slice(None), at % 16
            c.scales[index] = c.scales[index] * size
        c.set(b, np.arange(256, 300), 1, 0, 0.0, 0.0)
        c.set(b, np.arange(900, 1000), 1, 0, 0.0, 1.5)
        c.set(b, np.arange(600, 640), 0, 0, 0.0, 0.25)
    agrees(c, c.queries(q_heads) * 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,new", FORMS)
@pytest.mark.parametrize("up", [6, 13, 20, 45])
def test_values_as_large_as_their_weights_are_small(q_heads, new, dim, dtype, up):
    """Stretches of tokens whose values are 2^up above the others' and whose weights are about
    2^-up of theirs, so that both matter; after ordinary ones, before them, and among them (in so many requests that a block of
    the launch has several tiles of one)."""
    c = Cache(8, [(900, new)] * 24, 4, dim)
    q = (1 + 0.05 * c.queries(4 * q_heads)).to(dtype)
    c.scales[:, 1] /= 16                                # within fp16's range
    down = up * np.log(2) / dim ** 0.5                   # of a key's minimum, which sum(q) = dim multiplies
    for b, at in enumerate((np.arange(384, 640), np.arange(0, 200), np.arange(3, 700, 7))):
        page = c.table[b, at // 16], at % 16
        c.scales[page[0], 0, 0, page[1], 1] -= down
        c.scales[page[0], 1, 0, page[1]] *= 2.0 ** up
    agrees(c, q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,new", FORMS)
def test_sizes_that_change_within_the_tiles_of_one_block(q_heads, new, dim, dtype):
    """Many requests, so that a block of the launch goes through several tiles of one: values
    and keys whose sizes change from tile to tile, wide tiles among ordinary ones, and a
    large key and value that only the window's last row sees."""
    g = np.random.default_rng(9)
    c = Cache(9, [(1300, new)] * 16, 4, dim)
    sizes = [0, 0, 3, -9, 11, -12, 2, 14, -30, 0, 1]
    for b in range(16):
        order = g.permutation(sizes)
        for tile in range(11):
            at = np.arange(tile * 128, min(1300, tile * 128 + 128))
            page = c.table[b, at // 16], at % 16
            c.scales[page[0], 1, :, page[1]] *= 2.0 ** order[tile]
            if tile % 4 == b % 4:                           # keys too, of some tokens of some tiles
                some = at[g.random(len(at)) < 0.2]
                c.scales[c.table[b, some // 16], 0, :, some % 16] *= 2.0 ** -11
                c.scales[c.table[b, some // 16], 1, :, some % 16] *= 2.0 ** g.integers(-14, 3)
        if new > 1 and b % 2:
            for head in range(4):
                c.set(b, 1299, 0, head, 2.0 ** 40, 0.0)
                c.set(b, 1299, 1, head, 2.0 ** 70, 0.0)
    rows = np.ones((int(c.cu[-1]), 4 * q_heads), dtype=bool)
    rows[c.cu[1:] - 1] = new == 1
    agrees(c, c.queries(4 * q_heads, dtype), rows=rows)


# ---------------------------------------------------------------------------
# arguments
# ---------------------------------------------------------------------------

def test_more_kv_heads_than_a_launch_has_room_for_are_refused():
    heads = 65536
    codes = torch.zeros((1, 2, heads, 16, 32), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((1, 2, heads, 16, 2), dtype=torch.bfloat16, device="cuda")
    k, slots = torch.ones((1, heads, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    for call in (lambda: hc.hc_kv4_append(k, k, slots, codes, scales),
                 lambda: hc.hc_kv4_load(slots, codes, scales, torch.empty_like(k), torch.empty_like(k)),
                 lambda: hc.hc_kv4_attention(k, codes, scales, i32([[0]]), i32([0, 1]), i32([1]), 1, torch.empty_like(k))):
        with pytest.raises(hc.HcReadError) as e:
            call()
        assert e.value.code == hc.HC_ERR_ARG
    fewer = heads - 1
    codes, scales, k = codes[:, :, :fewer].contiguous(), scales[:, :, :fewer].contiguous(), k[:, :fewer].contiguous()
    hc.hc_kv4_append(k, k, slots, codes, scales)
    o, p = torch.empty_like(k), torch.empty_like(k)
    hc.hc_kv4_load(slots, codes, scales, o, p)
    assert torch.equal(o, k) and torch.equal(p, k)
    hc.hc_kv4_attention(k, codes, scales, i32([[0]]), i32([0, 1]), i32([1]), 1, o)
    assert torch.equal(o, k)


def test_the_stride_of_an_axis_of_one_does_not_matter():
    """One token, or one head, of rows of an odd length: what torch gives as that axis's
    stride is never used; another axis's still has to be whole 16 bytes."""
    wide = torch.randn(4 * 67, device="cuda").bfloat16()
    codes = torch.zeros((1, 2, 4, 16, 32), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((1, 2, 4, 16, 2), dtype=torch.bfloat16, device="cuda")
    one, odd = wide.as_strided((1, 4, 64), (67, 64, 1)), wide.as_strided((4, 1, 64), (64, 3, 1))
    slots = torch.zeros(1, dtype=torch.int64, device="cuda")
    back = torch.zeros((2, 1, 4, 64), device="cuda")
    hc.hc_kv4_append(one, one, slots, codes, scales)
    hc.hc_kv4_load(slots, codes, scales, back[0], back[1])
    want, s, m = (torch.from_numpy(np.asarray(x, dtype=np.float32)) for x in W.round_group(one[0].double().cpu().numpy()))
    assert torch.equal(back[0, 0].cpu(), m[:, None] + s[:, None] * want) and torch.equal(back[0], back[1])
    out = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    for q, o in ((one, out[0]), (one.contiguous().clone(), out[1])):
        hc.hc_kv4_attention(q, codes, scales, i32([[0]]), i32([0, 1]), i32([1]), 1, o)
    assert torch.equal(out[0], out[1]) and out.any()
    single = codes[:, :, :1].contiguous(), scales[:, :, :1].contiguous()
    hc.hc_kv4_append(odd, odd, torch.arange(4).cuda(), *single)
    other = codes[:, :, :1].contiguous(), scales[:, :, :1].contiguous()
    hc.hc_kv4_append(odd.contiguous().clone(), odd.contiguous().clone(), torch.arange(4).cuda(), *other)
    assert torch.equal(single[0], other[0]) and torch.equal(single[1].view(torch.int16), other[1].view(torch.int16))
    bad = torch.randn(4 * 67, device="cuda").bfloat16().as_strided((4, 1, 64), (67, 64, 1))
    with pytest.raises(hc.HcReadError) as e:
        hc.hc_kv4_append(bad, bad, torch.arange(4).cuda(), *single)
    assert e.value.code == hc.HC_ERR_ARG


# ---------------------------------------------------------------------------
# entries that are not valid
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("bad", ["held", "free"])
def test_plan_reports_blocks_that_are_none(bad):
    """A negative id of a block that the request holds, or of one on the free list: its tokens
    have no slot, which the write would skip without a word; the others' are right."""
    held, free = [-1 if bad == "held" else 4, 9], [3, 2, -7 if bad == "free" else 1]
    table = i32([[held[0], 55], [held[1], 55]])
    out = [torch.full((24,), -9, dtype=torch.int64, device="cuda"), i32([-9] * 24), i32([-9] * 24), i32([0] * 3), i32([0] * 2), i32([0])]
    hc.hc_window_plan(i32([10, 12]), i32([12, 10]), i32(free), i32([3]), 16, table, *out)
    assert hc.hc_read_status() == hc.HC_ERR_BOUNDS and hc.hc_read_status() == hc.HC_OK
    blocks = [[held[0], free[2]], [held[1], free[1]]]
    want = [blocks[b][p // 16] * 16 + p % 16 if blocks[b][p // 16] >= 0 else -1
            for b, (c, n) in enumerate(((10, 12), (12, 10))) for p in range(c, c + n)]
    assert out[0].tolist() == want + [-1] * 2 and out[4].tolist() == [22, 22] and int(out[5]) == 1


def test_a_slot_given_twice_holds_words_of_either_token_and_spoils_no_other():
    """Duplicates within a warp, between warps and between blocks of the launch: each 32-bit
    word is that of one of the tokens, and all other slots are as if there were none."""
    g = torch.Generator().manual_seed(2)
    tokens, heads, dim, block = 3000, 2, 128, 16
    k, v = (torch.randn(tokens, heads, dim, generator=g).bfloat16().cuda() for _ in range(2))
    slots = torch.randperm(4000, generator=g)[:tokens]
    pairs = [(0, 1), (5, 40), (7, 2900), (100, 1500)]
    for a, b in pairs:
        slots[b] = slots[a]

    def written(keep):
        codes = torch.zeros((250, 2, heads, block, dim // 2), dtype=torch.uint8, device="cuda")
        scales = torch.zeros((250, 2, heads, block, 2), dtype=torch.bfloat16, device="cuda")
        hc.hc_kv4_append(k, v, torch.where(keep, slots, -1).cuda(), codes, scales)
        return torch.cat([codes.view(torch.int32), scales.view(torch.int32)], -1).transpose(2, 3).reshape(250, 2, block, -1)

    first, second = torch.ones(tokens, dtype=torch.bool), torch.ones(tokens, dtype=torch.bool)
    for a, b in pairs:
        first[b] = second[a] = False
    one, two = written(first), written(second)
    for _ in range(5):
        both = written(torch.ones(tokens, dtype=torch.bool))
        assert ((both == one) | (both == two)).all()
        same = torch.ones(250, block, dtype=torch.bool)
        for a, _ in pairs:
            same[slots[a] // block, slots[a] % block] = False
        assert torch.equal(both.transpose(1, 2)[same.cuda()], one.transpose(1, 2)[same.cuda()])
