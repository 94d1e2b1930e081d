"""The operators of include/hc_serve.h on the GPU against the oracle (oracle/serve_oracle.py), at
the sizes, masks, values and settings where they can go wrong.

Tolerances (derived, per element):

* rotary: codes, steps, minima and rotated queries equal: all steps are single fp32 operations.
  Against the formula in 64 bits: a norm's sum has at most 8 roundings of positive terms, its
  scale 4 more (2^-24 each), a rotated element the products and their sum: 16 * 2^-24 of |a c| +
  |b s| in all, and half a step of the output type.
* shared attention: as of hc_kv4_attention (tests/test_gpu_window.py), of the prefix's and the own
  part each, which the join weighs with p; the join itself is a few fp32 operations, 2^-21 of the
  terms.
* sample: the oracle's token, but where it calls the decision nearer than 2^-27 (weights are
  within 2^-29 and their sums exact); logprob within 2^-20 of 1 + its size.
"""
import numpy as np
import pytest
import torch

import hyper_connection_residual_read_gb300 as hc

from oracle import serve_oracle as S
from oracle import window_oracle as W
from oracle.hc_oracle import bf16_bits_to_f64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


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


def bf16_bits(a):
    return (a.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


# ---------------------------------------------------------------------------
# rotary
# ---------------------------------------------------------------------------

def cos_sin(length, dim):
    i = np.arange(dim // 2)
    angle = np.arange(length)[:, None] * 10000.0 ** (-2.0 * i / max(dim, 1))
    return np.stack([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


class Rotary:
    def __init__(self, seed, tokens, q_heads, kv_heads, dim, rot, axes, interleaved, norm, dtype, block=16, length=300,
                 size=1.0):
        g = np.random.default_rng(seed)
        self.g, self.dtype, self.block, self.interleaved = g, dtype, block, interleaved
        fused = g.standard_normal((tokens, (q_heads + 2 * kv_heads) * dim)) * size
        fused[:, q_heads * dim:(q_heads + kv_heads) * dim] += g.standard_normal(kv_heads * dim) * size
        fused = torch.from_numpy(fused).to(DT[dtype]).cuda()
        cut = lambda a, n: fused[:, a * dim:(a + n) * dim].view(tokens, n, dim)  # noqa: E731
        self.q = cut(0, q_heads) if q_heads else None
        self.k, self.v = cut(q_heads, kv_heads), cut(q_heads + kv_heads, kv_heads)
        weights = lambda: torch.from_numpy(1 + 0.2 * g.standard_normal(dim)).to(DT[dtype]).cuda()  # noqa: E731
        self.qn, self.kn = (weights(), weights()) if norm else (None, None)
        self.table = cos_sin(length, rot) if rot else None
        self.positions = g.integers(0, length, (axes, tokens))
        self.axis_of = g.integers(0, axes, rot // 2) if axes > 1 else None
        blocks = tokens // block + 3
        self.codes = torch.full((blocks, 2, kv_heads, block, dim // 2), 0xA5, dtype=torch.uint8, device="cuda")
        self.scales = torch.full((blocks, 2, kv_heads, block, 2), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.slots = g.permutation(blocks * block)[:tokens].astype(np.int64)
        self.out = None if self.q is None else torch.full((tokens, q_heads, dim), 9.0, dtype=DT[dtype], device="cuda")

    def run(self, eps=1e-6, stream=None, **other):
        kw = dict(q=self.q, k=self.k, v=self.v, cos_sin=None if self.table is None else torch.from_numpy(self.table).cuda(),
                  positions=None if self.table is None else i32(self.positions), slots=torch.from_numpy(self.slots).cuda(),
                  codes=self.codes, scales=self.scales, q_out=self.out, q_norm=self.qn, k_norm=self.kn, eps=eps,
                  axis_of=None if self.axis_of is None else i32(self.axis_of), interleaved=self.interleaved, stream=stream)
        hc.hc_kv4_append_rotary(**dict(kw, **other))

    def want(self, eps=1e-6, wide=False):
        t = self.k.shape[0]
        if self.table is None:
            c = s = np.zeros((t, 0), dtype=np.float32)
        else:
            pos = np.clip(self.positions, 0, len(self.table) - 1)
            c, s = S.table_rows(self.table, pos, self.axis_of)
        n = lambda w: None if w is None else f64(w)  # noqa: E731
        return [None if x is None else S.norm_rotate(f64(x), n(w), eps, c, s, self.interleaved, wide)
                for x, w in ((self.q, self.qn), (self.k, self.kn))]

    def check(self, codes, scales, eps=1e-6, skip=()):
        """Against the cache as it was before, `codes` and `scales` (bits)."""
        q, k = self.want(eps)
        t = self.k.shape[0]
        there = np.ones(t, dtype=bool)
        there[list(skip)] = False
        if q is not None:
            want = torch.from_numpy(q).to(DT[self.dtype]).cpu()
            want[~there] = 9.0
            assert torch.equal(torch.nan_to_num(self.out.cpu().float(), 77.0), torch.nan_to_num(want.float(), 77.0))
        put = np.where(there, self.slots, -1)
        keep = put >= 0
        wc, ws = codes.copy(), scales.copy()
        for kv, x in enumerate((k, f64(self.v))):
            c, s, m = W.round_group(np.asarray(x, dtype=np.float64))
            wc[put[keep] // self.block, kv, :, put[keep] % self.block] = W.pack(c[keep])
            as_bits = np.stack([bf16_bits(s[keep]), bf16_bits(m[keep])], -1)
            as_bits[np.isnan(s[keep])] = 0x7FC0
            ws[put[keep] // self.block, kv, :, put[keep] % self.block] = as_bits
        assert np.array_equal(self.codes.cpu().numpy(), wc)
        assert np.array_equal(bits16(self.scales), ws)

    def before(self):
        return self.codes.cpu().numpy(), bits16(self.scales)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("tokens,q_heads,kv_heads,dim,rot,axes,interleaved,norm", [
    (1, 1, 1, 64, 64, 1, False, True), (1, 20, 4, 128, 128, 1, False, True), (5, 0, 3, 128, 128, 1, True, True),
    (17, 7, 1, 128, 96, 3, False, False), (33, 4, 2, 64, 32, 3, True, True), (40, 32, 8, 64, 48, 4, False, True),
    (200, 5, 5, 128, 16, 2, True, False), (3, 2, 2, 64, 0, 1, False, True), (300, 8, 2, 128, 64, 1, False, True),
    (1025, 3, 1, 64, 64, 1, True, False)])
def test_rotary(dtype, tokens, q_heads, kv_heads, dim, rot, axes, interleaved, norm):
    c = Rotary(tokens + dim, tokens, q_heads, kv_heads, dim, rot, axes, interleaved, norm, dtype)
    if tokens > 20:
        c.slots[[2, 7]] = [-1, -100]
    before = c.before()
    c.run()
    c.check(*before)
    # against the formula in 64 bits
    if q_heads:
        q = c.want(wide=True)[0]
        terms = np.abs(c.want(wide=True)[0])
        if rot:
            cs = S.table_rows(c.table, np.clip(c.positions, 0, len(c.table) - 1), c.axis_of)
            plain = S.norm_rotate(f64(c.q), None if c.qn is None else f64(c.qn), 1e-6, np.ones_like(cs[0]), np.zeros_like(cs[1]),
                                  interleaved, True)
            terms = S.norm_rotate(np.abs(plain), None, 0, np.abs(cs[0]), np.abs(cs[1]), interleaved, True)
            terms = np.maximum(terms, S.norm_rotate(np.abs(plain), None, 0, np.abs(cs[0]), -np.abs(cs[1]), interleaved, True))
        off = np.abs(f64(c.out) - q)
        assert (off <= HALF[dtype] * np.abs(q) + 2.0 ** -20 * terms + (2.0 ** -25 if dtype == "fp16" else 0)).all()


def test_rotary_is_the_plain_write_where_nothing_turns():
    """Without a norm and at position 0 the cache holds what hc_kv4_append writes, and the queries
    stay as they are."""
    c = Rotary(1, 50, 4, 2, 128, 128, 1, False, False, "bf16")
    c.positions[:] = 0
    c.run()
    codes, scales = torch.full_like(c.codes, 0xA5), torch.full_like(c.scales, float("nan"))
    hc.hc_kv4_append(c.k, c.v, torch.from_numpy(c.slots).cuda(), codes, scales)
    assert torch.equal(codes, c.codes) and np.array_equal(bits16(scales), bits16(c.scales))
    assert torch.equal(c.out, c.q)


def test_rotary_tokens_that_are_none():
    """A negative position on any axis: the row of q_out and the slot stay as they were."""
    c = Rotary(2, 60, 4, 2, 64, 64, 3, True, True, "bf16")
    c.positions[0, 5], c.positions[2, [9, 59]] = -1, -(1 << 31)
    before = c.before()
    c.run()
    c.check(*before, skip=(5, 9, 59))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_entries_outside_are_reported(interleaved):
    c = Rotary(3, 40, 4, 2, 128, 64, 2, interleaved, True, "fp16")
    c.positions[1, 7] = len(c.table)
    c.positions[0, 8] = (1 << 31) - 1
    before = c.before()
    c.run()
    assert hc.hc_read_status() == hc.HC_ERR_BOUNDS
    c.check(*before)                                     # they count as the last position
    axis = c.axis_of.copy()
    c.axis_of[3], c.axis_of[4] = 2, -1
    c.positions = np.clip(c.positions, 0, 10)
    c.run()
    assert hc.hc_read_status() == hc.HC_ERR_BOUNDS
    axis[[3, 4]] = 0
    c.axis_of = axis
    c.check(*before)
    c.slots[4] = 1 << 40
    c.run()
    assert hc.hc_read_status() == hc.HC_ERR_BOUNDS and hc.hc_read_status() == hc.HC_OK


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rotary_of_difficult_values(dtype):
    """Zeros, tiny and large values, NaN and infinities, with and without a norm."""
    for norm in (False, True):
        c = Rotary(4, 12, 2, 2, 64, 64, 1, False, norm, dtype)
        for x in (c.q, c.k, c.v):
            x[0] = 0
            x[1] *= 1e-25
            x[2] *= 1e15
            x[3, 0, 5] = float("nan")
            x[4, 1, 63] = float("inf")
            x[5, 0, 0] = float("-inf")
            x[6] = -2.5
        before = c.before()
        c.run()
        c.check(*before)


def test_rotary_of_several_sizes_of_eps():
    for eps in (0.0, 1e-5, 0.25):
        c = Rotary(5, 9, 2, 1, 128, 128, 1, False, True, "bf16", size=1e-2)
        before = c.before()
        c.run(eps)
        c.check(*before, eps=eps)


def test_rotary_strides_streams_and_graphs():
    c = Rotary(6, 77, 8, 2, 128, 128, 1, False, True, "bf16")
    before = c.before()
    c.run()
    c.check(*before)
    base = c.out.clone(), c.codes.clone()
    outer = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    side = torch.cuda.Stream()
    for stream in (None, side):
        c.out.fill_(9)
        c.codes.fill_(0xA5)
        args = dict(q=outer(c.q), k=outer(c.k), v=outer(c.v))
        torch.cuda.synchronize()
        c.run(stream=stream, **args)
        torch.cuda.synchronize()
        assert torch.equal(c.out, base[0]) and torch.equal(c.codes, base[1])
    table, pos, slots = torch.from_numpy(c.table).cuda(), i32(c.positions[0]), torch.from_numpy(c.slots).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hc.hc_kv4_append_rotary(c.q, c.k, c.v, table, pos, slots, c.codes, c.scales, c.out, c.qn, c.kn)
    pos.add_(1).remainder_(len(c.table))
    c.positions = pos.cpu().numpy()[None]
    graph.replay()
    c.check(*before)


# ---------------------------------------------------------------------------
# attention behind a shared prefix
# ---------------------------------------------------------------------------

class Shared:
    """`groups`: a prefix length and its requests' (own tokens, new tokens). Unused slots hold NaN
    and infinities."""

    def __init__(self, seed, groups, q_heads, kv_heads, dim, block, dtype, mask=None, offset=0.0, spread=0.3, q_size=1.0):
        g = np.random.default_rng(seed)
        self.block, self.dtype = block, dtype
        self.prefix = np.array([p for p, _ in groups])
        lens = [x for _, rs in groups for x in rs]
        self.cu_groups = np.concatenate([[0], np.cumsum([len(rs) for _, rs in groups])])
        self.kv, new = np.array([x for x, _ in lens]), np.array([y for _, y in lens])
        self.cu = np.concatenate([[0], np.cumsum(new)])
        lengths = np.concatenate([self.kv, self.prefix])
        have = -(-lengths // block)
        total = int(have.sum()) + 2
        order = g.permutation(total)
        tables = np.full((len(lengths), max(1, int(have.max())) + 1), -1)
        used, at = np.zeros((total, block), dtype=bool), 0
        for b, n in enumerate(have):
            tables[b, :n] = order[at:at + n]
            at += n
            for p in range(n):
                used[tables[b, p], : min(block, lengths[b] - p * block)] = True
        self.table, self.prefix_table = tables[:len(lens)], tables[len(lens):]
        self.codes = g.integers(0, 256, (total, 2, kv_heads, block, dim // 2)).astype(np.uint8)
        step = 0.25 * np.exp(spread * g.standard_normal((total, 2, kv_heads, block)))
        low = -7.5 * step + 0.2 * g.standard_normal(step.shape) + offset
        poison = np.where(g.random(used.shape) < 0.5, np.nan, np.inf)
        sm = np.where(used[:, None, None, :, None], np.stack([step, low], -1), poison[:, None, None, :, None])
        self.scales = torch.from_numpy(sm).bfloat16()
        tokens = int(new.sum())
        self.q = torch.from_numpy(g.standard_normal((tokens, q_heads, dim)) * q_size).to(DT[dtype])
        self.max_new = max(1, int(new.max()))
        self.max_shared = max(1, int(np.diff(self.cu[self.cu_groups]).max()))
        self.mask = None
        if mask is not None:
            self.mask = np.array([mask(int(i), int(m), g) for m in new for i in range(m)], dtype=np.uint64)

    def arguments(self, **other):
        q = self.q.cuda()
        t, h, d = q.shape
        mask = None if self.mask is None else torch.from_numpy(self.mask.view(np.int64)).cuda()
        kw = dict(q=q, codes=torch.from_numpy(self.codes).cuda(), scales=self.scales.cuda(), prefix_table=i32(self.prefix_table),
                  prefix_lens=i32(self.prefix), cu_groups=i32(self.cu_groups), max_shared=self.max_shared,
                  block_table=i32(self.table), cu_lens=i32(self.cu), kv_lens=i32(self.kv), max_new=self.max_new,
                  workspace=torch.full((t * h * (d + 2),), float("nan"), device="cuda"),
                  out=torch.full(q.shape, 55.0, dtype=q.dtype, device="cuda"), lse=torch.full((t, h), 55.0, device="cuda"), mask=mask)
        return dict(kw, **other)

    def run(self, **other):
        kw = self.arguments(**other)
        hc.hc_kv4_attention_shared(**kw)
        return kw["out"], kw["lse"]

    def check(self, out, lse, scale=None):
        d = self.q.shape[2]
        scale = 1 / np.sqrt(d) if scale is None else scale
        q, bits = f64(self.q), bits16(self.scales)
        want, wl, size = S.attention_shared(q, self.codes, bits, self.prefix_table, self.prefix, self.cu_groups, self.table,
                                            self.cu, self.kv, self.mask, scale)
        got, gl = f64(out), f64(lse)
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isneginf(gl), np.isneginf(wl))
        sm = bf16_bits_to_f64(bits)
        fine = np.where(np.isfinite(sm), sm, 0)
        step, base = np.abs(fine[..., 0]), np.abs(fine[..., 1] + 8 * fine[..., 0])
        keys = max(self.kv) + max(self.prefix)
        tol = HALF[self.dtype] * np.abs(want) + (2.0 ** -10 + 2.0 ** -21) * size + 2.0 ** -24 * 8 * step.max() * keys + 1e-7
        ok = np.isnan(want) | (np.abs(got - want) <= tol)
        assert ok.all(), (np.argwhere(~ok)[:5], got[~ok][:5], want[~ok][:5], tol[~ok][:5])
        terms = abs(scale) * np.abs(q).sum(-1) * (8 * step[:, 0].max() + base[:, 0].max())
        fin = np.isfinite(wl)
        assert (np.abs(gl - wl)[fin] <= (2.0 ** -19 * (1 + terms))[fin]).all()


def tree(i, n, g):
    return int(g.integers(0, 1 << n)) | (1 << i)


def holes(i, n, g):
    return 0 if i % 3 == 0 else int(g.integers(0, 1 << n))


SHARED_HEADS = [(8, 8, 64), (8, 2, 128), (20, 4, 128), (7, 1, 64)]
GROUPS = {
    "one request": [(40, [(1, 1)])],
    "single tokens": [(300, [(1, 1), (2, 1), (17, 1), (0, 1), (300, 1), (129, 1)])],
    "empty prefix": [(0, [(5, 1), (40, 3)]), (33, [(7, 2)])],
    "nothing of its own": [(200, [(0, 1), (0, 2), (0, 5)])],
    "windows": [(129, [(8, 8), (5, 8), (0, 3), (64, 1)]), (17, [(65, 5), (70, 0), (130, 7)]), (512, [(513, 8)])],
    "groups without tokens": [(50, []), (60, [(9, 0)]), (70, [(20, 4)]), (80, [])],
    "many groups": [(16 * (i % 5) + i, [(i, 1)] * (i % 3 + 1)) for i in range(1, 50)],
}


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", SHARED_HEADS, ids=str)
@pytest.mark.parametrize("groups", list(GROUPS))
def test_shared(heads, dtype, groups):
    c = Shared(1, GROUPS[groups], *heads, 16, dtype)
    c.check(*c.run())


@pytest.mark.parametrize("mask", [tree, holes])
@pytest.mark.parametrize("heads", SHARED_HEADS, ids=str)
def test_shared_with_masks(heads, mask):
    c = Shared(2, GROUPS["windows"] + GROUPS["empty prefix"], *heads, 32, "bf16", mask=mask)
    c.check(*c.run())


@pytest.mark.parametrize("heads", [(8, 2, 128), (14, 2, 64), (5, 1, 128)], ids=str)
@pytest.mark.parametrize("groups", [[(100, [(33, 33)])], [(500, [(64, 64), (100, 40), (40, 100)]), (77, [(0, 0), (300, 1)])],
                                    [(3001, [(257, 200), (640, 9)])], [(0, [(100, 60)])]], ids=str)
def test_shared_of_chunks(heads, groups):
    c = Shared(3, groups, *heads, 64, "bf16")
    c.check(*c.run())


@pytest.mark.parametrize("prefix", [4096, 20011])
@pytest.mark.parametrize("requests", [1, 3, 40])
def test_shared_of_long_prefixes(prefix, requests):
    """A prefix split over many blocks of the launch, read by few and by many rows."""
    c = Shared(4, [(prefix, [(5 * i, 1) for i in range(requests)]), (7, [(3, 1)])], 8, 2, 128, 64, "bf16")
    c.check(*c.run())


def test_shared_by_more_tokens_than_a_row_tile():
    c = Shared(5, [(700, [(1 + i % 40, 1 + i % 3) for i in range(150)])], 8, 4, 64, 16, "fp16")
    c.check(*c.run())


@pytest.mark.parametrize("requests", [2, 30])
@pytest.mark.parametrize("kind", ["large q", "small q", "offset", "spread", "zero scale", "negative scale"])
def test_shared_values(kind, requests):
    kw = {"large q": dict(q_size=20.0), "small q": dict(q_size=1e-3), "offset": dict(offset=6.0),
          "spread": dict(spread=2.5)}.get(kind, {})
    scale = {"zero scale": 0.0, "negative scale": -0.05}.get(kind)
    c = Shared(6, [(300, [(50 + i, 1) for i in range(requests)])], 8, 2, 64, 16, "bf16", **kw)
    c.check(*c.run(scale=scale), scale)


def test_shared_sees_nan_only_where_it_looks():
    """A prefix's key or value held as NaN makes every row of its group NaN, and no other's; a
    request's own one that request's."""
    c = Shared(7, [(200, [(20, 2), (30, 1)]), (100, [(40, 3)]), (90, [(50, 1), (60, 1)])], 4, 2, 64, 16, "bf16")
    page = c.prefix_table[1][3]
    c.scales[page, 0, 0, 5] = float("nan")
    c.scales[page, 1, 1, 6] = float("nan")
    c.scales[c.table[4][2], 1, :, 1] = float("nan")
    out, lse = c.run()
    rows, some = out.float().isnan().all(-1).cpu().numpy(), out.float().isnan().any(-1).cpu().numpy()
    want = np.zeros_like(rows)
    want[c.cu[2]:c.cu[3]] = True
    want[c.cu[4]:c.cu[5]] = True
    assert np.array_equal(rows, some) and np.array_equal(rows, want)


def test_shared_is_attention_where_no_prefix_is():
    """An empty prefix: the own part alone, as hc_kv4_attention computes it (not bit for bit: its sums
    may be cut in other places)."""
    c = Shared(8, [(0, [(300, 4), (77, 2)])], 8, 2, 128, 16, "bf16")
    out, lse = c.run()
    kw = c.arguments()
    o, l = torch.empty_like(out), torch.empty_like(lse)
    hc.hc_kv4_attention(kw["q"], kw["codes"], kw["scales"], kw["block_table"], kw["cu_lens"], kw["kv_lens"], kw["max_new"], o, lse=l)
    c.check(out, lse)
    c.check(o, l)


def test_shared_strides_streams_graphs_and_repeats():
    c = Shared(9, [(1300, [(30, 5), (77, 3)]), (64, [(12, 1)])], 8, 2, 128, 16, "bf16")
    base = c.run()
    c.check(*base)
    t, h, d = c.q.shape
    fused = torch.full((t, 3 * h * d), 7.0, dtype=c.q.dtype, device="cuda")
    fused[:, h * d:2 * h * d] = c.q.cuda().reshape(t, -1)
    side = torch.cuda.Stream()
    for stream in (None, side):
        kw = c.arguments(q=fused[:, h * d:2 * h * d].view(t, h, d), stream=stream)
        torch.cuda.synchronize()
        hc.hc_kv4_attention_shared(**kw)
        torch.cuda.synchronize()
        assert torch.equal(kw["out"], base[0]) and torch.equal(kw["lse"], base[1])
    kw = c.arguments()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hc.hc_kv4_attention_shared(**kw)
    for _ in range(3):
        kw["out"].zero_()
        kw["workspace"].fill_(float("nan"))
        graph.replay()
        assert torch.equal(kw["out"], base[0]) and torch.equal(kw["lse"], base[1])
    # other lengths in the same graph
    c.prefix, c.kv = np.array([900, 30]), np.array([25, 70, 3])
    kw["prefix_lens"].copy_(i32(c.prefix))
    kw["kv_lens"].copy_(i32(c.kv))
    graph.replay()
    c.check(kw["out"], kw["lse"])


def test_shared_of_bad_entries_is_reported():
    make = lambda: Shared(10, [(100, [(20, 2)]), (90, [(30, 2)])], 4, 2, 64, 16, "bf16")  # noqa: E731
    base = make().run()[0]
    c = make()
    c.prefix_table[0, 3] = 1 << 20
    out = c.run()[0]
    assert hc.hc_read_status() == hc.HC_ERR_BOUNDS and torch.equal(out[2:], base[2:])
    c = make()
    c.prefix[1] = 100000                                  # longer than its row of the table
    c.run()
    assert hc.hc_read_status() == hc.HC_ERR_BOUNDS
    for bad in ([0, 3, 2], [0, -1, 2], [0, 1, 1 << 30], [1, 0, 2]):
        c = make()
        c.cu_groups = np.array(bad)
        c.run()
        assert hc.hc_read_status() == hc.HC_ERR_BOUNDS, bad
    c = make()
    c.run(max_shared=1)
    assert hc.hc_read_status() == hc.HC_ERR_BOUNDS and hc.hc_read_status() == hc.HC_OK


# ---------------------------------------------------------------------------
# sample
# ---------------------------------------------------------------------------

def run_sample(x, u, stream=None, **settings):
    t = x.shape[0]
    tokens, logprobs = torch.full((t,), -77, dtype=torch.int32, device="cuda"), torch.full((t,), 77.0, device="cuda")
    to = lambda k, v: None if v is None else i32(v) if k == "top_k" else torch.as_tensor(np.asarray(v), dtype=torch.float32).cuda()  # noqa: E731
    hc.hc_sample_tokens(x, to("u", u), tokens, logprobs, **{k: to(k, v) for k, v in settings.items()}, stream=stream)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), logprobs.cpu().numpy()


def check_sample(x, u, stream=None, near=2.0 ** -27, **settings):
    got, lp = run_sample(x, u, stream, **settings)
    x64, skipped = f64(x), 0
    for t in range(x.shape[0]):
        each = {k: float(np.float32(v[t])) if k != "top_k" else int(v[t]) for k, v in settings.items() if v is not None}
        token, want, close = S.sample(x64[t], float(np.float32(u[t])), **each)
        if close < near:
            skipped += 1
            continue
        assert got[t] == token, (t, got[t], token, u[t], each, close)
        assert np.isnan(lp[t]) == np.isnan(want) and (np.isnan(want) or abs(lp[t] - want) <= 2.0 ** -20 * (1 + abs(want))), (t, lp[t], want)
    assert skipped <= 1 + x.shape[0] // 100
    return got


def settings_of(g, rows):
    return dict(temperature=g.choice([0.0, 0.3, 0.7, 1.0, 1.5, 4.0], rows), top_k=g.choice([0, 1, 2, 5, 40, 300, 100000], rows),
                top_p=g.choice([0.0, 0.1, 0.5, 0.9, 0.99, 1.0], rows), min_p=g.choice([0.0, 0.0, 0.02, 0.3, 1.0], rows))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (5, 7), (40, 33), (64, 1000), (3, 4099), (30, 32000), (9, 50257),
                                        (7, 131072), (2, 200003), (2, 262144), (400, 513)])
def test_sample(dtype, rows, vocab):
    g = np.random.default_rng(rows + vocab)
    x = torch.from_numpy(g.standard_normal((rows, vocab)) * 3).to(DT[dtype]).cuda()
    check_sample(x, g.random(rows), **settings_of(g, rows))
    check_sample(x, g.random(rows))
    for name, value in settings_of(g, rows).items():
        check_sample(x, g.random(rows), **{name: value})


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab", [8, 1003, 70001])
def test_sample_of_difficult_rows(dtype, vocab):
    """All equal; one finite; -inf but for a few; a huge peak; very negative; the type's lowest
    value; ascending and descending; both zeros; few values that repeat."""
    x = torch.zeros(12, vocab, dtype=torch.float64)
    x[1] = float("-inf")
    x[1, vocab - 1] = -4.5
    x[2] = float("-inf")
    x[2, ::5] = torch.arange(len(x[2, ::5]), dtype=torch.float64) * -0.25
    x[3, vocab // 2] = 1e30
    x[4] = -1e30
    low = torch.finfo(DT[dtype]).min
    x[5] = low
    x[5, 1] = 3.0
    x[6] = low
    x[7] = torch.arange(vocab, dtype=torch.float64) * 1e-3
    x[8] = -x[7]
    x[9, 1::2] = -0.0
    x[10] = torch.arange(vocab, dtype=torch.float64) % 3
    x[11] = -(torch.arange(vocab, dtype=torch.float64) % 7) * 4
    x = x.to(DT[dtype]).cuda()
    g = np.random.default_rng(vocab)
    for n in range(6):
        check_sample(x, g.random(12), near=2.0 ** -26, **settings_of(g, 12))
    check_sample(x, g.random(12), near=2.0 ** -26)


def test_sample_at_the_ends_of_uniform():
    g = np.random.default_rng(1)
    x = torch.from_numpy(g.standard_normal((8, 3001))).cuda().float()
    u = np.array([0.0, -1.0, 1 - 2.0 ** -24, 1.0, 5.0, 2.0 ** -149, 0.5, np.inf], dtype=np.float32)
    got, _ = run_sample(x, u, top_k=np.full(8, 7))
    seven = np.sort(np.argsort(-f64(x), kind="stable")[:, :7])
    assert got.tolist() == [int(seven[t][i]) if i is not None else int(got[t]) for t, i in enumerate([0, 0, 6, 6, 6, 0, None, 6])]


def test_sample_rows_that_are_none():
    """NaN, +inf, -inf alone; settings that are NaN or an infinite temperature."""
    x = torch.randn(9, 5000, device="cuda")
    x[1, 1234], x[2, 4999], x[3] = float("nan"), float("inf"), float("-inf")
    s = dict(temperature=np.ones(9), top_p=np.full(9, 0.9), min_p=np.zeros(9), top_k=np.zeros(9, dtype=int))
    s["temperature"][4], s["temperature"][5], s["top_p"][6], s["min_p"][7] = np.nan, np.inf, np.nan, np.nan
    u = np.full(9, 0.5)
    u[8] = np.nan
    got, lp = run_sample(x, u, **s)
    assert (got[1:] == -1).all() and np.isnan(lp[1:]).all() and got[0] >= 0 and np.isfinite(lp[0])


def test_sample_of_small_and_large_temperatures():
    g = np.random.default_rng(2)
    x = torch.from_numpy(g.standard_normal((10, 2000)) * 4).cuda().float()
    t = np.array([1e-30, 1e-19, 1e-10, 1e-3, 0.05, 50.0, 1e4, 1e20, 3e38, -1.0], dtype=np.float32)
    got = check_sample(x, g.random(10), temperature=t)
    assert got[[0, 9]].tolist() == x[[0, 9]].argmax(-1).tolist()


def test_sample_strides_ties_streams_and_graphs():
    g = np.random.default_rng(5)
    wide = torch.from_numpy(np.round(g.standard_normal((6, 3001)) * 2)).bfloat16().cuda()     # many ties
    for lo in range(4):
        check_sample(wide[:, lo:lo + 900 + lo], g.random(6), **settings_of(g, 6))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    check_sample(wide[::2], g.random(3), stream=side, **settings_of(g, 3))
    one = torch.from_numpy(g.standard_normal((1, 700))).bfloat16().cuda().expand(4, 700)       # row stride 0
    check_sample(one, g.random(4), **settings_of(g, 4))
    u = torch.from_numpy(g.random(6)).float().cuda()
    tokens, lp = torch.zeros(6, dtype=torch.int32, device="cuda"), torch.zeros(6, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hc.hc_sample_tokens(wide[:, :900], u, tokens, lp)
    for _ in range(2):
        u.copy_(torch.from_numpy(g.random(6)).float())
        graph.replay()
        want, wl = run_sample(wide[:, :900], u.cpu().numpy())
        assert tokens.tolist() == want.tolist() and lp.tolist() == wl.tolist()


def test_sample_draws_by_the_weights():
    """65536 evenly spread numbers: each token as often as its probability, to one."""
    x = torch.tensor([[0.3, -1.0, 2.0, -float("inf"), 1.1, 0.0]]).cuda().expand(65536, 6)
    u = (np.arange(65536) + 0.5) / 65536
    got, _ = run_sample(x, u, top_p=np.full(65536, 0.97), temperature=np.full(65536, 0.8))
    w = np.exp((np.array([0.3, -1.0, 2.0, -np.inf, 1.1, 0.0]) - 2) / np.float64(np.float32(0.8)))
    order = np.argsort(-w)
    before = np.cumsum(w[order]) - w[order]
    w[order[before >= 0.97 * w.sum()]] = 0
    assert (np.abs(np.bincount(got, minlength=6) - 65536 * w / w.sum()) <= 1).all()


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def refuses(f, *args, **kw):
    with pytest.raises(hc.HcReadError) as e:
        f(*args, **kw)
    assert e.value.code == hc.HC_ERR_ARG


def test_refusals_of_rotary():
    c = Rotary(20, 8, 4, 2, 64, 32, 2, False, True, "bf16")
    c.run()
    table, pos = torch.from_numpy(c.table).cuda(), i32(c.positions)
    odd = torch.zeros(8, 2 * 64 + 4, device="cuda", dtype=torch.bfloat16)
    for bad in (dict(q=None), dict(q_out=None), dict(q_out=c.q), dict(q=c.q.float()), dict(v=c.v.half()),
                dict(k=c.k[:, :1]), dict(cos_sin=None), dict(positions=None), dict(cos_sin=table[:, :, :12].contiguous()),
                dict(cos_sin=table.half()), dict(cos_sin=table[:0]), dict(positions=pos[:, :5]), dict(positions=pos.long()),
                dict(positions=pos.repeat(3, 1)), dict(axis_of=i32(c.axis_of)[:7]), dict(q_norm=c.qn[:32]),
                dict(q_norm=c.qn.float()), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(slots=torch.zeros(8, dtype=torch.int32, device="cuda")), dict(k=odd[:, :128].view(8, 2, 64)),
                dict(q_out=c.codes.flatten()[:8 * 4 * 64 * 2].view(torch.bfloat16).view(8, 4, 64)),
                dict(cos_sin=torch.zeros(4, 2, 40, device="cuda"), axis_of=None), dict(cos_sin=table.cpu()), dict(positions=pos.cpu())):
        refuses(c.run, **bad)
    c.run(q=None, q_out=None)
    c.run(cos_sin=None, positions=None, axis_of=None)


def test_refusals_of_shared():
    c = Shared(21, [(40, [(20, 2), (9, 1)])], 4, 2, 64, 16, "bf16")
    ok = c.arguments()
    hc.hc_kv4_attention_shared(**ok)
    q, work = ok["q"], ok["workspace"]
    many = torch.zeros(1, 2 * 129, 64, dtype=torch.bfloat16, device="cuda")
    mask = torch.ones(3, dtype=torch.int64, device="cuda")
    for bad in (dict(max_shared=0), dict(max_shared=-1), dict(max_new=-1), dict(workspace=work[:-1]), dict(workspace=work.half()),
                dict(workspace=work.cpu()), dict(workspace=ok["out"].flatten().view(torch.float32)), dict(scale=float("nan")),
                dict(out=q), dict(q=q.float(), out=ok["out"].float()), dict(cu_groups=ok["cu_groups"][:1]),
                dict(prefix_lens=ok["prefix_lens"].long()), dict(prefix_table=ok["prefix_table"][0]),
                dict(prefix_table=ok["prefix_table"].cpu()), dict(mask=mask, max_new=65), dict(mask=mask[:1]),
                dict(lse=ok["lse"][:1]), dict(q=many, out=torch.zeros_like(many), lse=None),
                dict(prefix_lens=ok["prefix_lens"][:0], cu_groups=ok["cu_groups"][:1], prefix_table=ok["prefix_table"][:0])):
        refuses(hc.hc_kv4_attention_shared, **dict(ok, **bad))
    hc.hc_kv4_attention_shared(**dict(ok, max_new=0, max_shared=0))                     # nothing to do


def test_refusals_of_sample():
    x = torch.zeros(2, 40, device="cuda")
    f, ids = torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    out = torch.zeros(2, device="cuda")
    hc.hc_sample_tokens(x, f, ids, out)
    for args, kw in (((x.double(), f, ids, out), {}), ((x, f[:1], ids, out), {}), ((x, f, ids.long(), out), {}),
                     ((x, f, ids, f), {}), ((x, f, ids, out), dict(temperature=out)), ((x, f, ids, out), dict(top_k=f)),
                     ((x, f, ids, out), dict(top_p=f[:1])), ((x, f, ids, out), dict(min_p=f.cpu())),
                     ((x.t().contiguous().t(), f, ids, out), {}), ((x[:, :0], f, ids, out), {}),
                     ((torch.zeros(2, hc.HC_SAMPLE_MAX_VOCAB + 1, device="cuda"), f, ids, out), {})):
        refuses(hc.hc_sample_tokens, *args, **kw)


def test_calls_of_nothing():
    e = torch.empty(0, device="cuda")
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    hc.hc_sample_tokens(torch.empty(0, 5, device="cuda"), e, i, e)
    codes = torch.zeros(1, 2, 1, 16, 32, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(1, 2, 1, 16, 2, dtype=torch.bfloat16, device="cuda")
    k = torch.empty(0, 1, 64, device="cuda")
    hc.hc_kv4_append_rotary(k, k, k, torch.zeros(4, 2, 16, device="cuda"), i, i.long(), codes, scales, k.clone())
    q = k.bfloat16()
    hc.hc_kv4_attention_shared(q, codes, scales, i.view(0, 3), i, i32([0]), 1, i.view(0, 3), i32([0]), i, 1, e, q.clone())
