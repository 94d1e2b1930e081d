"""The operators of include/hc_serve.h at the edges of what their header allows: lengths next to
2^31, memory past 32 bits, the most tokens, tables far wider than their requests, and graphs that
take turns. Against the 64-bit oracle or exact expectations."""
import numpy as np
import pytest
import torch

import hyper_connection_residual_read_gb300 as hc

from oracle import serve_oracle as S
from oracle import window_oracle as W
from test_gpu_serve import Rotary, Shared, bits16, check_sample, cos_sin, f64, i32, run_sample, settings_of, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def context():
    hc.hc_read_init(0, 64, 1e-6)
    yield
    assert hc.hc_read_status() == hc.HC_OK


# ---------------------------------------------------------------------------
# attention behind a shared prefix
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("q_heads,new", [(8, 1), (4, 3), (1, 40)])
@pytest.mark.parametrize("where", ["prefix", "own"])
def test_shared_over_lengths_next_to_the_largest(where, q_heads, new):
    """2^31 - 1 tokens of a prefix, or of a request's own: all pages but the last are one block, and the
    last one's keys have logits that make up for their number; the slot behind the end is NaN. A
    lane sums up to 2^17 terms or tiles in fp32, 2^-8 relative at worst: so much of lse, and of
    values 4 apart twice that, and half an ulp of bf16 below 8."""
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
    far = torch.zeros((1, width), dtype=torch.int32, device="cuda")
    far[0, -1] = 1
    near = torch.full((1, 1), -1, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(q).cuda(), torch.zeros((new, q_heads), device="cuda")
    tables = dict(prefix_table=far, prefix_lens=i32([kv]), block_table=near, kv_lens=i32([0]))
    if where == "own":
        tables = dict(prefix_table=near, prefix_lens=i32([0]), block_table=far, kv_lens=i32([kv]))
    hc.hc_kv4_attention_shared(q.cuda(), torch.from_numpy(codes).cuda(), scales, cu_groups=i32([0, 1]), max_shared=new,
                               cu_lens=i32([0, new]), max_new=new, workspace=torch.empty(new * q_heads * (d + 2), device="cuda"),
                               out=out, lse=lse, **tables)
    assert hc.hc_read_status() == hc.HC_OK
    value = low[..., None] + step[..., None] * W.unpack(codes)              # [block][kv][1][token][d]
    x = np.einsum("nhd,btd->nhbt", q.double().numpy(), value[:, 0, 0]) / 8
    times = np.ones((new, 2, block))
    times[:, 0] = width - 1
    for i in range(new):                                # every row sees a whole prefix
        times[i, 1, 255 if where == "prefix" else 255 - new + i + 1:] = 0
    p = np.exp(x) * times[:, None]
    part = p[:, :, 1].sum(-1) / p.sum((-1, -2))
    assert 0.05 < part.min() and part.max() < 0.95, "the last page matters, and not alone"
    want = np.einsum("nhbt,btd->nhd", p, value[:, 1, 0]) / p.sum((-1, -2))[..., None]
    assert np.abs(lse.double().cpu().numpy() - np.log(p.sum((-1, -2)))).max() <= 2.0 ** -8
    assert np.abs(out.double().cpu().numpy() - want).max() <= 2 * 4 * 2.0 ** -8 + 2.0 ** -6


def widened(c, columns):
    """A table with room for far more than its requests hold."""
    return i32(np.concatenate([c.table, np.full((c.table.shape[0], columns), -1)], 1))


@pytest.mark.parametrize("columns", [0, 300, 5000])
@pytest.mark.parametrize("heads,new", [((8, 8, 64), 1), ((16, 4, 128), 2), ((8, 4, 128), 1), ((6, 2, 64), 4)], ids=str)
def test_shared_of_many_short_requests(heads, new, columns):
    """Requests taken as a whole by CTAs of few and of many warps, and cut in runs: the table's width
    chooses among them."""
    g = np.random.default_rng(1)
    own = [(int(g.integers(0, 90)) * (1 + 5 * (i % 7 == 0)), int(g.integers(0, new + 1))) for i in range(90)]
    c = Shared(2, [(130, own[:40]), (0, own[40:41]), (17, own[41:])], *heads, 16, "bf16")
    c.check(*c.run(block_table=widened(c, columns), max_new=new))


def test_shared_of_one_long_request_among_short_ones():
    own = [(3 + i % 5, 1) for i in range(60)] + [(9000, 1)]
    c = Shared(3, [(50, own)], 8, 4, 64, 16, "fp16")
    c.check(*c.run())


@pytest.mark.parametrize("groups", [31, 33, 3000])
def test_shared_of_many_groups(groups):
    g = np.random.default_rng(groups)
    c = Shared(4, [(int(g.integers(0, 40)), [(int(g.integers(0, 20)), int(g.integers(0, 3))) for _ in range(int(g.integers(0, 3)))])
                   for _ in range(groups)], 2, 1, 64, 16, "bf16")
    c.check(*c.run())


@pytest.mark.parametrize("prefix,new", [(4000, 30), (4000, 100), (777, 300)])
def test_shared_prefixes_in_pieces_and_whole(prefix, new):
    """Row tiles of a prefix that one CTA reads and that many do, in one call."""
    c = Shared(5, [(prefix, [(new, new)]), (0, [(40, 40)]), (33, [(20, 20), (9, 3)])], 4, 2, 64, 32, "bf16")
    c.check(*c.run())


def test_two_graphs_of_shared_attention_in_turns():
    """They share the context's scratch, and their workspaces are their own."""
    a = Shared(6, [(3000, [(30 + i, 2) for i in range(20)])], 8, 2, 128, 16, "bf16", mask=tree)
    b = Shared(7, [(900, [(10, 60)]), (70, [(300, 1)])], 4, 4, 64, 16, "fp16")
    runs = []
    for c in (a, b):
        want = c.run()
        kw = c.arguments()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            hc.hc_kv4_attention_shared(**kw)
        runs.append((graph, kw, want))
    for i in (0, 1, 1, 0, 1, 0, 0):
        graph, kw, want = runs[i]
        kw["out"].zero_()
        graph.replay()
        assert torch.equal(kw["out"], want[0]) and torch.equal(kw["lse"], want[1])


@pytest.mark.parametrize("heads,groups", [
    ((32, 8, 128), [(2001, [(30 + i, 1) for i in range(8)])]),
    ((32, 8, 128), [(2001, [(50 + 3 * i, 1) for i in range(40)])]),
    ((20, 4, 128), [(3000, [(100, 8)] * 4), (500, [(700, 8), (1, 3), (90, 8)])]),
    ((8, 2, 64), [(300, [(1000, 1), (5, 1)])]),
    ((4, 1, 64), [(9000, [(3000 + i, 1) for i in range(24)])]),
    ((4, 4, 64), [(700, [(60, 60), (0, 0), (200, 200)]), (0, [(90, 70)])]),
], ids=str)
def test_shared_directly_behind_the_write_of_what_it_reads(heads, groups):
    """Writes of all keys and values and calls that read them, one after the other without a pause, with one
    workspace: what each call returns is what it returns alone."""
    c = Shared(11, groups, *heads, 16, "bf16")
    kw = c.arguments()
    t, _, d = c.q.shape
    at = [(b, n) for b, n in enumerate(np.concatenate([c.kv, c.prefix]))]
    tables = np.concatenate([c.table, c.prefix_table])
    slots = torch.from_numpy(np.concatenate([tables[b, np.arange(n) // 16] * 16 + np.arange(n) % 16 for b, n in at])).cuda()
    g = torch.Generator(device="cuda").manual_seed(3)
    rows = [[torch.randn(len(slots), heads[1], d, generator=g, device="cuda").bfloat16() for _ in range(2)] for _ in range(2)]
    qs = [torch.randn(kw["q"].shape, generator=g, device="cuda").bfloat16() for _ in range(2)]
    outs = [torch.empty_like(kw["out"]) for _ in range(12)]
    lses = [torch.empty_like(kw["lse"]) for _ in range(12)]

    def step(i):
        hc.hc_kv4_append(*rows[i % 2], slots, kw["codes"], kw["scales"])
        hc.hc_kv4_attention_shared(**dict(kw, q=qs[i // 2 % 2], out=outs[i], lse=lses[i]))

    want = []
    for i in range(12):
        torch.cuda.synchronize()
        step(i)
        torch.cuda.synchronize()
        want.append((outs[i].clone(), lses[i].clone()))
    assert not torch.equal(want[0][0], want[1][0]) and torch.equal(want[0][0], want[4][0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(12):
            step(i)
    for run in (lambda: [step(i) for i in range(12)], graph.replay, graph.replay):
        for x in outs + lses:
            x.zero_()
        run()
        torch.cuda.synchronize()
        for i in range(12):
            assert torch.equal(outs[i], want[i][0]) and torch.equal(lses[i], want[i][1])


# ---------------------------------------------------------------------------
# rotary
# ---------------------------------------------------------------------------

def test_rotary_into_a_cache_beyond_32_bits():
    blocks, h, block, d = 70001, 8, 64, 128
    codes = torch.zeros((blocks, 2, h, block, d // 2), dtype=torch.uint8, device="cuda")
    assert codes.numel() > 1 << 32
    scales = torch.full((blocks, 2, h, block, 2), float("nan"), dtype=torch.bfloat16, device="cuda")
    c = Rotary(1, 150, 16, h, d, d, 1, False, True, "bf16", block=block)
    pages = np.array([blocks - 1, 3, blocks - 2])
    slots = pages[np.arange(150) // block] * block + np.arange(150) % block
    c.run(codes=codes, scales=scales, slots=torch.from_numpy(slots).cuda())
    q, k = c.want()
    assert torch.equal(c.out.cpu(), torch.from_numpy(q).bfloat16())
    for kv, x in enumerate((k, f64(c.v))):
        codes_of, s, m = W.round_group(np.asarray(x, dtype=np.float64))
        got = codes[torch.from_numpy(pages).cuda()].cpu().numpy()[:, kv].transpose(0, 2, 1, 3).reshape(-1, h, d // 2)[:150]
        assert np.array_equal(got, W.pack(codes_of))


def test_rotary_of_the_most_tokens():
    """2^31 - 1 tokens of one key and value (strides of 0), two of which have slots and positions."""
    n = 2 ** 31 - 1
    slots, at = torch.full((n,), -1, dtype=torch.int64, device="cuda"), torch.full((n,), -1, dtype=torch.int32, device="cuda")
    slots[7], slots[-1], at[7], at[-1] = 3, 17, 5, 9
    codes = torch.zeros((2, 2, 1, 16, 32), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((2, 2, 1, 16, 2), dtype=torch.bfloat16, device="cuda")
    x = torch.randn(64, generator=torch.Generator().manual_seed(1)).bfloat16()
    table = cos_sin(10, 64)
    one = x.cuda().expand(n, 1, 64)
    hc.hc_kv4_append_rotary(None, one, one, torch.from_numpy(table).cuda(), at, slots, codes, scales, None)
    want_codes, want_scales = np.zeros((2, 2, 1, 16, 32), dtype=np.uint8), np.zeros((2, 2, 1, 16, 2))
    for slot, p in ((3, 5), (17, 9)):
        k = S.norm_rotate(f64(x)[None, None], None, 0, table[p:p + 1, 0], table[p:p + 1, 1], False)[0, 0]
        for kv, y in enumerate((k, f64(x))):
            c, s, m = W.round_group(np.asarray(y, dtype=np.float64))
            want_codes[slot // 16, kv, 0, slot % 16] = W.pack(c)
            want_scales[slot // 16, kv, 0, slot % 16] = s, m
    assert np.array_equal(codes.cpu().numpy(), want_codes) and np.array_equal(f64(scales), want_scales)


def test_rotary_of_rows_far_apart():
    """Token strides that pass 32 bits."""
    stride = (1 << 30) + 8
    far = torch.zeros(2 * stride + 512, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    rows = far.as_strided((3, 4, 64), (stride, 64, 1))
    rows.copy_(x)
    table, at, slots = torch.from_numpy(cos_sin(9, 64)).cuda(), i32([2, 8, 0]), torch.tensor([5, 6, 30]).cuda()
    results = []
    for q, k, v in ((rows[:, :2], rows[:, 2:3], rows[:, 3:]), (x[:, :2], x[:, 2:3], x[:, 3:])):
        codes = torch.zeros((2, 2, 1, 16, 32), dtype=torch.uint8, device="cuda")
        scales, out = torch.zeros((2, 2, 1, 16, 2), dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
        hc.hc_kv4_append_rotary(q, k, v, table, at, slots, codes, scales, out, eps=0.0)
        results.append((codes, scales, out))
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("q_heads,kv_heads", [(200, 1), (3, 190), (65, 65)])
def test_rotary_of_many_heads(q_heads, kv_heads):
    c = Rotary(3, 5, q_heads, kv_heads, 64, 64, 1, True, True, "fp16")
    before = c.before()
    c.run()
    c.check(*before)


# ---------------------------------------------------------------------------
# sample
# ---------------------------------------------------------------------------

def test_sample_of_more_rows_than_a_launch_has():
    n = (1 << 27) + 5
    x = torch.tensor([[0.0, 1.0]]).cuda().expand(n, 2)
    u = torch.zeros(n, device="cuda")
    u[-3:] = 0.5
    tokens, lp = torch.full((n,), -7, dtype=torch.int32, device="cuda"), torch.zeros(n, device="cuda")
    hc.hc_sample_tokens(x, u, tokens, lp)
    assert int(tokens[:-3].max()) == 0 and int(tokens[:-3].min()) == 0 and tokens[-3:].tolist() == [1, 1, 1]
    assert float(lp.max()) < 0


def test_sample_of_rows_far_apart():
    stride = (1 << 31) + 3
    far = torch.zeros(stride + 6000, dtype=torch.bfloat16, device="cuda")
    rows = far.as_strided((2, 5000), (stride, 1))
    g = np.random.default_rng(1)
    rows.copy_(torch.from_numpy(g.standard_normal((2, 5000)) * 3).bfloat16())
    check_sample(rows, g.random(2), top_k=np.array([40, 0]), top_p=np.array([1.0, 0.9]))


@pytest.mark.parametrize("kind", ["flat", "ties", "two values", "long tail", "steep"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_sample_of_lists_of_every_length(kind, dtype):
    """Distributions whose filters leave few and nearly all of a row: lists that one CTA ends, that a
    cluster does, and that do not fit."""
    g = np.random.default_rng(4)
    rows, vocab = 12, 70001
    x = {"flat": lambda: 0.01 * g.standard_normal((rows, vocab)), "ties": lambda: np.round(g.standard_normal((rows, vocab)) * 2),
         "two values": lambda: np.where(g.random((rows, vocab)) < 0.4, 1.5, -1.0), "long tail": lambda: -8 * np.log1p(g.random((rows, vocab)) * 3000),
         "steep": lambda: 30 * g.standard_normal((rows, vocab))}[kind]()
    x = torch.from_numpy(x).to(dtype).cuda()
    for settings in (dict(top_p=np.linspace(0.05, 0.999, rows)), dict(top_k=np.geomspace(1, 69999, rows).astype(int)),
                     dict(top_k=np.geomspace(2, 69999, rows).astype(int), top_p=np.full(rows, 0.97)), dict(min_p=np.geomspace(1e-6, 1, rows)),
                     dict(top_k=np.full(rows, 257), top_p=np.full(rows, 0.6), min_p=np.full(rows, 0.2)), settings_of(g, rows)):
        check_sample(x, g.random(rows), **settings)


def test_sample_of_one_large_row_batch_is_that_of_its_rows():
    """Rows of a batch that fills the GPU, and each alone: the same tokens (clusters of other sizes)."""
    g = np.random.default_rng(6)
    x = torch.from_numpy(g.standard_normal((400, 30001)).astype(np.float32) * 3).cuda()
    u, settings = g.random(400), settings_of(g, 400)
    got, lp = run_sample(x, u, **settings)
    for t in range(0, 400, 40):
        one = run_sample(x[t:t + 1], u[t:t + 1], **{k: v[t:t + 1] for k, v in settings.items()})
        assert one[0][0] == got[t] and one[1][0] == lp[t]


@pytest.mark.parametrize("kind", ["deep", "blind", "top"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_sample_where_every_eighth_logit_misleads(kind, dtype):
    """Rows whose logits at the places 8 j + j % 8 are unlike the others: of little weight but much of it in
    eighths, none, or all of the largest. An estimate from them is wrong to either side."""
    vocab, rows = 65536, 12
    g = np.random.default_rng(5)
    at = np.arange(vocab)
    eighth = at % 8 == at // 8 % 8
    x = np.zeros((rows, vocab))
    if kind == "deep":                           # 1, 2.03 and 0.155 of weight
        x[:] = np.where(eighth, -10.875, -10.25)
        x[:, 8] = 0.0
    elif kind == "blind":
        x[:] = np.where(eighth, -np.inf, g.integers(-64, 64, (rows, vocab)) / 16)
    else:
        x[:] = np.where(eighth, 4.0, -4.0) + g.integers(-16, 16, (rows, vocab)) / 16
    x = torch.from_numpy(x).to(dtype).cuda()
    p = np.array([0.1, 0.3, 0.5, 0.7, 0.8, 0.8425, 0.85, 0.9, 0.95, 0.97, 0.99, 0.999])
    k = np.array([1, 100, 1000, 1025, 1500, 3000, 8191, 8192, 8193, 20000, 40000, 65535])
    check_sample(x, g.random(rows), top_p=p)
    check_sample(x, g.random(rows), top_k=k)
    check_sample(x, g.random(rows), top_k=k[::-1].copy(), top_p=p)
    check_sample(x, g.random(rows), top_p=p, temperature=np.full(rows, 0.5), min_p=np.full(rows, 1e-5))
