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
