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
