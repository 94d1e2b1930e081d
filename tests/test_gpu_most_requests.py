"""Attention of 2^31 - 1 requests of which the last few have tokens: what the kernels share out among
their threads, and the extents of the index arrays, pass 31 bits in the sums on the way. Values
against the oracle, tolerances as in test_gpu_serve.py (Shared.check)."""
import numpy as np
import pytest
import torch

import hyper_connection_residual_read_gb300 as hc

from test_gpu_serve import Shared

pytestmark = pytest.mark.gpu

MOST = (1 << 31) - 1


@pytest.fixture(scope="module", autouse=True)
def context():
    hc.hc_read_init(0, 64, 1e-6)
    yield
    torch.cuda.empty_cache()
    assert hc.hc_read_status() == hc.HC_OK


@pytest.mark.parametrize("new", [2, 40], ids=["window", "chunk"])
def test_attention_of_the_most_requests(new):
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 26 GB for the requests' arrays")
    c = Shared(new, [(0, [(14, new), (9, 1), (0, 2)])], 4, 2, 64, 16, "bf16")
    c.kv = np.minimum(c.kv, 14)
    kw = c.arguments()
    n = len(c.kv)
    c.table = c.table[:, :1]
    table = torch.zeros((MOST, 1), dtype=torch.int32, device="cuda")
    table[-n:] = kw["block_table"][:, :1]
    kv = torch.zeros(MOST, dtype=torch.int32, device="cuda")
    kv[-n:] = torch.from_numpy(c.kv).int().cuda()
    cu = torch.zeros(MOST + 1, dtype=torch.int32, device="cuda")
    cu[-n:] = kw["cu_lens"][1:]
    hc.hc_kv4_attention(kw["q"], kw["codes"], kw["scales"], table, cu, kv, kw["max_new"], kw["out"], lse=kw["lse"])
    c.check(kw["out"], kw["lse"])
