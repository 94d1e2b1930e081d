"""hc_kv4_attention_shared of very many groups, and of more 8-row shares than a launch has CTAs: with
the oracle's values, and each as a call of the groups that have tokens gives them.

Tolerances as in test_gpu_serve.py (Shared.check). Two calls over the same lengths cut a prefix in
different places and are not equal bit by bit.
"""
import numpy as np
import pytest
import torch

import hyper_connection_residual_read_gb300 as hc

from test_gpu_serve import Shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def context():
    hc.hc_read_init(0, 64, 1e-6)
    yield
    assert hc.hc_read_status() == hc.HC_OK


def among(c, groups, at):
    """The arguments of `c` with its groups from number `at` on, and groups without requests around."""
    kw = c.arguments()
    table = torch.full((groups, kw["prefix_table"].shape[1]), -1, dtype=torch.int32, device="cuda")
    lens = torch.full((groups,), 7, dtype=torch.int32, device="cuda")
    cu = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    n = len(c.prefix)
    table[at:at + n], lens[at:at + n] = kw["prefix_table"], kw["prefix_lens"]
    cu[at:at + n + 1], cu[at + n + 1:] = kw["cu_groups"], int(c.cu_groups[-1])
    lens.clamp_(max=16 * kw["prefix_table"].shape[1])
    return dict(kw, prefix_table=table, prefix_lens=lens, cu_groups=cu)


@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 2, 128)], ids=str)
@pytest.mark.parametrize("groups,at", [(2, 0), (129, 60), (257, 254), (1000, 0), (1000, 997), (40000, 20011)])
def test_shared_of_few_groups_among_many(heads, groups, at):
    """Pieces of prefixes are joined wherever their groups lie among those without tokens."""
    c = Shared(groups, [(2600, [(5 + i, 9) for i in range(4)]), (1111, [(1, 40), (60, 33)])], *heads, 16, "bf16")
    kw = among(c, groups, at)
    hc.hc_kv4_attention_shared(**kw)
    c.check(kw["out"], kw["lse"])


@pytest.mark.parametrize("dim", [64, 128])
def test_shared_of_groups_of_every_size(dim):
    """Whole row tiles, cut ones and ones of a few rows, several hundred of them."""
    g = np.random.default_rng(dim)
    groups = [(int(g.integers(0, 700)), [(int(g.integers(0, 9)), int(g.integers(0, 30))) for _ in range(int(g.integers(0, 4)))])
              for _ in range(300)]
    groups[100] = (5000, [(3, 64)])
    c = Shared(3, groups, 4, 1, dim, 16, "bf16")
    c.check(*c.run())


def test_shared_of_more_shares_than_a_launch_has():
    """65,536 groups of 32,768 kv heads are 2^31 (group, head)s."""
    heads, tokens = 32768, 20
    c = Shared(1, [(30, [(1, 1)] * tokens)], 1, 1, 64, 16, "bf16")
    kw = among(c, 65536, 40000)
    wide = lambda t, axis: t.repeat_interleave(heads, axis)  # noqa: E731
    kw.update(q=wide(kw["q"], 1), codes=wide(kw["codes"], 2), scales=wide(kw["scales"], 2),
              workspace=torch.empty(tokens * heads * 66, device="cuda"),
              out=torch.full((tokens, heads, 64), 55.0, dtype=torch.bfloat16, device="cuda"), lse=torch.empty(tokens, heads, device="cuda"))
    hc.hc_kv4_attention_shared(**kw)
    assert not (kw["out"] == 55.0).any()
    for h in (0, 1, 17001, heads - 1):
        c.check(kw["out"][:, h:h + 1], kw["lse"][:, h:h + 1])
    # the others are within two roundings of these
    first = kw["out"][:, :1].float()
    assert ((kw["out"].float() - first).abs() <= 2.0 ** -6 * first.abs() + 2.0 ** -8).all()


def test_shared_of_the_largest_bound_of_many_groups():
    """2^34 (group, head)s of up to 2^38 rows each, as far as the host knows: 2^64 row tiles."""
    kv_heads, groups = 1 << 12, 1 << 22
    c = Shared(2, [(40, [(1, 1)])], 128, 1, 64, 16, "bf16")
    kw = among(c, groups, groups - 3)
    wide = lambda t, axis: t.repeat_interleave(kv_heads, axis)  # noqa: E731
    q = kw["q"].repeat(1, kv_heads, 1)
    kw.update(q=q, codes=wide(kw["codes"], 2), scales=wide(kw["scales"], 2), workspace=torch.empty(q.shape[1] * 66, device="cuda"),
              out=torch.full_like(q, 55.0), lse=torch.empty(1, q.shape[1], device="cuda"), max_shared=(1 << 31) - 1)
    hc.hc_kv4_attention_shared(**kw)
    for h in (0, 1, 2049, kv_heads - 1):
        c.check(kw["out"][:, 128 * h:128 * (h + 1)], kw["lse"][:, 128 * h:128 * (h + 1)])
