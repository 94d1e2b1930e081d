"""The operators together, as a speculative decoder uses them."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import hyper_connection_residual_read_gb300 as hc
    from hyper_connection_residual_read_gb300 import verify_window as vw


def prompts(decoder, lens):
    g = np.random.default_rng(1)
    return [g.integers(0, decoder.vocab, n).tolist() for n in lens]


def test_a_prompt_and_a_window():
    d = vw.Decoder(3, layers=2, blocks=16, block_size=32)
    p = prompts(d, [5, 33, 100])
    r = d.step(p)
    assert d.cu.tolist() == [0, 5, 38, 138] and d.kv.tolist() == [5, 33, 100]
    assert r["positions"].tolist() == [*range(5), *range(33), *range(100)]
    assert r["request_of"].tolist() == [0] * 5 + [1] * 33 + [2] * 100
    assert int(d.free_left) == 16 - (1 + 2 + 4)
    # the step's numbers belong to its logits
    x = r["logits"].double()
    logp = x - torch.logsumexp(x, -1, keepdim=True)
    follow = r["follow"].long()
    has = follow >= 0
    want = logp.gather(1, follow.clamp(min=0)[:, None])[:, 0]
    assert torch.allclose(r["logprob"].double()[has], want[has], atol=1e-4, rtol=0)
    assert bool(torch.isneginf(r["logprob"][~has]).all())
    assert torch.allclose(r["entropy"].double(), -(logp.exp() * logp).sum(-1), atol=1e-3, rtol=0)
    assert torch.equal(r["rank"][has].long(), (x > x.gather(1, follow.clamp(min=0)[:, None])).sum(-1)[has])
    # the cache holds the last layer's keys and values to within a step of their groups
    for mine, back in zip(r["last_keys_values"], d.read_back(1, r["slots"])):
        mine, back = mine.double(), back.double()
        wide = mine.amax(-1) - mine.amin(-1)
        assert bool(((mine - back).abs().amax(-1) <= 0.04 * wide + 0.01 * mine.abs().amax(-1)).all())
    best = r["top_ids"][:, 0].tolist()
    assert d.accept(p, r["top_ids"], prompt=True) == [[best[4]], [best[37]], [best[137]]]
    # drafts that are wrong take nothing but their first token, and give their blocks back
    windows = [[1, *[(best[4] + 1) % d.vocab] * 40], [], [2, 3]]
    r = d.step(windows)
    assert d.kv.tolist() == [46, 33, 102] and int(d.free_left) == 8
    ids = r["top_ids"].clone()
    ids[:, 0] = -5
    assert d.accept(windows, ids) == [[-5], [], [-5]]
    assert d.cached.tolist() == [6, 33, 101] and int(d.free_count) == 9
    table, free = d.table.cpu().numpy(), d.free[:9].tolist()
    held = [*table[0, :1], *table[1, :2], *table[2, :4]]
    assert sorted([*held, *free]) == list(range(16))
    assert hc.hc_read_status() == hc.HC_OK


def test_generation_accepts_right_drafts():
    d = vw.Decoder(4, layers=2)
    p = prompts(d, [3, 40, 65, 7])
    texts, steps, _ = vw.generate(d, p, 24, propose=lambda text, n: [])
    assert steps == 23 and all(len(t) == len(q) + 24 for t, q in zip(texts, p))
    whole = {tuple(q): t for q, t in zip(p, texts)}

    def recall(text, n):
        known = next(t for q, t in whole.items() if tuple(text[:len(q)]) == q)
        return known[len(text):len(text) + n]
    d = vw.Decoder(4, layers=2)
    _, fewer, accepted = vw.generate(d, p, 24, propose=recall)
    # nearly all of 80: windows of other sizes round differently, and a text that departs from
    # the recalled one is no longer drafted right
    assert fewer <= steps and len(accepted) > 24
    assert hc.hc_read_status() == hc.HC_OK


def test_a_request_without_blocks_waits():
    d = vw.Decoder(2, layers=1, blocks=4, block_size=32)
    p = prompts(d, [90, 60])
    r = d.step(p)
    assert d.kv.tolist() == [90, 0] and int(d.free_left) == 1
    assert bool((r["slots"][90:] == -1).all())
    gained = d.accept(p, r["top_ids"], prompt=True)
    assert len(gained[0]) == 1 and gained[1] == [] and d.cached.tolist() == [90, 0]
    assert hc.hc_read_status() == hc.HC_OK


def test_operators_called_one_after_the_other_wait_for_each_other():
    """Each kernel is set up while the one before it runs: the results are those of calls
    with a synchronisation between them, bit for bit."""
    heads, dim, block, requests = 4, 128, 16, 6
    ints = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    hc.hc_read_init(0, 512, 1e-6)

    def run(pause):
        wait = torch.cuda.synchronize if pause else (lambda: None)
        gen = torch.Generator().manual_seed(5)
        codes = torch.zeros((256, 2, heads, block, dim // 2), dtype=torch.uint8, device="cuda")
        scales = torch.zeros((256, 2, heads, block, 2), dtype=torch.bfloat16, device="cuda")
        cached, table = ints(requests), ints(requests, 64)
        free, count, left = torch.arange(256, dtype=torch.int32, device="cuda"), ints(1) + 256, ints(1)
        cu, kv = ints(requests + 1), ints(requests)
        results = []
        for new in (40, 1, 8, 1, 33, 3, 1, 8):
            total = new * requests
            x = torch.randn((total, 4 * heads + 2 * heads, dim), generator=gen).bfloat16().cuda()
            q, k, v = x.split([4 * heads, heads, heads], 1)
            lens = ints(requests) + new
            slots, at, pos = torch.empty(total, dtype=torch.int64, device="cuda"), ints(total), ints(total)
            o, ko, vo = torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous()), torch.empty_like(v.contiguous())
            n = total * 4 * heads
            f32 = [torch.empty(n, device="cuda") for _ in range(3)]
            rank, ids, top = ints(n), ints(n, 3), torch.empty((n, 3), device="cuda")
            token = (torch.arange(n, device="cuda") % dim).int()
            wait()
            hc.hc_window_plan(cached, lens, free, count, block, table, slots, at, pos, cu, kv, left)
            wait()
            hc.hc_kv4_append(k, v, slots, codes, scales)
            wait()
            hc.hc_kv4_attention(q, codes, scales, table, cu, kv, new, o)
            wait()
            hc.hc_kv4_load(slots, codes, scales, ko, vo)
            wait()
            hc.hc_token_logprobs(o.view(n, dim), token, *f32, rank, ids, top)
            wait()
            cached, kv, count, left = kv, cached, left, count
            results += [o, ko, vo, slots, *f32, rank, ids, top]
        torch.cuda.synchronize()
        return results

    first = run(False)
    for _ in range(3):
        for a, b in zip(run(True), first):
            assert torch.equal(a, b)
        for a, b in zip(run(False), first):
            assert torch.equal(a, b)
    assert hc.hc_read_status() == hc.HC_OK
