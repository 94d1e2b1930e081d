"""The operators of include/hc_serve.h together with the others, as a decoder with positions, a
shared prompt and sampling uses them."""
import numpy as np
import pytest
import torch

from oracle import serve_oracle as S

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import hyper_connection_residual_read_gb300 as hc
    from hyper_connection_residual_read_gb300 import verify_window as vw

SAMPLING = dict(temperature=0.9, top_k=40, top_p=0.95, min_p=0.01)


def tokens(seed, *lens):
    g = np.random.default_rng(seed)
    return [g.integers(0, 4096, n).tolist() for n in lens]


def test_a_shared_prompt_gives_what_whole_prompts_give():
    """One layer: a token's logits depend on its attention over the prompt alone. Attention is
    within 2^-9 of the values' sizes either way (tests/test_gpu_window.py), its rounding to bf16
    2^-8; the logits are products with rows of unit length on average: 2^-5 of the largest."""
    common, *own = tokens(3, 200, 5, 1, 40, 17)
    a = vw.Decoder(4, layers=1, positions=True)
    a.share(common)
    assert int(a.free_count) == 512 - 7 and a.cached.tolist() == [0] * 4
    ra = a.step(own)
    b = vw.Decoder(4, layers=1, positions=True)
    rb = b.step([common + p for p in own])
    last = np.cumsum([len(common) + len(p) for p in own])
    rows = np.concatenate([np.arange(e - len(p), e) for e, p in zip(last, own)])
    x, y = ra["logits"].float(), rb["logits"].float()[torch.from_numpy(rows).cuda()]
    assert (x - y).abs().max() <= 2.0 ** -5 * y.abs().max()
    # queries, keys and values are the same ones: the caches of the own tokens hold the same
    for u, v in zip(a.read_back(0, ra["slots"]), b.read_back(0, rb["slots"][torch.from_numpy(rows).cuda()])):
        assert torch.equal(u, v)
    assert hc.hc_read_status() == hc.HC_OK


def test_what_is_drawn_are_the_oracles_tokens():
    d = vw.Decoder(3, layers=2, positions=True, sampling=SAMPLING)
    d.share(tokens(5, 70)[0])
    r = d.step(tokens(6, 4, 20, 1))
    x, drawn = r["logits"].double().cpu().numpy(), r["next"][:, 0].tolist()
    for t in range(25):
        each = {k: float(np.float32(v)) if k != "top_k" else v for k, v in SAMPLING.items()}
        token, lp, near = S.sample(x[t], float(r["uniform"][t]), **each)
        assert near < 2.0 ** -27 or (drawn[t] == token and abs(float(r["drawn"][t]) - lp) <= 2.0 ** -20 * (1 + abs(lp)))
    gained = d.accept([[1] * 4, [1] * 20, [1]], r["next"], prompt=True)
    assert gained == [[drawn[3]], [drawn[23]], [drawn[24]]]
    assert hc.hc_read_status() == hc.HC_OK


@pytest.mark.parametrize("shared", [0, 33, 500])
def test_generation_with_positions_and_sampling(shared):
    d = vw.Decoder(4, layers=2, positions=True, sampling=SAMPLING)
    if shared:
        d.share(tokens(7, shared)[0])
    free = int(d.free_count)
    p = tokens(8, 3, 40, 65, 7)
    texts, steps, _ = vw.generate(d, p, 20)
    assert all(len(t) >= len(q) + 20 and t[:len(q)] == q for t, q in zip(texts, p)) and steps <= 19
    assert int(d.free_count) == free and hc.hc_read_status() == hc.HC_OK


def test_operators_called_one_after_the_other_wait_for_each_other():
    """Each kernel is set up while the one before it runs: the results are those of calls with a
    synchronisation between them, bit for bit."""
    heads, dim, block, requests = 4, 128, 16, 6
    ints = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    hc.hc_read_init(0, 512, 1e-6)
    angle = torch.arange(1000)[:, None] * 10000.0 ** (-torch.arange(0, dim, 2).double() / dim)
    table_cs = torch.stack([angle.cos(), angle.sin()], 1).float().cuda()

    def run(pause):
        wait = torch.cuda.synchronize if pause else (lambda: None)
        gen = torch.Generator().manual_seed(5)
        codes = torch.randint(0, 256, (300, 2, heads, block, dim // 2), generator=gen, dtype=torch.uint8).cuda()
        scales = torch.rand((300, 2, heads, block, 2), generator=gen).bfloat16().cuda()
        cached, table = ints(requests), ints(requests, 64)
        prefix_table = torch.arange(256, 300, dtype=torch.int32, device="cuda").view(2, 22)
        prefix_lens, groups = ints(2) + 341, torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
        free, count, left = torch.arange(256, dtype=torch.int32, device="cuda"), ints(1) + 256, ints(1)
        cu, kv = ints(requests + 1), ints(requests)
        results = []
        for new in (40, 1, 8, 1, 33, 3, 1, 8):
            total = new * requests
            x = torch.randn((total, 6 * heads, dim), generator=gen).bfloat16().cuda()
            q, k, v = x.split([4 * heads, heads, heads], 1)
            lens = ints(requests) + new
            slots, of, at = torch.empty(total, dtype=torch.int64, device="cuda"), ints(total), ints(total)
            turned, o = torch.empty_like(q.contiguous()), torch.empty_like(q.contiguous())
            work = torch.empty(total * 4 * heads * (dim + 2), device="cuda")
            n = total * 4 * heads
            ids, lp, u = ints(n), torch.empty(n, device="cuda"), torch.rand(n, generator=gen).cuda()
            p, top_k = torch.full((n,), 0.9, device="cuda"), ints(n) + 20
            wait()
            hc.hc_window_plan(cached, lens, free, count, block, table, slots, of, at, cu, kv, left)
            wait()
            hc.hc_kv4_append_rotary(q, k, v, table_cs, at, slots, codes, scales, turned)
            wait()
            hc.hc_kv4_attention_shared(turned, codes, scales, prefix_table, prefix_lens, groups, 4 * new, table, cu, kv, new, work, o)
            wait()
            hc.hc_sample_tokens(o.view(n, dim), u, ids, lp, top_k=top_k, top_p=p)
            wait()
            cached, kv, count, left = kv, cached, left, count
            results += [turned, o, ids, lp, slots, codes.clone(), table.clone()]
            wait()
        torch.cuda.synchronize()
        return results

    first = run(False)
    for _ in range(3):
        for a, b in zip(run(True), first):
            assert torch.equal(a, b)
        for a, b in zip(run(False), first):
            assert torch.equal(a, b)
    assert hc.hc_read_status() == hc.HC_OK
