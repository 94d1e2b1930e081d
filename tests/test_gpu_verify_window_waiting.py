"""Requests that have to wait for blocks, in the speculative decoder's example."""
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


def test_a_request_that_waited_has_its_whole_prompt_cached():
    d = vw.Decoder(2, layers=1, blocks=4, block_size=32)        # three of them for the first prompt
    p = prompts(d, [90, 60])
    seen = []
    step = d.step

    def watch(windows, *args):
        before = d.cached.tolist()
        r = step(windows, *args)
        seen.append(([len(w) for w in windows], before, d.kv.tolist()))
        return r
    d.step = watch
    texts, steps, _ = vw.generate(d, p, 3, propose=lambda text, n: [])
    assert [len(t) for t in texts] == [93, 63] and [t[:n] for t, n in zip(texts, (90, 60))] == p
    for lens, before, kv in seen:
        for n, cached, held, prompt in zip(lens, before, kv, p):
            assert cached == 0 or cached >= len(prompt), "a cache that lacks part of its prompt"
            assert held in (cached, cached + n)
    assert d.cached.tolist() == [0, 0] and int(d.free_count) == 4
    assert sorted(d.free.tolist()) == [0, 1, 2, 3]
    assert hc.hc_read_status() == hc.HC_OK


def test_a_prompt_is_sent_again_until_there_are_blocks():
    """Four blocks: the second request waits until the first is done, and then gives the text
    that it gives alone."""
    d = vw.Decoder(2, layers=1, blocks=4, block_size=32)
    p = prompts(d, [90, 60])
    texts, steps, _ = vw.generate(d, p, 4, propose=lambda text, n: [])
    alone = vw.Decoder(1, layers=1, blocks=4, block_size=32)
    want, fewer, _ = vw.generate(alone, [p[1]], 4, propose=lambda text, n: [])
    assert [len(t) for t in texts] == [94, 64] and steps >= fewer + 3
    assert texts[1] == want[0]
    assert int(d.free_count) == 4 and hc.hc_read_status() == hc.HC_OK


def test_requests_that_never_fit_are_an_error():
    d = vw.Decoder(1, layers=1, blocks=2, block_size=32)
    with pytest.raises(RuntimeError):
        vw.generate(d, prompts(d, [90]), 4)
