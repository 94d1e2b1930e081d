"""The read and the window operators one after the other on a stream, each on what the one
before it wrote and nothing in between: every kernel is set up while the one before it
runs, and the results are those of calls with a synchronisation between them, bit for bit."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import hyper_connection_residual_read_gb300 as hc
    from hyper_connection_residual_read_gb300 import synth

STREAMS, WIDTH, HEADS, DIM, BLOCK = 4, 2560, 80, 128, 16       # 4 x 2560 = 80 x 128


def chain(tokens, read, pause, rounds=4):
    """A read's bf16 image is the keys, values and queries of a window; the cache read back
    in fp32 is the streams and the pending write of the next read, whose output is scored."""
    wait = torch.cuda.synchronize if pause else (lambda: None)
    ints = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    act = synth.make_activations(5, tokens, True)
    w = {k: torch.from_numpy(np.ascontiguousarray(v).view(np.int16)).cuda() for k, v in synth.make_weights(0).items()}
    f32 = lambda *shape: torch.zeros(shape, device="cuda")  # noqa: E731
    R, P, mix = (torch.from_numpy(np.ascontiguousarray(act[k])).cuda() for k in ("R", "P", "Rmix"))
    blocks = rounds * tokens // BLOCK + 2
    codes = torch.zeros((blocks, 2, HEADS, BLOCK, DIM // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((blocks, 2, HEADS, BLOCK, 2), dtype=torch.bfloat16, device="cuda")
    cached, new, table = ints(1), ints(1) + tokens, ints(1, blocks)
    free, count, left = torch.arange(blocks, dtype=torch.int32, device="cuda"), ints(1) + blocks, ints(1)
    slots, of, at, cu, kv = torch.zeros(tokens, dtype=torch.int64, device="cuda"), ints(tokens), ints(tokens), ints(2), ints(1)
    out, b16, h16 = f32(tokens, STREAMS, WIDTH), *(torch.zeros((tokens, STREAMS, WIDTH), dtype=torch.int16, device="cuda") for _ in range(2))
    o, lse = torch.zeros((tokens, HEADS, DIM), dtype=torch.bfloat16, device="cuda"), f32(tokens, HEADS)
    ids, rank, top, toplp, lp, ent, sums = ints(tokens), ints(tokens), ints(tokens, 5), f32(tokens, 5), f32(tokens), f32(tokens), f32(tokens)
    results = []
    wait()
    for _ in range(rounds):
        hc.hc_window_plan(cached, new, free, count, BLOCK, table, slots, of, at, cu, kv, left)
        wait()
        read(tokens, R, P, w["w_norm"], w["W_down"], w["W_up"], mix, out, b16, h16)
        wait()
        kvq = b16.view(torch.bfloat16).view(tokens, HEADS, DIM)
        hc.hc_kv4_append(kvq, kvq, slots, codes, scales)
        wait()
        hc.hc_kv4_attention(kvq, codes, scales, table, cu, kv, tokens, o, lse=lse)
        wait()
        hc.hc_kv4_load(slots, codes, scales, R.view(tokens, HEADS, DIM), P.view(tokens, HEADS, DIM))
        wait()
        hc.hc_token_logprobs(out.view(tokens, -1), ids, lp, ent, sums, rank, top, toplp)
        wait()
        cached, kv, count, left = kv, cached, left, count
        results += [x.clone() for x in (out, b16, h16, o, lse, R, P, lp, ent, sums, rank, top, toplp, slots, table)]
        wait()
    torch.cuda.synchronize()
    assert hc.hc_read_status() == hc.HC_OK
    return results


def back_to_back(tokens, read):
    hc.hc_read_init(0, 512, 1e-6)
    want = chain(tokens, read, True)
    assert all(bool(torch.isfinite(x.float()).all()) for x in want if x.dtype is torch.float32)
    for _ in range(3):
        for a, b in zip(chain(tokens, read, False), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("tokens", [1, 8, 40, 130])
def test_read_and_window_operators_back_to_back(tokens):
    """The decode kernels (up to 48 tokens, which ask for the next kernel before they wait) and
    the tile path."""
    back_to_back(tokens, lambda *a: hc.hc_read(*a))


@pytest.mark.parametrize("tokens", [3, 8])
def test_one_kernel_read_and_window_operators_back_to_back(tokens):
    back_to_back(tokens, lambda *a: hc.hc_read_path(hc.HC_PATH_DECODE_ONE_KERNEL, *a))


def test_allocation_free_read_and_window_operators_back_to_back():
    back_to_back(17, lambda *a: hc.hc_read_noalloc(*a))
