"""Speculative decoding around the hyper-connection read: ``python -m
hyper_connection_residual_read_gb300.verify_window``.

A decoder of a few layers with random weights generates for several requests at once. A
step takes each request's window of new tokens (a prompt at first, then its last token and
the drafted ones) through

    hc_window_plan                      blocks, slots and positions of the new tokens
    per layer:  hc_read                 the layer's input from the residual streams
                hc_kv4_append           its keys and values into the cache, 4 bits each
                hc_kv4_attention        each new token against its request's cache
    hc_token_logprobs                   the drafted tokens under the step's logits

A drafted token is accepted while it is the most likely one (greedy verification). Drafts
come from the request's own text: what followed the last token when it occurred before.

With ``positions`` queries and keys are normed by head and rotated (hc_kv4_append_rotary in place
of hc_kv4_append); with ``sampling`` a token is drawn for each of the window's
(hc_sample_tokens), and a drafted one is accepted while it is the one drawn, which leaves the
text as likely as without drafts; and a prompt that all requests begin with is cached once
(``share``) and read once a step for all of them (hc_kv4_attention_shared).

The matrix products between the operators (projections, logits) are torch's. Everything a
step launches reads its lengths from device memory; the host reads back one small table a
step, the verified tokens.
"""
from __future__ import annotations

import argparse

import numpy as np
import torch

import hyper_connection_residual_read_gb300 as hc
from hyper_connection_residual_read_gb300 import synth

WIDTH, STREAMS = synth.WIDTH, synth.N_STREAMS
Q_HEADS, KV_HEADS, HEAD_DIM = 20, 4, 128


class Decoder:
    """Random weights, and one paged 4-bit cache a layer with a table shared by them."""

    def __init__(self, requests: int, layers: int = 2, vocab: int = 4096, blocks: int = 512,
                 block_size: int = 32, max_tokens: int = 4096, drafts: int = 7, seed: int = 0,
                 positions: bool = False, sampling: dict | None = None, longest: int = 8192):
        g = torch.Generator().manual_seed(seed)
        normal = lambda *shape, scale: (torch.randn(shape, generator=g) * scale).bfloat16().cuda()  # noqa: E731
        self.requests, self.block_size, self.drafts, self.vocab = requests, block_size, drafts, vocab
        self.embed, self.unembed = normal(vocab, WIDTH, scale=1.0), normal(vocab, WIDTH, scale=WIDTH ** -0.5)
        self.layers = []
        for n in range(layers):
            read = {k: torch.from_numpy(v.view(np.int16)).cuda() for k, v in synth.make_weights(seed + n).items()}
            self.layers.append({
                **read,
                "qkv": normal((Q_HEADS + 2 * KV_HEADS) * HEAD_DIM, WIDTH, scale=WIDTH ** -0.5),
                "out": normal(WIDTH, Q_HEADS * HEAD_DIM, scale=WIDTH ** -0.5),
                "codes": torch.zeros((blocks, 2, KV_HEADS, block_size, HEAD_DIM // 2), dtype=torch.uint8, device="cuda"),
                "scales": torch.zeros((blocks, 2, KV_HEADS, block_size, 2), dtype=torch.bfloat16, device="cuda"),
            })
        mix = torch.softmax(torch.randn((STREAMS, STREAMS), generator=g), -1)
        self.mix = mix.cuda()
        ints = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
        self.cached, self.new, self.kv = ints(requests), ints(requests), ints(requests)
        self.cu, self.table = ints(requests + 1), ints(requests, blocks)
        self.free = torch.arange(blocks, dtype=torch.int32, device="cuda")
        self.free_count = torch.full((1,), blocks, dtype=torch.int32, device="cuda")
        self.free_left = ints(1)
        self.sampling, self.uniform = sampling, torch.Generator(device="cuda").manual_seed(seed)
        self.cos_sin = None
        if positions:
            angle = torch.arange(longest)[:, None] * 10000.0 ** (-torch.arange(0, HEAD_DIM, 2).double() / HEAD_DIM)
            self.cos_sin = torch.stack([angle.cos(), angle.sin()], 1).float().cuda()
            for w in self.layers:
                w["q_norm"], w["k_norm"] = ((1 + 0.1 * torch.randn(HEAD_DIM, generator=g)).bfloat16().cuda() for _ in range(2))
        # the blocks that all requests share, if any
        self.prefix_table, self.prefix_len = None, torch.zeros(1, dtype=torch.int32, device="cuda")
        self.one_group = torch.tensor([0, requests], dtype=torch.int32, device="cuda")
        hc.hc_read_init(torch.cuda.current_device(), max_tokens, 1e-6)

    def step(self, windows, top: int = 4) -> dict:
        """One pass over ``windows``, a list of token ids a request (a token and what is
        drafted after it). Returns the plan and, a token, the log probability of the next
        token of its window and the ``top`` most likely ones."""
        lens = [len(w) for w in windows]
        total, ints = sum(lens), dict(dtype=torch.int32, device="cuda")
        self.new.copy_(torch.tensor(lens, dtype=torch.int32))
        tokens = torch.tensor([t for w in windows for t in w], **ints)
        follow = torch.tensor([t for w in windows for t in (*w[1:], *([-1] if w else []))], **ints)   # -1: nothing to verify
        slots = torch.empty(total, dtype=torch.int64, device="cuda")
        request_of, positions = torch.empty(total, **ints), torch.empty(total, **ints)
        hc.hc_window_plan(self.cached, self.new, self.free, self.free_count, self.block_size, self.table,
                          slots, request_of, positions, self.cu, self.kv, self.free_left)
        at = positions + self.prefix_len
        if self.prefix_table is not None:
            workspace = torch.empty(total * Q_HEADS * (HEAD_DIM + 2), device="cuda")
        R = self.embed[tokens.long()].float()[:, None].repeat(1, STREAMS, 1).contiguous()
        P = None
        Rmix = self.mix.expand(total, STREAMS, STREAMS).contiguous()
        for w in self.layers:
            mixed = torch.empty((total, STREAMS, WIDTH), device="cuda")
            image, image16 = (torch.empty_like(mixed, dtype=torch.int16) for _ in range(2))
            hc.hc_read(total, R, P, w["w_norm"], w["W_down"], w["W_up"], Rmix, mixed, image, image16)
            qkv = image.view(torch.bfloat16)[:, 0] @ w["qkv"].T
            q, k, v = qkv.view(total, -1, HEAD_DIM).split([Q_HEADS, KV_HEADS, KV_HEADS], 1)
            if self.cos_sin is None:
                hc.hc_kv4_append(k, v, slots, w["codes"], w["scales"])
            else:
                turned = torch.empty((total, Q_HEADS, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
                hc.hc_kv4_append_rotary(q, k, v, self.cos_sin, at, slots, w["codes"], w["scales"], turned, w["q_norm"], w["k_norm"])
                q = turned
            o = torch.empty((total, Q_HEADS, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
            if self.prefix_table is None:
                hc.hc_kv4_attention(q, w["codes"], w["scales"], self.table, self.cu, self.kv, max(lens), o)
            else:
                hc.hc_kv4_attention_shared(q, w["codes"], w["scales"], self.prefix_table, self.prefix_len, self.one_group, total,
                                           self.table, self.cu, self.kv, max(lens), workspace, o)
            # the layer's result is the pending write of the next read
            R, P = mixed, (o.view(total, -1) @ w["out"].T).float()[:, None].repeat(1, STREAMS, 1).contiguous()
        logits = (R + P).mean(1).bfloat16() @ self.unembed.T
        flat = lambda dtype: torch.empty(total, dtype=dtype, device="cuda")  # noqa: E731
        r = {"logprob": flat(torch.float32), "entropy": flat(torch.float32), "lse": flat(torch.float32),
             "rank": flat(torch.int32), "top_ids": torch.empty((total, top), **ints),
             "top_logprobs": torch.empty((total, top), device="cuda")}
        hc.hc_token_logprobs(logits, follow, *r.values())
        r["next"] = r["top_ids"]
        if self.sampling is not None:
            r["next"], r["drawn"] = torch.empty((total, 1), **ints), flat(torch.float32)
            r["uniform"] = torch.rand(total, generator=self.uniform, device="cuda")
            settings = {k: torch.full((total,), v, dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda")
                        for k, v in self.sampling.items()}
            hc.hc_sample_tokens(logits, r["uniform"], r["next"].view(-1), r["drawn"], **settings)
        return {**r, "logits": logits, "follow": follow, "slots": slots, "request_of": request_of,
                "positions": positions, "last_keys_values": (k, v)}

    def share(self, prompt) -> None:
        """Caches what every request begins with, once; before any of them has a cache."""
        self.step([prompt, *[[]] * (self.requests - 1)])
        if int(self.kv[0]) != len(prompt):
            raise RuntimeError("no blocks left for the shared prompt")
        held = -(-len(prompt) // self.block_size)
        self.prefix_table = self.table[:1, :held].clone()
        self.prefix_len += len(prompt)
        self.free_count.copy_(self.free_left)

    def accept(self, windows, top_ids, prompt=False) -> list:
        """The tokens that each window gained: its drafted ones as far as each is the first of
        ``top_ids`` (the most likely, or drawn), and one more. The cache keeps what was verified (a prompt as a whole: ``prompt``
        says of all windows, or of each, that they are), and blocks past it are free again. A
        request whose blocks were not granted gains nothing."""
        prompt = [prompt] * len(windows) if isinstance(prompt, bool) else prompt
        best, size = top_ids[:, 0].tolist(), self.block_size
        had, cached, left = self.kv.tolist(), self.cached.tolist(), int(self.free_left)
        gained, at = [], 0
        for b, w in enumerate(windows):
            n = 0
            if had[b] == cached[b]:
                gained.append([])
            elif prompt[b]:
                gained.append([best[at + len(w) - 1]])
                cached[b] = had[b]
            else:
                while n + 1 < len(w) and w[n + 1] == best[at + n]:
                    n += 1
                gained.append([*w[1:n + 1], best[at + n]])
                cached[b] += n + 1
            at += len(w)
            kept, taken = -(-cached[b] // size), -(-had[b] // size)
            self.free[left:left + taken - kept] = self.table[b, kept:taken]
            left += taken - kept
        self.cached.copy_(torch.tensor(cached, dtype=torch.int32))
        self.free_count.fill_(left)
        return gained

    def release(self, request: int) -> None:
        """Drops what the cache holds of a request; its blocks are free again."""
        held, left = -(-int(self.cached[request]) // self.block_size), int(self.free_count)
        self.free[left:left + held] = self.table[request, :held]
        self.free_count.fill_(left + held)
        self.cached[request] = 0

    def read_back(self, layer: int, slots):
        """Keys and values that the cache holds in ``slots``."""
        w = self.layers[layer]
        k, v = (torch.empty((slots.numel(), KV_HEADS, HEAD_DIM), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        hc.hc_kv4_load(slots, w["codes"], w["scales"], k, v)
        return k, v


def draft(text: list, count: int) -> list:
    """What followed the last token where it occurred before, at most ``count`` tokens."""
    for i in range(len(text) - 2, -1, -1):
        if text[i] == text[-1]:
            return text[i + 1:i + 1 + count]
    return []


def generate(decoder: Decoder, prompts: list, tokens: int, propose=draft) -> tuple:
    """Continues ``prompts`` by at least ``tokens`` tokens each; returns the texts, the
    steps after the prompt and the log probabilities of the accepted drafts. A request
    that finds no blocks for its prompt waits and sends it again; one that is done gives its
    blocks back."""
    texts, steps, accepted = [list(p) for p in prompts], -1, []
    goal = [len(p) + tokens for p in prompts]
    waits, held = [True] * len(prompts), [False] * len(prompts)      # for its prompt to be cached; is cached
    while any(len(t) < n for t, n in zip(texts, goal)):
        windows = [[] if len(t) >= n else list(t) if w else [t[-1], *propose(t, decoder.drafts)]
                   for t, n, w in zip(texts, goal, waits)]
        r = decoder.step(windows)
        gained = decoder.accept(windows, r["next"], prompt=waits)
        logprob, at = r["logprob"].tolist(), 0
        for b, (text, window, more) in enumerate(zip(texts, windows, gained)):
            text += more
            if more and not waits[b]:
                accepted += logprob[at:at + len(more) - 1]
            if more:
                waits[b], held[b] = False, True
            at += len(window)
        freed = [b for b, t in enumerate(texts) if held[b] and len(t) >= goal[b]]
        for b in freed:
            decoder.release(b)
            held[b] = False
        if not any(gained) and not freed:
            raise RuntimeError("no blocks left for any request")
        steps += 1
    return texts, max(steps, 0), accepted


def main() -> None:
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--requests", type=int, default=8)
    parser.add_argument("--tokens", type=int, default=64)
    parser.add_argument("--layers", type=int, default=2)
    parser.add_argument("--positions", action="store_true", help="norm and rotate queries and keys")
    parser.add_argument("--shared", type=int, default=0, help="tokens of a prompt that all requests begin with")
    parser.add_argument("--temperature", type=float, help="draw tokens instead of taking the most likely (1 where a filter is given)")
    parser.add_argument("--top-k", type=int, default=0)
    parser.add_argument("--top-p", type=float, default=1.0)
    parser.add_argument("--min-p", type=float, default=0.0)
    args = parser.parse_args()
    g = np.random.default_rng(0)
    sampling = None
    if args.temperature is not None or args.top_k > 0 or args.top_p < 1 or args.min_p > 0:
        sampling = dict(temperature=1.0 if args.temperature is None else args.temperature, top_k=args.top_k,
                        top_p=args.top_p, min_p=args.min_p)
    shared = np.random.default_rng(1).integers(0, 4096, args.shared).tolist()

    def make():
        decoder = Decoder(args.requests, args.layers, positions=args.positions, sampling=sampling)
        if shared:
            decoder.share(shared)
        return decoder
    decoder = make()
    prompts = [g.integers(0, decoder.vocab, 20 + 30 * b).tolist() for b in range(args.requests)]
    texts, steps, accepted = generate(decoder, prompts, args.tokens)
    # the same text again, drafted from what was generated
    again = make()
    known = {tuple(p): t for p, t in zip(prompts, texts)}

    def recall(text, count):
        for prompt, whole in known.items():
            if tuple(text[:len(prompt)]) == prompt:
                return whole[len(text):len(text) + count]
        return []
    texts2, steps2, accepted2 = generate(again, prompts, args.tokens, recall)
    torch.cuda.synchronize()
    code = hc.hc_read_status()
    if code != hc.HC_OK:
        raise SystemExit(f"device status {code}: {hc.strerror(code)}")
    for name, s, a in (("drafts from the text", steps, accepted), ("drafts from an earlier run", steps2, accepted2)):
        mean = f", mean log probability {sum(a) / len(a):.2f}" if a else ""
        print(f"{name}: {args.requests} requests x {args.tokens} tokens in {s} steps, {len(a)} drafted tokens accepted{mean}")


if __name__ == "__main__":
    main()
