"""The verify-window operators as cases to measure: what each call is given, its plain
form in elementary torch operations, the call of this package that does the same, and
what the result is in 64 bits.

One step of a serving loop over a paged cache held in 4 bits runs them in this order:

* ``plan``: block tables, slots and positions of the step's new tokens, from the
  requests' lengths;
* ``cache``: the new tokens' keys and values rounded to 4 bits into their slots, and
  read back from there;
* ``attention``: each new token against its request's cache;
* ``logprobs``: the drafted tokens scored on the step's logits.

The cache: ``codes`` [blocks][2][kv heads][block size][head dim / 2] bytes, keys at 0 and
values at 1, element 2i in the low half of byte i; ``scales`` [blocks][2][kv heads]
[block size][2] bf16, a step s and a minimum m per token and head: value = m + s * code.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ITEM = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed() -> list[dict]:
    return [
        # one verify step of a small batch: the call between two layers' worth of work,
        # where latency is all
        dict(name="plan_verify", op="plan", requests=32, new=8, cached=8192, block=16, pool=0.5),
        # a full server's step that takes up chunks of prompts, with a pool that runs out
        dict(name="plan_chunks", op="plan", requests=1024, new=128, cached=32768, block=16, pool=0.9),
        # the write of one verify window: 8 requests of 4 tokens
        dict(name="cache_window", op="cache", tokens=32, kv_heads=8, q_heads=32, dim=128, block=16,
             dtype="bf16"),
        # the write of an 8K prefill chunk (an odd count), fp16, wide blocks
        dict(name="cache_chunk", op="cache", tokens=8191, kv_heads=8, q_heads=32, dim=128, block=64,
             dtype="fp16"),
        # one request, one token: the smallest decode call
        dict(name="attn_single", op="attention", requests=1, new=1, cached=4001, ragged=False,
             q_heads=32, kv_heads=8, dim=128, block=16, dtype="bf16", mask=False),
        # a decode batch of ragged lengths: the cache's bytes bound it
        dict(name="attn_decode", op="attention", requests=64, new=1, cached=16384, ragged=True,
             q_heads=32, kv_heads=8, dim=128, block=16, dtype="bf16", mask=False),
        # verify windows of up to 8 drafted tokens in a tree, 20 query heads on 4 (a width
        # of 2560), long caches
        dict(name="attn_verify", op="attention", requests=16, new=8, cached=32768, ragged=True,
             q_heads=20, kv_heads=4, dim=128, block=32, dtype="bf16", mask=True),
        # chunks of prompts of several requests at once, odd lengths, narrow heads, fp16
        dict(name="attn_ragged_chunks", op="attention", requests=6, new=1001, cached=3000, ragged=True,
             q_heads=16, kv_heads=16, dim=64, block=16, dtype="fp16", mask=False),
        # an 8K prefill chunk behind 8K cached tokens: the tensor cores bound it
        dict(name="attn_chunk", op="attention", requests=1, new=8192, cached=8192, ragged=False,
             q_heads=32, kv_heads=8, dim=128, block=64, dtype="bf16", mask=False),
        # one verify window scored
        dict(name="score_window", op="logprobs", tokens=8, vocab=131072, top=8, dtype="bf16"),
        # a batch of windows, odd vocabulary (rows of no alignment), fp32 logits
        dict(name="score_batch", op="logprobs", tokens=96, vocab=50257, top=5, dtype="fp32"),
        # a prompt chunk scored
        dict(name="score_chunk", op="logprobs", tokens=4096, vocab=131072, top=20, dtype="bf16"),
    ]


def _log_int(rng, lo: int, hi: int) -> int:
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng) -> dict:
    op = rng.choice(["plan", "cache", "attention", "attention", "attention", "logprobs"])
    if op == "plan":
        return dict(op="plan", requests=_log_int(rng, 1, 1024), new=_log_int(rng, 1, 128),
                    cached=_log_int(rng, 16, 32768), block=rng.choice([16, 32, 64]),
                    pool=round(rng.uniform(0.2, 1.0), 3))
    if op == "cache":
        kv_heads = rng.choice([1, 2, 4, 8])
        return dict(op="cache", tokens=_log_int(rng, 1, 8192), kv_heads=kv_heads,
                    q_heads=kv_heads * rng.choice([1, 2, 4, 5]), dim=rng.choice([64, 128]),
                    block=rng.choice([16, 32, 64]), dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "logprobs":
        vocab = _log_int(rng, 1000, 131072)
        return dict(op="logprobs", tokens=_log_int(rng, 1, min(4096, (1 << 28) // vocab)), vocab=vocab,
                    top=rng.choice([0, 1, 5, 8, 20]), dtype=rng.choice(["bf16", "fp16", "fp32"]))
    kind = rng.choice(["decode", "verify", "chunk"])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 4, 5, 7, 8])
    case = dict(op="attention", ragged=rng.random() < 0.7, q_heads=kv_heads * group, kv_heads=kv_heads,
                dim=rng.choice([64, 128]), block=rng.choice([16, 32, 64, 128]),
                dtype=rng.choice(["bf16", "fp16"]), mask=kind == "verify" and rng.random() < 0.5)
    if kind == "chunk":
        case["requests"] = _log_int(rng, 1, 8)
        case["new"] = _log_int(rng, 64, 4096 // case["requests"])
        case["cached"] = _log_int(rng, 16, 8192)
    else:
        case["new"] = 1 if kind == "decode" else rng.randint(2, 8)
        case["cached"] = _log_int(rng, 16, 32768)
        case["requests"] = _log_int(rng, 1, max(1, min(128, (1 << 19) // case["cached"])))
    return case


def _lens(case: dict) -> tuple[np.ndarray, np.ndarray]:
    """Cached and new tokens of each request: part of the case, the same for every seed."""
    n = case["requests"]
    r = np.random.RandomState(n * 7919 + case["new"] * 31 + case["cached"])
    if not case["ragged"]:
        return np.full(n, case["cached"]), np.full(n, case["new"])
    cached = r.randint(0, case["cached"] + 1, n)
    new = r.randint(1, case["new"] + 1, n)
    cached[r.randint(n)], new[r.randint(n)] = case["cached"], case["new"]
    return cached, new


def work(case: dict) -> dict:
    op = case["op"]
    if op == "plan":
        n, tokens = case["requests"], case["requests"] * (case["new"] + 1) / 2
        new_blocks = tokens / case["block"]
        return dict(bytes=4 * (2 * n + 1) + 4 * (2 * n + 2) + 16 * tokens + 8 * new_blocks, flops=0)
    if op == "cache":
        values = 2 * case["tokens"] * case["kv_heads"] * case["dim"]
        held = 2 * case["tokens"] * case["kv_heads"] * (case["dim"] // 2 + 4)
        return dict(bytes=2 * values * ITEM[case["dtype"]] + 2 * held + 8 * case["tokens"], flops=0)
    if op == "logprobs":
        return dict(bytes=case["tokens"] * (case["vocab"] * ITEM[case["dtype"]] + 20 + 8 * case["top"]),
                    flops=0)
    cached, new = (x.astype(np.float64) for x in _lens(case))
    pairs = float((new * cached + new * (new + 1) / 2).sum())
    tokens = float(new.sum())
    held = 2 * case["kv_heads"] * (case["dim"] // 2 + 4) * float((cached + new).sum())
    rows = 2 * ITEM[case["dtype"]] * tokens * case["q_heads"] * case["dim"] + 4 * tokens * case["q_heads"]
    return dict(bytes=held + rows, flops=4.0 * pairs * case["q_heads"] * case["dim"])


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)


def _int32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def _pages(gen, blocks: int, kv_heads: int, block: int, dim: int):
    """A cache pool as earlier steps left it: codes near normal about the middle, steps
    and minima of keys and values of about unit size."""
    codes = torch.empty(blocks, 2, kv_heads, block, dim // 2, dtype=torch.uint8, device="cuda")
    for i in range(0, blocks, 8192):
        n = min(8192, blocks - i)
        c = _randn(gen, n, 2, kv_heads, block, dim).mul_(2.8).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
        codes[i:i + n] = c[..., 0::2] | (c[..., 1::2] << 4)
    step = 0.36 * torch.exp(0.3 * _randn(gen, blocks, 2, kv_heads, block))
    low = -7.5 * step + 0.1 * _randn(gen, blocks, 2, kv_heads, block)
    return codes, torch.stack([step, low], dim=-1).to(torch.bfloat16)


def _prepare_plan(case: dict, seed: int) -> dict:
    r = np.random.RandomState(seed % (1 << 31))
    n, bs = case["requests"], case["block"]
    cached = r.randint(0, case["cached"] + 1, n)
    new = r.randint(1, case["new"] + 1, n)
    have, total = -(-cached // bs), -(-(cached + new) // bs)
    width = -(-(case["cached"] + case["new"]) // bs)
    free = max(1, int(case["pool"] * max(1, int((total - have).sum()))))
    order = r.permutation(int(have.sum()) + free)
    table = np.full((n, width), -1)
    table[np.arange(width)[None, :] < have[:, None]] = order[: int(have.sum())]
    capacity = n * case["new"]
    z = lambda *shape, dtype=torch.int32: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    return dict(cached=_int32(cached), new=_int32(new), free=_int32(order[int(have.sum()):]),
                free_count=_int32([free]), block=bs, table=_int32(table),
                slots=z(capacity, dtype=torch.int64), request_of=z(capacity), positions=z(capacity),
                cu=z(n + 1), kv=z(n), free_left=z(1))


def _prepare_cache(case: dict, seed: int) -> dict:
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t, h, d, bs, dt = case["tokens"], case["kv_heads"], case["dim"], case["block"], DTYPES[case["dtype"]]
    hq = case["q_heads"]
    # keys and values are slices of the fused projection's rows
    qkv = _randn(gen, t, (hq + 2 * h) * d)
    qkv[:, hq * d:(hq + h) * d] += _randn(gen, h * d)      # keys have an offset by channel
    qkv = qkv.to(dt)
    blocks = -(-t // bs) + 8
    codes, scales = _pages(gen, blocks, h, bs, d)
    pages = torch.randperm(blocks, generator=gen, device="cuda")[: -(-t // bs)]
    at = torch.arange(t, device="cuda")
    slots = pages[at // bs] * bs + at % bs
    return dict(k=qkv[:, hq * d:(hq + h) * d].view(t, h, d), v=qkv[:, (hq + h) * d:].view(t, h, d),
                slots=slots, codes=codes, scales=scales,
                k_out=torch.empty(t, h, d, dtype=dt, device="cuda"),
                v_out=torch.empty(t, h, d, dtype=dt, device="cuda"))


def _prepare_attention(case: dict, seed: int) -> dict:
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cached, new = _lens(case)
    n, bs, d, h, hq = case["requests"], case["block"], case["dim"], case["kv_heads"], case["q_heads"]
    kv, tokens = cached + new, int(new.sum())
    have = -(-kv // bs)
    width, blocks = int(have.max()), int(have.sum()) + 4
    codes, scales = _pages(gen, blocks, h, bs, d)
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    held = torch.from_numpy(np.arange(width)[None, :] < have[:, None]).cuda()
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    table[held] = order[: int(have.sum())]
    # what lies behind a request's end in its last block was never written
    end = torch.from_numpy(have * bs - kv).cuda()
    last = table[torch.arange(n, device="cuda"), torch.from_numpy(have - 1).cuda()].long()
    blank = torch.arange(bs, device="cuda")[None, :] >= bs - end[:, None]
    tail = scales[last]
    tail.masked_fill_(blank[:, None, None, :, None], float("nan"))
    scales[last] = tail
    qkv = (_randn(gen, tokens, (hq + 2 * h) * d) * 1.5).to(DTYPES[case["dtype"]])
    mask = None
    if case["mask"]:
        # a draft tree: each token sees its ancestors and itself
        r = np.random.RandomState(seed % (1 << 31))
        bits = []
        for m in new:
            for i in range(int(m)):
                up = bits[len(bits) - i + r.randint(i)] if i else 0
                bits.append(up | (1 << i))
        mask = torch.from_numpy(np.array(bits, dtype=np.int64)).cuda()
    cu = np.concatenate([[0], np.cumsum(new)])
    return dict(q=qkv[:, : hq * d].view(tokens, hq, d), codes=codes, scales=scales, table=table,
                cu=_int32(cu), kv=_int32(kv), max_new=int(new.max()), max_kv=int(kv.max()), mask=mask,
                scale=1.0 / math.sqrt(d), out=torch.empty(tokens, hq, d, dtype=qkv.dtype, device="cuda"),
                lse=torch.empty(tokens, hq, dtype=torch.float32, device="cuda"))


def _prepare_logprobs(case: dict, seed: int) -> dict:
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t, v, k = case["tokens"], case["vocab"], case["top"]
    logits = torch.empty(t, v, dtype=DTYPES[case["dtype"]], device="cuda")
    for i in range(0, t, 512):
        x = _randn(gen, min(512, t - i), v).mul_(2.5)
        x[:, ::997] += 6.0                                   # a few likely tokens
        logits[i:i + 512] = x
    logits[:, 7 % v] = float("-inf")                         # a token the sampler forbids
    tokens = torch.randint(0, v, (t,), generator=gen, device="cuda")
    tokens = torch.where(torch.arange(t, device="cuda") % 3 == 0, tokens, tokens // 997 * 997)
    e = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    return dict(logits=logits, tokens=tokens.to(torch.int32), logprob=e(t), entropy=e(t), lse=e(t),
                rank=e(t, dtype=torch.int32), top_ids=e(t, k, dtype=torch.int32), top_logprobs=e(t, k))


def prepare(case: dict, seed: int) -> dict:
    made = dict(plan=_prepare_plan, cache=_prepare_cache, attention=_prepare_attention,
                logprobs=_prepare_logprobs)[case["op"]](case, seed)
    made["op"] = case["op"]
    return made


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _plain_plan(s: dict) -> dict:
    bs, table = s["block"], s["table"]
    n, width = table.shape
    cached, new = s["cached"].long().clamp(min=0), s["new"].long().clamp(min=0)
    have, total = (cached + bs - 1) // bs, (cached + new + bs - 1) // bs
    fits = total <= width
    want = torch.where(fits, total - have, 0)
    upto = want.cumsum(0)
    granted = fits & ((want == 0) | (upto <= s["free_count"]))
    col = torch.arange(width, device=table.device)[None, :]
    take = s["free_count"] - 1 - (upto - want)[:, None] - (col - have[:, None])
    fresh = granted[:, None] & (col >= have[:, None]) & (col < total[:, None])
    table.copy_(torch.where(fresh, s["free"][torch.where(fresh, take, 0)], table))
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    t = torch.arange(s["slots"].shape[0], device=table.device)
    of = torch.searchsorted(cu[1:], t, right=True)
    there = of < n
    of = of.clamp(max=n - 1)
    pos = cached[of] + t - cu[of]
    put = there & granted[of]
    slot = table[of, (pos // bs).clamp(max=width - 1)].long() * bs + pos % bs
    return dict(table=table, slots=torch.where(put, slot, -1),
                request_of=torch.where(there, of, -1).int(), positions=torch.where(there, pos, -1).int(),
                cu=cu.int(), kv=(cached + torch.where(granted, new, 0)).int(),
                free_left=(s["free_count"] - (want * granted).sum()).int())


def _bf16_floor(x):
    bits = x.view(torch.int32)
    cut = bits & -65536
    return torch.where((x < 0) & (cut != bits), cut + 65536, cut).view(torch.float32)


def _bf16_ceil(x):
    return -_bf16_floor(-x)


def _plain_round(x):
    """Codes, step and minimum of each row of the last axis."""
    x = x.float()
    low, high = x.amin(-1), x.amax(-1)
    m = _bf16_floor(low)
    s = _bf16_ceil((high - m) * (1.0 / 15.0))
    s = torch.where((s > 0) & (s < 2.0 ** -126), 2.0 ** -126, s)
    r = torch.where(s > 0, torch.ones_like(s) / s, 0.0)
    code = ((x - m[..., None]) * r[..., None]).round().clamp(0, 15)
    fine = torch.isfinite(low) & torch.isfinite(high) & torch.isfinite(s)
    code = torch.where(fine[..., None], code, 0.0).to(torch.uint8)
    nan = torch.full_like(m, float("nan"))
    return code, torch.where(fine, s, nan), torch.where(fine, m, nan)


def _plain_values(codes, scales):
    low = (codes & 15).float()
    high = (codes >> 4).float()
    c = torch.stack([low, high], dim=-1).flatten(-2)
    return scales[..., 1:].float() + scales[..., :1].float() * c


def _plain_cache(s: dict) -> dict:
    codes, scales, bs = s["codes"], s["scales"], s["codes"].shape[3]
    blk, off = s["slots"] // bs, s["slots"] % bs
    ck, sk, mk = _plain_round(s["k"])
    cv, sv, mv = _plain_round(s["v"])
    c = torch.stack([ck, cv], dim=1)
    codes[blk, :, :, off] = c[..., 0::2] | (c[..., 1::2] << 4)
    scales[blk, :, :, off] = torch.stack([torch.stack([sk, mk], -1), torch.stack([sv, mv], -1)],
                                         dim=1).to(torch.bfloat16)
    kv = _plain_values(codes[blk, :, :, off], scales[blk, :, :, off]).to(s["k"].dtype)
    return dict(k=kv[:, 0], v=kv[:, 1])


def _plain_attention(s: dict) -> dict:
    q, table, cu, kv = s["q"], s["table"].long(), s["cu"].long(), s["kv"].long()
    codes, scales = s["codes"], s["scales"]
    tokens, hq, d = q.shape
    h, bs = codes.shape[2], codes.shape[3]
    n, g, w = table.shape[0], hq // h, s["max_new"]
    j = torch.arange(s["max_kv"], device=q.device)
    held = j < kv[:, None]
    blk = torch.where(held, table[:, j // bs], 0)
    off = (j % bs).expand_as(blk)
    sc = torch.where(held[:, :, None, None], scales[blk, 0, :, off], 0)
    k = _plain_values(codes[blk, 0, :, off], sc).transpose(1, 2)              # [n][h][kv][d]
    sc = torch.where(held[:, :, None, None], scales[blk, 1, :, off], 0)
    v = _plain_values(codes[blk, 1, :, off], sc).transpose(1, 2)
    new = cu[1:] - cu[:-1]
    i = torch.arange(w, device=q.device)
    here = (cu[:-1, None] + i).clamp(max=tokens - 1)                          # [n][w]
    rows = q.float()[here].view(n, w, h, g, d).permute(0, 2, 3, 1, 4).reshape(n, h, g * w, d)
    a = torch.matmul(rows, k.transpose(2, 3)).mul_(s["scale"]).view(n, h, g, w, -1)
    first = (kv - new)[:, None, None]
    if s["mask"] is None:
        sees = j <= first + i[:, None]
    else:
        bit = (s["mask"][here][:, :, None] >> (j - first).clamp(0, 63)) & 1
        sees = (j < first) | (bit == 1)
    a.masked_fill_(~(sees & held[:, None, :])[:, None, None], float("-inf"))
    top = a.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    a.sub_(top).exp_()
    total = a.sum(-1, keepdim=True)
    o = torch.matmul(a.view(n, h, g * w, -1), v).view(n, h, g, w, d) / torch.where(total > 0, total, 1.0)
    lse = (total.log() + top).squeeze(-1)
    t = torch.arange(tokens, device=q.device)
    of = torch.searchsorted(cu[1:], t, right=True)
    at = t - cu[of]
    return dict(out=o[of, :, :, at].reshape(tokens, hq, d).to(q.dtype),
                lse=lse[of, :, :, at].reshape(tokens, hq))


def _plain_logprobs(s: dict) -> dict:
    x = s["logits"].float()
    rows, v = x.shape
    k = s["top_ids"].shape[1]
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    lse = top + total.log()
    mine = x.gather(1, s["tokens"].long()[:, None])
    below = torch.where(e > 0, e * (x - top), 0.0).sum(-1, keepdim=True)
    entropy = total.log() - below / total
    # order by value, then by index: one whole number for both
    bits = (x + 0.0).view(torch.int32)
    bits = bits ^ ((bits >> 31) & 0x7FFFFFFF)
    key = (bits.long() << 32) | torch.arange(v - 1, -1, -1, device=x.device)
    ids = v - 1 - (key.topk(k, dim=1).values & 0xFFFFFFFF)
    return dict(logprob=(mine - lse)[:, 0], entropy=entropy[:, 0], lse=lse[:, 0],
                rank=(x > mine).sum(-1).int(), top_ids=ids.int(), top_logprobs=x.gather(1, ids) - lse)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

_hc = None


def _library():
    global _hc
    if _hc is None:
        import hyper_connection_residual_read_gb300 as hc
        hc.hc_read_init(torch.cuda.current_device(), 8)
        _hc = hc
    return _hc


def _own_plan(s: dict) -> dict:
    _library().hc_window_plan(s["cached"], s["new"], s["free"], s["free_count"], s["block"], s["table"],
                              s["slots"], s["request_of"], s["positions"], s["cu"], s["kv"],
                              s["free_left"])
    return dict(table=s["table"], slots=s["slots"], request_of=s["request_of"],
                positions=s["positions"], cu=s["cu"], kv=s["kv"], free_left=s["free_left"])


def _own_cache(s: dict) -> dict:
    hc = _library()
    hc.hc_kv4_append(s["k"], s["v"], s["slots"], s["codes"], s["scales"])
    hc.hc_kv4_load(s["slots"], s["codes"], s["scales"], s["k_out"], s["v_out"])
    return dict(k=s["k_out"], v=s["v_out"])


def _own_attention(s: dict) -> dict:
    _library().hc_kv4_attention(s["q"], s["codes"], s["scales"], s["table"], s["cu"], s["kv"],
                                s["max_new"], s["out"], lse=s["lse"], mask=s["mask"], scale=s["scale"])
    return dict(out=s["out"], lse=s["lse"])


def _own_logprobs(s: dict) -> dict:
    _library().hc_token_logprobs(s["logits"], s["tokens"], s["logprob"], s["entropy"], s["lse"],
                                 s["rank"], s["top_ids"], s["top_logprobs"])
    return {k: s[k] for k in ("logprob", "entropy", "lse", "rank", "top_ids", "top_logprobs")}


_PLAIN = dict(plan=_plain_plan, cache=_plain_cache, attention=_plain_attention, logprobs=_plain_logprobs)
_OWN = dict(plan=_own_plan, cache=_own_cache, attention=_own_attention, logprobs=_own_logprobs)


def run(state: dict) -> dict:
    return (_OWN if own else _PLAIN)[state["op"]](state)


# ---------------------------------------------------------------------------
# in 64 bits
# ---------------------------------------------------------------------------

def _exact_cache(s: dict) -> dict:
    """What the slots stand for. The codes are those of the definition, whose two steps
    are single fp32 roundings: each is exact in 64 bits before it is rounded to fp32."""
    out = {}
    for name in ("k", "v"):
        x = s[name].double().cpu().numpy()
        low, high = x.min(-1), x.max(-1)
        f32 = lambda a: a.astype(np.float32).astype(np.float64)  # noqa: E731

        def bf16(a, towards):
            frac, e = np.frexp(a)
            unit = np.exp2(np.maximum(e, -125).astype(np.float64) - 8)
            return towards(a / unit) * unit

        m = bf16(low, np.floor)
        s0 = f32(f32(high - m) * np.float64(np.float32(1.0 / 15.0)))
        step = bf16(s0, np.ceil)
        step = np.where((step > 0) & (step < 2.0 ** -126), 2.0 ** -126, step)
        r = np.where(step > 0, f32(1.0 / np.where(step > 0, step, 1.0)), 0.0)
        code = np.clip(np.rint(f32(f32(x - m[..., None]) * r[..., None])), 0, 15)
        out[name] = m[..., None] + step[..., None] * code
    return out


def _exact_attention(case: dict, s: dict):
    """Request by request and head by head in 64 bits."""
    tokens, hq, d = s["q"].shape
    h, bs = s["codes"].shape[2], s["codes"].shape[3]
    g = hq // h
    out = torch.zeros(tokens, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((tokens, hq), float("-inf"), dtype=torch.float64, device="cuda")
    cu, kv = s["cu"].tolist(), s["kv"].tolist()
    for b, length in enumerate(kv):
        a0, a1 = cu[b], cu[b + 1]
        if a1 == a0 or length == 0:
            continue
        pages = s["table"][b, : -(-length // bs)].long()
        held = s["codes"][pages].permute(1, 2, 0, 3, 4).reshape(2, h, -1, d // 2)[:, :, :length]
        sm = s["scales"][pages].permute(1, 2, 0, 3, 4).reshape(2, h, -1, 2)[:, :, :length].double()
        c = torch.empty(2, h, length, d, dtype=torch.float64, device="cuda")
        c[..., 0::2], c[..., 1::2] = held.bitwise_and(15).double(), held.bitwise_right_shift(4).double()
        c = c * sm[..., 0:1] + sm[..., 1:2]
        where = torch.arange(length, device="cuda")
        for lo in range(a0, a1, 1024):
            hi = min(a1, lo + 1024)
            at = torch.arange(lo - a0, hi - a0, device="cuda")
            if s["mask"] is None:
                hidden = where[None, :] > (length - (a1 - a0) + at)[:, None]
            else:
                back = where - (length - (a1 - a0))
                set_ = torch.bitwise_and(s["mask"][lo:hi, None], torch.ones_like(back) << back.clamp(0, 62)) != 0
                hidden = (back >= 0)[None, :] & ~set_
            for head in range(hq):
                z = s["q"][lo:hi, head].double() @ c[0, head // g].T * s["scale"]
                z = z.masked_fill(hidden, float("-inf"))
                lse[lo:hi, head] = torch.logsumexp(z, -1)
                out[lo:hi, head] = torch.exp(z - lse[lo:hi, head, None]).nan_to_num(0.0) @ c[1, head // g]
    return dict(out=out, lse=lse)


def _exact_logprobs(s: dict) -> dict:
    parts = []
    for i in range(0, s["logits"].shape[0], 256):
        x = s["logits"][i:i + 256].double()
        lse = torch.logsumexp(x, -1, keepdim=True)
        lp = x - lse
        p = lp.exp()
        top = x.sort(-1, descending=True).values[:, : s["top_ids"].shape[1]]
        parts.append(dict(logprob=lp.gather(1, s["tokens"][i:i + 256].long()[:, None])[:, 0],
                          entropy=-torch.where(p > 0, p * lp, 0.0).sum(-1), lse=lse[:, 0],
                          top_logprobs=top - lse))
    made = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    return dict(made, rank=None, top_ids=None)


def exact(case: dict, seed: int):
    """None for whole numbers, which the plain form gives exactly, and where 64 bits would
    take too long."""
    if case["op"] == "plan" or (case["op"] == "attention" and work(case)["flops"] > 4e12):
        return None
    s = prepare(case, seed)
    if case["op"] == "cache":
        return _exact_cache(s)
    return _exact_logprobs(s) if case["op"] == "logprobs" else _exact_attention(case, s)
