"""More operators around the verify window as cases to measure: what each call is given, its
plain form in elementary torch operations, the call of this package that does the same, and
what the result is in 64 bits.

* ``rotary``: the queries and keys that a layer's projection made, normed by head and rotated
  by their positions (one or several axes), the keys and the values rounded to 4 bits into
  their slots of the paged cache, and read back from there;
* ``shared``: attention of requests that share a long prefix, each token against the prefix
  and its request's own cache;
* ``sample``: the next tokens drawn from the logits with temperature, top-k, top-p and min-p
  from given uniform numbers.

The cache is that of ``perf/operators.py``: ``codes`` [blocks][2][kv heads][block size][head
dim / 2] bytes, element 2i in the low half of byte i; ``scales`` [blocks][2][kv heads][block
size][2] bf16, a step s and a minimum m per token and head: value = m + s * code.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ITEM = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed() -> list[dict]:
    return [
        # one verify step of a small batch, 8 requests of 4 tokens, 20 query heads on 4 (a
        # width of 2560): the call between two products, where latency is all
        dict(name="rotary_window", op="rotary", tokens=32, q_heads=20, kv_heads=4, dim=128, rotary=128,
             axes=1, interleaved=False, norm=True, block=32, dtype="bf16", length=8192),
        # an 8K prefill chunk (an odd count), the usual shape: memory bounds it
        dict(name="rotary_chunk", op="rotary", tokens=8191, q_heads=32, kv_heads=8, dim=128, rotary=128,
             axes=1, interleaved=False, norm=True, block=64, dtype="bf16", length=32768),
        # images and video: three axes, neighbouring pairs, half of narrow heads rotated, no norm
        dict(name="rotary_video", op="rotary", tokens=4099, q_heads=16, kv_heads=16, dim=64, rotary=32,
             axes=3, interleaved=True, norm=False, block=16, dtype="fp16", length=4096),
        # several answers to one question: a short common prompt, the smallest decode call
        dict(name="shared_small", op="shared", groups=1, requests=8, new=1, prefix=2001, cached=200,
             ragged=True, q_heads=32, kv_heads=8, dim=128, block=16, dtype="bf16", mask=False),
        # a decode batch behind one long document
        dict(name="shared_decode", op="shared", groups=1, requests=64, new=1, prefix=16384, cached=1024,
             ragged=True, q_heads=32, kv_heads=8, dim=128, block=16, dtype="bf16", mask=False),
        # verify windows of up to 8 drafted tokens in a tree behind three long prompts
        dict(name="shared_verify", op="shared", groups=3, requests=16, new=8, prefix=32768, cached=2048,
             ragged=True, q_heads=20, kv_heads=4, dim=128, block=32, dtype="bf16", mask=True),
        # users' turns taken up behind a system prompt, narrow heads, fp16, odd lengths
        dict(name="shared_chunks", op="shared", groups=2, requests=6, new=501, prefix=5003, cached=300,
             ragged=True, q_heads=16, kv_heads=16, dim=64, block=16, dtype="fp16", mask=False),
        # one verify window sampled
        dict(name="sample_window", op="sample", tokens=8, vocab=131072, dtype="bf16"),
        # a batch of windows, odd vocabulary (rows of no alignment), fp32 logits
        dict(name="sample_batch", op="sample", tokens=96, vocab=50257, dtype="fp32"),
        # a full server's step
        dict(name="sample_server", op="sample", tokens=512, vocab=131072, dtype="bf16"),
    ]


def _log_int(rng, lo: int, hi: int) -> int:
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng) -> dict:
    op = rng.choice(["rotary", "shared", "shared", "sample"])
    if op == "sample":
        vocab = _log_int(rng, 1000, 131072)
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        most = min(512, (1 << 26) // vocab) // (2 if dtype == "fp32" else 1)
        return dict(op="sample", tokens=_log_int(rng, 1, most), vocab=vocab, dtype=dtype)
    kv_heads = rng.choice([1, 2, 4, 8])
    q_heads = kv_heads * rng.choice([1, 2, 4, 5])
    dim = rng.choice([64, 128])
    if op == "rotary":
        return dict(op="rotary", tokens=_log_int(rng, 1, 8191), q_heads=min(q_heads, 32), kv_heads=kv_heads,
                    dim=dim, rotary=rng.choice([32, dim // 2, dim, dim]), axes=rng.choice([1, 1, 2, 3]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.6,
                    block=rng.choice([16, 32, 64]), dtype=rng.choice(["bf16", "fp16"]),
                    length=_log_int(rng, 64, 32768))
    kind = rng.choice(["decode", "decode", "verify", "chunk"])
    case = dict(op="shared", ragged=rng.random() < 0.7, q_heads=min(q_heads, 32), kv_heads=kv_heads, dim=dim,
                block=rng.choice([16, 32, 64]), dtype=rng.choice(["bf16", "fp16"]),
                mask=kind == "verify" and rng.random() < 0.5)
    case["new"] = 1 if kind == "decode" else rng.randint(2, 8) if kind == "verify" else _log_int(rng, 64, 512)
    case["requests"] = _log_int(rng, 1, 64 if kind == "decode" else 16 if kind == "verify" else 4)
    case["groups"] = rng.randint(1, min(4, case["requests"]))
    case["prefix"] = _log_int(rng, 16, 4096 if kind == "chunk" else 32768 // (1 + case["requests"] // 33))
    case["cached"] = _log_int(rng, 1, 1024)
    return case


def _lens(case: dict) -> dict:
    """The lengths of a shared case: part of the case, the same for every seed."""
    n, groups = case["requests"], case["groups"]
    r = np.random.RandomState(n * 7919 + case["new"] * 31 + case["cached"] + case["prefix"])
    cached, new = np.full(n, case["cached"]), np.full(n, case["new"])
    prefix = np.full(groups, case["prefix"])
    if case["ragged"]:
        cached, new = r.randint(0, case["cached"] + 1, n), r.randint(1, case["new"] + 1, n)
        prefix = r.randint(case["prefix"] // 2, case["prefix"] + 1, groups)
        prefix[0], new[r.randint(n)] = case["prefix"], case["new"]
    cuts = np.sort(r.choice(np.arange(1, n), groups - 1, replace=False)) if groups > 1 else []
    return dict(cached=cached, new=new, prefix=prefix, cu_groups=np.concatenate([[0], cuts, [n]]).astype(int))


def work(case: dict) -> dict:
    if case["op"] == "sample":
        return dict(bytes=case["tokens"] * (case["vocab"] * ITEM[case["dtype"]] + 28), flops=0)
    h, d = case["kv_heads"], case["dim"]
    if case["op"] == "rotary":
        t, item = case["tokens"], ITEM[case["dtype"]]
        held = 2 * h * (d // 2 + 4)
        # the rotated queries, and the keys and values read back, are written
        return dict(bytes=t * ((2 * case["q_heads"] + 4 * h) * d * item + 2 * held + 8 + 4 * case["axes"] +
                               4 * case["rotary"]), flops=0)
    n = _lens(case)
    cached, new, prefix = (n[k].astype(np.float64) for k in ("cached", "new", "prefix"))
    of = np.repeat(np.arange(case["groups"]), np.diff(n["cu_groups"]))
    pairs = float((new * (cached + prefix[of]) + new * (new + 1) / 2).sum())
    tokens = float(new.sum())
    held = 2 * h * (d // 2 + 4) * float((cached + new).sum() + prefix.sum())
    rows = 2 * ITEM[case["dtype"]] * tokens * case["q_heads"] * d + 4 * tokens * case["q_heads"]
    return dict(bytes=held + rows, flops=4.0 * pairs * case["q_heads"] * d)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _rand(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda")


def _int32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def _pages(gen, blocks: int, kv_heads: int, block: int, dim: int):
    """A cache pool as earlier steps left it."""
    codes = torch.empty(blocks, 2, kv_heads, block, dim // 2, dtype=torch.uint8, device="cuda")
    for i in range(0, blocks, 8192):
        n = min(8192, blocks - i)
        c = _randn(gen, n, 2, kv_heads, block, dim).mul_(2.8).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
        codes[i:i + n] = c[..., 0::2] | (c[..., 1::2] << 4)
    step = 0.36 * torch.exp(0.3 * _randn(gen, blocks, 2, kv_heads, block))
    low = -7.5 * step + 0.1 * _randn(gen, blocks, 2, kv_heads, block)
    return codes, torch.stack([step, low], dim=-1).to(torch.bfloat16)


def _cos_sin(length: int, rotary: int):
    """[length][2][rotary / 2] fp32, cosines first: the angles in 64 bits."""
    i = torch.arange(rotary // 2, dtype=torch.float64, device="cuda")
    angle = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2.0 * i / rotary)
    return torch.stack([angle.cos(), angle.sin()], dim=1).float().contiguous()


def _prepare_rotary(case: dict, seed: int) -> dict:
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t, h, hq, d, bs = case["tokens"], case["kv_heads"], case["q_heads"], case["dim"], case["block"]
    rot, axes, length, dt = case["rotary"], case["axes"], case["length"], DTYPES[case["dtype"]]
    # queries, keys and values are slices of the fused projection's rows
    qkv = _randn(gen, t, (hq + 2 * h) * d) * 1.5
    qkv[:, hq * d:(hq + h) * d] += _randn(gen, h * d)      # keys have an offset by channel
    qkv = qkv.to(dt)
    norms = [(1 + 0.1 * _randn(gen, d)).to(dt) if case["norm"] else None for _ in range(2)]
    at = torch.arange(t, device="cuda")
    start = int(torch.randint(0, max(1, length - t + 1), (1,), generator=gen, device="cuda"))
    if axes == 1:
        positions = ((start + at) % length)[None]
        axis_of = None
    else:
        # frames of 16 x 16 patches; frequencies dealt to the axes in runs
        place = [at // 256, at // 16 % 16, at % 16][:axes]
        positions = torch.stack([(start + p) % length for p in place])
        axis_of = (torch.arange(rot // 2, device="cuda") * axes // (rot // 2)).to(torch.int32)
    blocks = -(-t // bs) + 8
    codes, scales = _pages(gen, blocks, h, bs, d)
    pages = torch.randperm(blocks, generator=gen, device="cuda")[: -(-t // bs)]
    return dict(q=qkv[:, : hq * d].view(t, hq, d), k=qkv[:, hq * d:(hq + h) * d].view(t, h, d),
                v=qkv[:, (hq + h) * d:].view(t, h, d), q_norm=norms[0], k_norm=norms[1],
                positions=positions.to(torch.int32).contiguous(), axis_of=axis_of,
                cos_sin=_cos_sin(length, rot), interleaved=case["interleaved"],
                slots=pages[at // bs] * bs + at % bs, codes=codes, scales=scales,
                q_out=torch.empty(t, hq, d, dtype=dt, device="cuda"),
                k_out=torch.empty(t, h, d, dtype=dt, device="cuda"),
                v_out=torch.empty(t, h, d, dtype=dt, device="cuda"))


def _prepare_shared(case: dict, seed: int) -> dict:
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens = _lens(case)
    n, groups, bs = case["requests"], case["groups"], case["block"]
    d, h, hq = case["dim"], case["kv_heads"], case["q_heads"]
    new, kv, prefix, cu_groups = lens["new"], lens["cached"] + lens["new"], lens["prefix"], lens["cu_groups"]
    tokens = int(new.sum())
    have, have_p = -(-kv // bs), -(-prefix // bs)
    blocks = int(have.sum() + have_p.sum()) + 4
    codes, scales = _pages(gen, blocks, h, bs, d)
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)

    def table(count, ids):
        held = torch.from_numpy(np.arange(int(count.max()))[None, :] < count[:, None]).cuda()
        t = torch.full(held.shape, -1, dtype=torch.int32, device="cuda")
        t[held] = ids[: int(count.sum())]
        return t

    block_table, prefix_table = table(have, order), table(have_p, order[int(have.sum()):])
    # what lies behind an end in the last block was never written
    for t, count, length in ((block_table, have, kv), (prefix_table, have_p, prefix)):
        last = t[torch.arange(len(count), device="cuda"), torch.from_numpy(count - 1).cuda()].long()
        end = torch.from_numpy(count * bs - length).cuda()
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
    return dict(q=qkv[:, : hq * d].view(tokens, hq, d), codes=codes, scales=scales,
                prefix_table=prefix_table, prefix_lens=_int32(prefix), cu_groups=_int32(cu_groups),
                max_shared=int(np.diff(cu[cu_groups]).max()), table=block_table, cu=_int32(cu), kv=_int32(kv),
                max_new=int(new.max()), max_kv=int(kv.max()), max_prefix=int(prefix.max()), mask=mask,
                scale=1.0 / math.sqrt(d), out=torch.empty(tokens, hq, d, dtype=qkv.dtype, device="cuda"),
                lse=torch.empty(tokens, hq, dtype=torch.float32, device="cuda"),
                workspace=torch.empty(tokens * hq * (d + 2), dtype=torch.float32, device="cuda"))


def _prepare_sample(case: dict, seed: int) -> dict:
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t, v = case["tokens"], case["vocab"]
    logits = torch.empty(t, v, dtype=DTYPES[case["dtype"]], device="cuda")
    for i in range(0, t, 512):
        x = _randn(gen, min(512, t - i), v).mul_(2.5)
        x[:, ::997] += 6.0                                   # a few likely tokens
        logits[i:i + 512] = x
    logits[:, 7 % v] = float("-inf")                         # a token the sampler forbids
    pick = lambda values, dtype: torch.tensor(values, dtype=dtype, device="cuda")[  # noqa: E731
        torch.randint(0, len(values), (t,), generator=gen, device="cuda")]
    # each request's own settings; 0 and 1 switch a filter off, temperature 0 takes the largest
    return dict(logits=logits, uniform=_rand(gen, t),
                temperature=pick([0.0, 0.6, 0.7, 0.8, 1.0, 1.0, 1.2], torch.float32),
                top_k=pick([0, 0, 20, 50, 200, 1000], torch.int32),
                top_p=pick([0.5, 0.8, 0.9, 0.95, 1.0], torch.float32),
                min_p=pick([0.0, 0.0, 0.01, 0.05], torch.float32),
                tokens=torch.empty(t, dtype=torch.int32, device="cuda"),
                logprobs=torch.empty(t, dtype=torch.float32, device="cuda"))


def prepare(case: dict, seed: int) -> dict:
    made = dict(rotary=_prepare_rotary, shared=_prepare_shared, sample=_prepare_sample)[case["op"]](case, seed)
    made["op"] = case["op"]
    return made


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _bf16_floor(x):
    bits = x.view(torch.int32)
    cut = bits & -65536
    return torch.where((x < 0) & (cut != bits), cut + 65536, cut).view(torch.float32)


def _bf16_ceil(x):
    return -_bf16_floor(-x)


def _plain_round(x):
    """Codes, step and minimum of each row of the last axis."""
    low, high = x.amin(-1), x.amax(-1)
    m = _bf16_floor(low)
    s = _bf16_ceil((high - m) * (1.0 / 15.0))
    s = torch.where((s > 0) & (s < 2.0 ** -126), 2.0 ** -126, s)
    r = torch.where(s > 0, torch.ones_like(s) / s, 0.0)
    code = ((x - m[..., None]) * r[..., None]).round().clamp(0, 15)
    return code.to(torch.uint8), s, m


def _plain_values(codes, scales):
    c = torch.stack([(codes & 15).float(), (codes >> 4).float()], dim=-1).flatten(-2)
    return scales[..., 1:].float() + scales[..., :1].float() * c


def _plain_normed(x, weight):
    """Each step of it one fp32 operation; squares are added to their neighbours, these sums
    to theirs, and so on."""
    x = x.float()
    if weight is None:
        return x
    y = x * x
    while y.shape[-1] > 1:
        y = y[..., 0::2] + y[..., 1::2]
    return x * (1.0 / torch.sqrt(y / x.shape[-1] + EPS)) * weight.float()


def _plain_rotated(x, c, s, interleaved):
    rot = 2 * c.shape[-1]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_rotary(s: dict) -> dict:
    codes, scales, bs = s["codes"], s["scales"], s["codes"].shape[3]
    pos, half = s["positions"].long(), s["cos_sin"].shape[2]
    if s["axis_of"] is None:
        row = pos[0][:, None].expand(-1, half)
    else:
        row = pos[s["axis_of"].long()].t()                             # [tokens][half]
    i = torch.arange(half, device=pos.device)
    c, sn = s["cos_sin"][row, 0, i][:, None], s["cos_sin"][row, 1, i][:, None]
    q = _plain_rotated(_plain_normed(s["q"], s["q_norm"]), c, sn, s["interleaved"])
    k = _plain_rotated(_plain_normed(s["k"], s["k_norm"]), c, sn, s["interleaved"])
    blk, off = s["slots"] // bs, s["slots"] % bs
    ck, sk, mk = _plain_round(k)
    cv, sv, mv = _plain_round(s["v"].float())
    code = torch.stack([ck, cv], dim=1)
    codes[blk, :, :, off] = code[..., 0::2] | (code[..., 1::2] << 4)
    scales[blk, :, :, off] = torch.stack([torch.stack([sk, mk], -1), torch.stack([sv, mv], -1)],
                                         dim=1).to(torch.bfloat16)
    # what the slots stand for
    kv = _plain_values(codes[blk, :, :, off], scales[blk, :, :, off]).to(s["k"].dtype)
    return dict(q=q.to(s["q"].dtype), k=kv[:, 0], v=kv[:, 1])


def _plain_keys(s: dict, table, lens, most: int):
    """Keys and values [n][kv heads][most][dim] of a table's rows; 0 behind their ends."""
    codes, scales, bs = s["codes"], s["scales"], s["codes"].shape[3]
    j = torch.arange(most, device=table.device)
    held = j < lens[:, None]
    blk = torch.where(held, table.long()[:, j // bs], 0)
    off = (j % bs).expand_as(blk)
    return [_plain_values(codes[blk, kv, :, off],
                          torch.where(held[:, :, None, None], scales[blk, kv, :, off], 0)).transpose(1, 2)
            for kv in range(2)]


def _plain_shared(s: dict) -> dict:
    q, cu, kv, prefix, cg = s["q"], s["cu"].long(), s["kv"].long(), s["prefix_lens"].long(), s["cu_groups"].long()
    tokens, hq, d = q.shape
    h = s["codes"].shape[2]
    n, groups, g, w, ws = kv.shape[0], prefix.shape[0], hq // h, s["max_new"], s["max_shared"]
    t = torch.arange(tokens, device=q.device)
    rows = q.float().view(tokens, h, g, d)

    def against(starts, count, k, v, hidden):
        """Softmax sums of rows [starts[b], starts[b] + count) against keys b: the largest
        logit, the sum and the weighted values of every row, [n][h][g][count]."""
        here = (starts[:, None] + torch.arange(count, device=q.device)).clamp(max=tokens - 1)
        x = rows[here].permute(0, 2, 3, 1, 4).reshape(len(starts), h, g * count, d)
        a = torch.matmul(x, k.transpose(2, 3)).mul_(s["scale"]).view(len(starts), h, g, count, -1)
        a.masked_fill_(hidden, float("-inf"))
        top = a.amax(-1)
        a.sub_(torch.where(torch.isinf(top), 0.0, top)[..., None]).exp_()
        o = torch.matmul(a.view(len(starts), h, g * count, -1), v).view(len(starts), h, g, count, d)
        return top, a.sum(-1), o

    # the prefixes, once a group
    first = cu[cg[:-1]]
    of_g = torch.searchsorted(cu[cg[1:]], t, right=True)
    k, v = _plain_keys(s, s["prefix_table"], prefix, s["max_prefix"])
    j = torch.arange(s["max_prefix"], device=q.device)
    one = against(first, ws, k, v, (j >= prefix[:, None])[:, None, None, None, :])
    one = [x[of_g, :, :, t - first[of_g]] for x in one]
    # each request's own tokens
    k, v = _plain_keys(s, s["table"], kv, s["max_kv"])
    j = torch.arange(s["max_kv"], device=q.device)
    i = torch.arange(w, device=q.device)
    behind = (kv - (cu[1:] - cu[:-1]))[:, None, None]
    if s["mask"] is None:
        sees = j <= behind + i[:, None]
    else:
        here = (cu[:-1, None] + i).clamp(max=tokens - 1)
        bit = (s["mask"][here][:, :, None] >> (j - behind).clamp(0, 63)) & 1
        sees = (j < behind) | (bit == 1)
    of = torch.searchsorted(cu[1:], t, right=True)
    two = against(cu[:-1], w, k, v, ~(sees & (j < kv[:, None])[:, None, :])[:, None, None])
    two = [x[of, :, :, t - cu[of]] for x in two]
    top = torch.maximum(one[0], two[0])
    by = [torch.exp(x[0] - torch.where(torch.isinf(top), 0.0, top)) for x in (one, two)]
    total = one[1] * by[0] + two[1] * by[1]
    out = (one[2] * by[0][..., None] + two[2] * by[1][..., None]) / torch.where(total > 0, total, 1.0)[..., None]
    return dict(out=out.reshape(tokens, hq, d).to(q.dtype), lse=(total.log() + top).reshape(tokens, hq))


def _plain_sample(s: dict) -> dict:
    """Sorted once; the weights and their sums in 64 bits, where a token's border is as near
    to the drawn number as it happens to be."""
    x, ids = s["logits"].float().sort(dim=-1, descending=True, stable=True)
    v = x.shape[1]
    hot = s["temperature"] > 0
    wide = x.double()
    w = ((wide - wide[:, :1]) / torch.where(hot, s["temperature"], 1.0).double()[:, None]).exp()
    at = torch.arange(v, device=x.device)
    k = torch.where((s["top_k"] > 0) & (s["top_k"] < v), s["top_k"], v)[:, None]
    w = torch.where(at < torch.where(hot[:, None], k, 1), w, 0.0)
    upto = w.cumsum(-1)
    p = s["top_p"].double()[:, None]
    within = (upto - w < p * upto[:, -1:]) | (p >= 1) | (at == 0)
    w = torch.where(within & (w >= s["min_p"].double()[:, None].clamp(max=1)), w, 0.0)
    by_id = torch.zeros_like(w).scatter_(1, ids, w)
    upto = by_id.cumsum(-1)
    total = upto[:, -1:]
    passed = (upto > s["uniform"].double()[:, None] * total) & (by_id > 0)
    token = passed.int().argmax(-1)
    mine = by_id.gather(1, token[:, None])
    return dict(tokens=token.int(), logprobs=(mine / total).log()[:, 0].float())


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


def _own_rotary(s: dict) -> dict:
    hc = _library()
    hc.hc_kv4_append_rotary(s["q"], s["k"], s["v"], s["cos_sin"], s["positions"], s["slots"], s["codes"],
                            s["scales"], s["q_out"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS,
                            axis_of=s["axis_of"], interleaved=s["interleaved"])
    hc.hc_kv4_load(s["slots"], s["codes"], s["scales"], s["k_out"], s["v_out"])
    return dict(q=s["q_out"], k=s["k_out"], v=s["v_out"])


def _own_shared(s: dict) -> dict:
    _library().hc_kv4_attention_shared(s["q"], s["codes"], s["scales"], s["prefix_table"], s["prefix_lens"],
                                       s["cu_groups"], s["max_shared"], s["table"], s["cu"], s["kv"],
                                       s["max_new"], s["workspace"], s["out"], lse=s["lse"], mask=s["mask"],
                                       scale=s["scale"])
    return dict(out=s["out"], lse=s["lse"])


def _own_sample(s: dict) -> dict:
    _library().hc_sample_tokens(s["logits"], s["uniform"], s["tokens"], s["logprobs"],
                                temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                min_p=s["min_p"])
    return dict(tokens=s["tokens"], logprobs=s["logprobs"])


_PLAIN = dict(rotary=_plain_rotary, shared=_plain_shared, sample=_plain_sample)
_OWN = dict(rotary=_own_rotary, shared=_own_shared, sample=_own_sample)


def run(state: dict) -> dict:
    return (_OWN if own else _PLAIN)[state["op"]](state)


# ---------------------------------------------------------------------------
# in 64 bits
# ---------------------------------------------------------------------------

def _exact_rotary(s: dict) -> dict:
    """The queries in 64 bits. What the cache holds of a key follows from single fp32
    operations by definition, so that its codes are the same everywhere: they are numpy's."""
    f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    pos, table = s["positions"].cpu().numpy(), f(s["cos_sin"])
    half = table.shape[2]
    axis = np.zeros(half, int) if s["axis_of"] is None else s["axis_of"].cpu().numpy()
    row = pos[axis].T                                                  # [tokens][half]
    c, sn = (table[row, i, np.arange(half)][:, None] for i in range(2))
    first = np.arange(half) * 2 if s["interleaved"] else np.arange(half)
    second = first + (1 if s["interleaved"] else half)

    def turn(x, c, sn):
        y = x.copy()
        y[..., first] = x[..., first] * c - x[..., second] * sn
        y[..., second] = x[..., second] * c + x[..., first] * sn
        return y

    q, k, v = f(s["q"]), f(s["k"]).astype(np.float32), f(s["v"]).astype(np.float32)
    if s["q_norm"] is not None:
        q = q / np.sqrt((q * q).mean(-1, keepdims=True) + EPS) * f(s["q_norm"])
        d, total = k.shape[-1], k * k
        for n in range(int(math.log2(d))):
            total = total.reshape(*k.shape[:-1], d >> (n + 1), 2).sum(-1)
        mean = total * np.float32(1 / d) + np.float32(EPS)
        k = k * (np.float32(1) / np.sqrt(mean)) * f(s["k_norm"]).astype(np.float32)
    k = turn(k, c.astype(np.float32), sn.astype(np.float32))
    out = dict(q=turn(q, c, sn))
    f32 = lambda a: a.astype(np.float32).astype(np.float64)  # noqa: E731

    def bf16(a, towards):
        frac, e = np.frexp(a)
        unit = np.exp2(np.maximum(e, -125).astype(np.float64) - 8)
        return towards(a / unit) * unit

    for name, x in (("k", k.astype(np.float64)), ("v", v.astype(np.float64))):
        low, high = x.min(-1), x.max(-1)
        m = bf16(low, np.floor)
        step = bf16(f32(f32(high - m) * np.float64(np.float32(1.0 / 15.0))), np.ceil)
        step = np.where((step > 0) & (step < 2.0 ** -126), 2.0 ** -126, step)
        r = np.where(step > 0, f32(1.0 / np.where(step > 0, step, 1.0)), 0.0)
        code = np.clip(np.rint(f32(f32(x - m[..., None]) * r[..., None])), 0, 15)
        out[name] = m[..., None] + step[..., None] * code
    return out


def _exact_shared(s: dict) -> dict:
    """Request by request and head by head, a prefix and the request's own tokens as one
    sequence."""
    tokens, hq, d = s["q"].shape
    h, bs = s["codes"].shape[2], s["codes"].shape[3]
    g = hq // h
    out = torch.zeros(tokens, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((tokens, hq), float("-inf"), dtype=torch.float64, device="cuda")
    cu, kv, cg, lens = (s[k].tolist() for k in ("cu", "kv", "cu_groups", "prefix_lens"))

    def values(pages, length):
        pages = pages[: -(-length // bs)].long()
        held = s["codes"][pages].permute(1, 2, 0, 3, 4).reshape(2, h, -1, d // 2)[:, :, :length]
        sm = s["scales"][pages].permute(1, 2, 0, 3, 4).reshape(2, h, -1, 2)[:, :, :length].double()
        c = torch.empty(2, h, length, d, dtype=torch.float64, device="cuda")
        c[..., 0::2], c[..., 1::2] = held.bitwise_and(15).double(), held.bitwise_right_shift(4).double()
        return c * sm[..., 0:1] + sm[..., 1:2]

    for group, before in enumerate(lens):
        common = values(s["prefix_table"][group], before)
        for b in range(cg[group], cg[group + 1]):
            a0, a1 = cu[b], cu[b + 1]
            c = torch.cat([common, values(s["table"][b], kv[b])], dim=2)
            back = torch.arange(c.shape[2], device="cuda") - (before + kv[b] - (a1 - a0))
            at = torch.arange(a1 - a0, device="cuda")
            if s["mask"] is None:
                hidden = back[None, :] > at[:, None]
            else:
                set_ = torch.bitwise_and(s["mask"][a0:a1, None], torch.ones_like(back) << back.clamp(0, 62)) != 0
                hidden = (back >= 0)[None, :] & ~set_
            for head in range(hq):
                z = s["q"][a0:a1, head].double() @ c[0, head // g].T * s["scale"]
                z = z.masked_fill(hidden, float("-inf"))
                lse[a0:a1, head] = torch.logsumexp(z, -1)
                out[a0:a1, head] = torch.exp(z - lse[a0:a1, head, None]).nan_to_num(0.0) @ c[1, head // g]
    return dict(out=out, lse=lse)


def _exact_sample(s: dict) -> dict:
    """Row by row. Tokens are whole numbers, which the plain form gives; here they only say
    whose probability it is."""
    logprobs = []
    settings = [s[k].tolist() for k in ("uniform", "temperature", "top_k", "top_p", "min_p")]
    for x, u, t, k, p, least in zip(s["logits"], *settings):
        x = x.double()
        if t <= 0:
            logprobs.append(0.0)
            continue
        w = torch.exp((x - x.max()) / t)
        order = torch.argsort(x, descending=True, stable=True)
        if 0 < k < len(order):
            order = order[:k]
        if p < 1:
            mass = w[order].cumsum(0)
            order = order[: 1 + int((mass[:-1] < p * mass[-1]).sum())]
        order = order[w[order] >= min(least, 1.0)].sort().values
        mass = w[order].cumsum(0)
        i = int((mass <= u * mass[-1]).sum())
        logprobs.append(math.log(float(w[order[min(i, len(order) - 1)]] / mass[-1])))
    return dict(tokens=None, logprobs=torch.tensor(logprobs, dtype=torch.float64, device="cuda"))


def exact(case: dict, seed: int):
    """None where 64 bits would take too long."""
    if case["op"] == "shared" and work(case)["flops"] > 4e11:
        return None
    s = prepare(case, seed)
    return dict(rotary=_exact_rotary, shared=_exact_shared, sample=_exact_sample)[case["op"]](s)
