"""Measured cases of the four-bit serving path's operators.

The path: a projection's queries and keys are normalised per head and rotated by their positions
(``qk_norm_rope``); a prompt attends over its own fresh keys and values, or over its cached context
and them (``prompt_attention``); keys and values are stored in a paged cache that holds four bits
per value (``reshape_and_cache_int4``), read back as fp16 rows where a later chunk of the prompt
needs them (``gather_cache_int4``), and single tokens attend over that cache
(``paged_attention_decode_int4``).

A case is a dict of plain values; ``run`` computes its operator in plain torch operations, or with
``own`` through the package's binding.  A row of D values held in four bits is D/2 bytes (value 2j
in the low half of byte j, 2j + 1 in the high half), with an fp16 scale and an fp16 zero point: it
stands for zero + scale * n.  A cache is uint8 [blocks, heads, B * (D/2 + 4)]: the B rows of a
(block, head), then their B (scale, zero) pairs.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one decode step of a 64-sequence batch, ordinary positions: latency counts
        {"name": "rope_decode_64", "op": "rope", "tokens": 64, "heads": 40, "kv_heads": 40, "head_dim": 128,
         "rotary_dim": 128, "axes": 1, "interleaved": False, "norm": True, "max_pos": 2048},
        # a prompt batch of image and video tokens: three position axes, grouped heads, far positions
        {"name": "rope_prompt_axes", "op": "rope", "tokens": 32768, "heads": 40, "kv_heads": 8, "head_dim": 128,
         "rotary_dim": 128, "axes": 3, "interleaved": False, "norm": True, "max_pos": 1000000},
        # one decode step's new keys and values into the four-bit cache, and the rows read back
        {"name": "write_decode_64", "op": "write", "tokens": 64, "heads": 40, "head_dim": 128, "block_size": 16},
        # a prompt batch's keys and values into the cache, and the rows read back
        {"name": "write_prompt", "op": "write", "tokens": 16411, "heads": 40, "head_dim": 128, "block_size": 16},
        # the 1024-token cached prefix of one request, as the next chunk of its prompt needs it
        {"name": "gather_prefix", "op": "gather", "seqs": 1, "lo": 1024, "hi": 1024, "lens": 1, "heads": 40,
         "head_dim": 128, "block_size": 16},
        # the cached contexts of a batch of long prompts of ragged lengths, grouped heads
        {"name": "gather_long", "op": "gather", "seqs": 16, "lo": 2048, "hi": 16384, "lens": 2, "heads": 8,
         "head_dim": 128, "block_size": 32},
        # one 2048-token sequence: the smallest decode step
        {"name": "decode_one", "op": "decode", "seqs": 1, "lo": 2048, "hi": 2048, "lens": 3, "heads": 40,
         "kv_heads": 40, "head_dim": 128, "block_size": 16},
        # the 64-sequence batch of contexts from 128 to 2048
        {"name": "decode_batch", "op": "decode", "seqs": 64, "lo": 128, "hi": 2048, "lens": 4, "heads": 40,
         "kv_heads": 40, "head_dim": 128, "block_size": 16},
        # long ragged contexts, eight query heads to a cached head
        {"name": "decode_long_grouped", "op": "decode", "seqs": 32, "lo": 8192, "hi": 32768, "lens": 5, "heads": 64,
         "kv_heads": 8, "head_dim": 128, "block_size": 32},
        # a batch of short prompts of ragged lengths, packed
        {"name": "prompt_short", "op": "prompt", "seqs": 32, "lo": 1, "hi": 512, "lens": 6, "cached": 0, "heads": 40,
         "kv_heads": 40, "head_dim": 128},
        # new chunks over a 1024-token cached context, grouped heads
        {"name": "prompt_chunk", "op": "prompt", "seqs": 16, "lo": 32, "hi": 512, "lens": 7, "cached": 1024,
         "heads": 32, "kv_heads": 8, "head_dim": 64},
        # eight long prompts, five query heads to a key head
        {"name": "prompt_long", "op": "prompt", "seqs": 8, "lo": 4096, "hi": 4096, "lens": 8, "cached": 0, "heads": 40,
         "kv_heads": 8, "head_dim": 128},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "write", "gather", "decode", "prompt"])
    head_dim = rng.choice([64, 128, 128])
    block_size = rng.choice([4, 8, 16, 16, 32])
    kv_heads = rng.choice([1, 2, 5, 8, 12, 40])
    if op == "rope":
        rotary = rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4])
        return {"op": op, "tokens": spread(1, 16384), "heads": kv_heads * rng.choice([1, 2, 4]), "kv_heads": kv_heads,
                "head_dim": head_dim, "rotary_dim": rotary, "axes": rng.choice([1, 2, 3]),
                "interleaved": rng.random() < 0.3, "norm": rng.random() < 0.8, "max_pos": spread(64, 1000000)}
    if op == "write":
        return {"op": op, "tokens": spread(1, 12000), "heads": kv_heads, "head_dim": head_dim, "block_size": block_size}
    lens = rng.randrange(1 << 20)
    if op == "gather":
        hi = spread(1, 4096)
        return {"op": op, "seqs": spread(1, 24), "lo": max(1, hi // 8), "hi": hi, "lens": lens, "heads": kv_heads,
                "head_dim": head_dim, "block_size": block_size}
    group = rng.choice([1, 1, 2, 3, 4, 7, 8, 16]) if kv_heads < 40 else 1
    if op == "decode":
        hi = spread(1, 32768)
        most = max(1, min(200, (1 << 20) // (hi * kv_heads) * 8))
        return {"op": op, "seqs": spread(1, most), "lo": rng.choice([0, hi // 8, hi // 2]), "hi": hi, "lens": lens,
                "heads": kv_heads * group, "kv_heads": kv_heads, "head_dim": head_dim, "block_size": block_size}
    group = min(group, max(1, 40 // kv_heads))
    hi = spread(1, 2500)
    most = max(1, min(64, (8 * 4096 * 4096 // 4) // (hi * hi)))
    return {"op": op, "seqs": spread(1, most), "lo": max(1, hi // rng.choice([1, 8, 64])), "hi": hi, "lens": lens,
            "cached": rng.choice([0, 0, spread(1, 1000)]), "heads": kv_heads * group, "kv_heads": kv_heads,
            "head_dim": head_dim}


def lengths(case):
    """The case's sequence lengths, the longest among them at a place of its own."""
    r = random.Random(case["lens"])
    got = [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    got[r.randrange(len(got))] = case["hi"]
    return got


def starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


def axis_of_pair(case):
    """Which position axis turns each of the rotary_dim / 2 pairs: a quarter of them time, the rest halved."""
    pairs, axes = case["rotary_dim"] // 2, case["axes"]
    first = pairs if axes == 1 else pairs // 2 if axes == 2 else pairs // 4
    second = pairs - first if axes == 2 else (pairs - first) // 2
    return np.minimum(np.repeat([0, 1, 2], [first, second, pairs - first - second]), axes - 1).astype(np.int32)


# ---- what a program has in hand ---------------------------------------------------------------

def gauss(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float16)


def quantised(x):
    """(n, scale, zero) of rows x [..., D]: zero the least value, scale = (greatest - least) / 15 in
    32 bits rounded to fp16, n the nearest whole number to (x - zero) / scale, halves to even."""
    x = x.float()
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = ((hi - lo) / 15).half()
    n = ((x - lo).double() / scale.double()).round().clamp_(0, 15)
    n = torch.where(scale > 0, n, torch.zeros_like(n)).to(torch.uint8)
    return n, scale.squeeze(-1), lo.half().squeeze(-1)


def packed(x):
    """A four-bit cache of rows x [N, H, B, D]."""
    N, H, B, D = x.shape
    n, scale, zero = quantised(x)
    pool = torch.empty(N, H, B * (D // 2 + 4), dtype=torch.uint8, device=x.device)
    pool[:, :, :B * D // 2] = (n[..., 0::2] | (n[..., 1::2] << 4)).reshape(N, H, -1)
    pool[:, :, B * D // 2:] = torch.stack([scale, zero], -1).view(torch.uint8).reshape(N, H, -1)
    return pool


def paged(case, g, lens):
    """Two caches with the sequences' blocks in random places, and their tables.  Slots past a
    sequence's end hold scales and zero points that are not numbers."""
    H, D, B = case.get("kv_heads", case["heads"]), case["head_dim"], case["block_size"]
    blocks = [-(-n // B) for n in lens]
    N = sum(blocks) + 5
    order = torch.randperm(N, generator=g, device=DEV).to(torch.int32)
    most = max(1, max(blocks))
    col = torch.arange(most, device=DEV)
    count = torch.tensor(blocks, device=DEV)
    first = torch.tensor(starts(blocks)[:-1], device=DEV)
    have = col[None] < count[:, None]
    tables = torch.where(have, order[(first[:, None] + col[None]).clamp(max=N - 1)], -1).to(torch.int32)
    ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
    caches = []
    at = torch.arange(most * B, device=DEV)
    past = (at[None] >= ctx[:, None]) & have.repeat_interleave(B, 1)
    blk = tables.long().repeat_interleave(B, 1)[past]
    row = (at % B)[None].expand(len(lens), -1)[past]
    for _ in range(2):
        pool = torch.cat([packed(gauss(g, min(2048, N - i), H, B, D)) for i in range(0, N, 2048)])
        meta = pool[:, :, B * D // 2:].view(torch.float16).view(N, H, B, 2)
        meta[blk, :, row] = float("nan")
        caches.append(pool)
    return caches, tables, ctx


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    op, D = case["op"], case["head_dim"]
    if op == "rope":
        T, H, Hk, A = case["tokens"], case["heads"], case["kv_heads"], case["axes"]
        # the projection's output: queries, keys and values of a token side by side
        qkv = gauss(g, T, H + 2 * Hk, D)
        s["q"], s["key"] = qkv[:, :H], qkv[:, H:H + Hk]
        s["q_weight"] = (1 + 0.2 * gauss(g, D)) if case["norm"] else None
        s["k_weight"] = (1 + 0.2 * gauss(g, D)) if case["norm"] else None
        s["positions"] = torch.randint(0, case["max_pos"], (A, T), generator=g, device=DEV, dtype=torch.int32)
        s["positions"][1:] %= 1024
        pairs = case["rotary_dim"] // 2
        inv = 10000.0 ** (-np.arange(pairs) / pairs)
        s["inv_freq"] = torch.tensor(inv, dtype=torch.float64, device=DEV)
        # the same as parts of a turn per position, in units of 2^-64 turns
        s["frequencies"] = torch.tensor([int(f / (2 * math.pi) * 2.0 ** 64) for f in inv], dtype=torch.int64, device=DEV)
        s["pair_axis"] = torch.tensor(axis_of_pair(case), device=DEV)
    elif op == "write":
        T, H, B = case["tokens"], case["heads"], case["block_size"]
        kv = gauss(g, T, 2 * H, D)
        s["key"], s["value"] = kv[:, :H], kv[:, H:]
        N = -(-T // B) + 9
        s["k_cache"] = torch.zeros(N, H, B * (D // 2 + 4), dtype=torch.uint8, device=DEV)
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        t = torch.arange(T, device=DEV)
        s["slots"] = torch.randperm(N, generator=g, device=DEV)[t // B] * B + t % B
    elif op in ("gather", "decode"):
        lens = lengths(case)
        (s["k_cache"], s["v_cache"]), s["tables"], s["ctx"] = paged(case, g, lens)
        B = case["block_size"]
        if op == "gather":
            seq = torch.tensor(np.repeat(np.arange(len(lens)), lens), device=DEV)
            t = torch.tensor(np.concatenate([np.arange(n) for n in lens]), device=DEV)
            s["slots"] = s["tables"][seq, t // B].long() * B + t % B
        else:
            s["q"] = gauss(g, len(lens), case["heads"], D)
    else:
        lens = lengths(case)
        H, Hk, past = case["heads"], case["kv_heads"], case["cached"]
        s["q"] = gauss(g, sum(lens), H, D)
        kv = gauss(g, sum(lens) + past * len(lens), 2 * Hk, D)
        s["key"], s["value"] = kv[:, :Hk], kv[:, Hk:]
        s["query_start"] = torch.tensor(starts(lens), dtype=torch.int32, device=DEV)
        s["key_start"] = torch.tensor(starts([n + past for n in lens]), dtype=torch.int32, device=DEV)
        s["max_len"] = max(lens)
    s["scale"] = 1 / math.sqrt(D)
    return s


# ---- the plain forms ------------------------------------------------------------------------------

def rotated(x, weight, cos, sin, interleaved):
    """x [T, H, D] normalised per head (where it has a weight) and its first 2 * pairs values turned."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
    R = 2 * cos.shape[-1]
    turned, rest = x[..., :R], x[..., R:]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :R // 2], turned[..., R // 2:])
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)
    return torch.cat([turned, rest], -1).half()


def plain_rope(s):
    at = s["positions"][s["pair_axis"].long()].double()                   # [pairs, T]
    angle = (at * s["inv_freq"][:, None]).T[:, None]                        # [T, 1, pairs]
    cos, sin = angle.cos().float(), angle.sin().float()
    inter = s["case"]["interleaved"]
    return rotated(s["q"], s["q_weight"], cos, sin, inter), rotated(s["key"], s["k_weight"], cos, sin, inter)


def plain_store(pool, x, slots, B):
    T, H, D = x.shape
    n, scale, zero = quantised(x)
    blk, row = slots // B, slots % B
    N = pool.shape[0]
    pool[:, :, :B * D // 2].view(N, H, B, D // 2)[blk, :, row] = n[..., 0::2] | (n[..., 1::2] << 4)
    pool[:, :, B * D // 2:].view(torch.float16).view(N, H, B, 2)[blk, :, row] = torch.stack([scale, zero], -1)


def plain_rows(pool, blk, row, B):
    """The rows (blk, row) of a cache in 32 bits: [..., H, D]."""
    N, H, tile = pool.shape
    D = (tile // B - 4) * 2
    b = pool[:, :, :B * D // 2].view(N, H, B, D // 2)[blk, :, row]
    meta = pool[:, :, B * D // 2:].view(torch.float16).view(N, H, B, 2)[blk, :, row].float()
    n = torch.stack([b & 15, b >> 4], -1).flatten(-2).float()
    return meta[..., 1:] + meta[..., :1] * n


def softmax_of(x, live):
    """Softmax over the last axis of the live places; a row without any is zeros."""
    x = torch.where(live, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = (x - torch.where(m == -math.inf, 0.0, m)).exp()
    return e / e.sum(-1, keepdim=True).clamp(min=1e-30)


def plain_decode(s):
    c, q, ctx, tables = s["case"], s["q"].float(), s["ctx"], s["tables"]
    B, Hk = c["block_size"], c["kv_heads"]
    S, H, D = q.shape
    t = torch.arange(tables.shape[1] * B, device=q.device)
    live = t[None] < ctx[:, None]                                           # [S, L]
    blk, row = tables.long()[:, t // B].clamp(min=0), (t % B).expand(S, -1)
    k = plain_rows(s["k_cache"], blk, row, B).permute(0, 2, 3, 1)          # [S, Hk, D, L]
    x = q.view(S, Hk, H // Hk, D) @ k * s["scale"]
    p = softmax_of(x, live[:, None, None])
    del k, x
    v = plain_rows(s["v_cache"], blk, row, B).permute(0, 2, 1, 3)          # [S, Hk, L, D]
    v = torch.where(live[:, None, :, None], v, 0.0)
    return (p @ v).reshape(S, H, D).half()


def padded(x, start, L):
    """Rows start[s] .. start[s + 1] of x [T, H, D] as [S, L, H, D] in 32 bits, and which places hold one."""
    n = start[1:] - start[:-1]
    i = torch.arange(L, device=x.device)
    live = i[None] < n[:, None]
    at = (start[:-1, None] + i[None]).clamp(max=x.shape[0] - 1).long()
    return torch.where(live[..., None, None], x[at].float(), 0.0), live


def plain_prompt(s):
    c = s["case"]
    H, Hk, L, Lk = c["heads"], c["kv_heads"], s["max_len"], s["max_len"] + c["cached"]
    q, live = padded(s["q"], s["query_start"], L)
    k, _ = padded(s["key"], s["key_start"], Lk)
    v, _ = padded(s["value"], s["key_start"], Lk)
    S, D = q.shape[0], q.shape[-1]
    q = q.view(S, L, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).reshape(S, Hk, -1, D)
    x = (q @ k.permute(0, 2, 3, 1)).view(S, Hk, H // Hk, L, Lk) * s["scale"]
    seen = torch.arange(Lk, device=q.device)[None] <= torch.arange(L, device=q.device)[:, None] + c["cached"]
    p = softmax_of(x, seen).view(S, Hk, -1, Lk)
    del x
    o = (p @ v.permute(0, 2, 1, 3)).view(S, Hk, H // Hk, L, D).permute(0, 3, 1, 2, 4)
    return o.reshape(S, L, H, D)[live].half()


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from paged_kv_cache_73_gb300 import binding as pkv
        if op == "rope":
            return pkv.qk_norm_rope(s["q"], s["key"], s["positions"], s["frequencies"], s["q_weight"], s["k_weight"],
                                    pair_axis=s["pair_axis"], interleaved=c["interleaved"])
        if op == "write":
            pkv.reshape_and_cache_int4(s["key"], s["value"], s["k_cache"], s["v_cache"], s["slots"], c["block_size"])
        if op in ("write", "gather"):
            return pkv.gather_cache_int4(s["k_cache"], s["v_cache"], s["slots"], c["block_size"])
        if op == "decode":
            return pkv.paged_attention_decode_int4(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["ctx"],
                                                   s["scale"], c["block_size"])
        return pkv.prompt_attention(s["q"], s["key"], s["value"], s["query_start"], s["scale"], s["max_len"],
                                    key_start=s["key_start"])
    if op == "rope":
        return plain_rope(s)
    if op == "decode":
        return plain_decode(s)
    if op == "prompt":
        return plain_prompt(s)
    B = c["block_size"]
    if op == "write":
        plain_store(s["k_cache"], s["key"], s["slots"], B)
        plain_store(s["v_cache"], s["value"], s["slots"], B)
    blk, row = s["slots"] // B, s["slots"] % B
    return plain_rows(s["k_cache"], blk, row, B).half(), plain_rows(s["v_cache"], blk, row, B).half()


def work(case):
    """Bytes: inputs once, outputs once (a cached value is half a byte, and four bytes a row).  Flops: the
    products of the attention forms, a few operations a value in the others."""
    op, D, H = case["op"], case["head_dim"], case["heads"]
    row = D // 2 + 4
    if op == "rope":
        n = case["tokens"] * (H + case["kv_heads"]) * D
        return {"bytes": 4 * n + 4 * case["tokens"] * case["axes"], "flops": 8 * n}
    if op == "write":
        n = 2 * case["tokens"] * H
        return {"bytes": n * (4 * D + 2 * row) + 8 * case["tokens"], "flops": 8 * n * D}
    lens = lengths(case)
    total = sum(lens)
    if op == "gather":
        return {"bytes": 2 * total * H * (row + 2 * D) + 8 * total, "flops": 4 * total * H * D}
    Hk = case["kv_heads"]
    if op == "decode":
        return {"bytes": 2 * total * Hk * row + 4 * case["seqs"] * H * D + 4 * total // case["block_size"],
                "flops": 4 * total * H * D}
    past = case["cached"]
    pairs = sum(n * past + n * (n + 1) // 2 for n in lens)
    return {"bytes": 4 * total * H * D + 4 * (total + past * len(lens)) * Hk * D, "flops": 4 * pairs * H * D}


# ---- the definitions in 64 bits -----------------------------------------------------------------------

def stored_exactly(x):
    """What rows x [..., D] stand for once they are held in four bits."""
    top, least = x.max(-1, keepdim=True).values.float(), x.min(-1, keepdim=True).values.float()
    step = ((top - least) / 15.0).half().double()
    count = torch.round((x.double() - least.double()) / torch.where(step == 0, 1.0, step))
    return least.double() + step * torch.where(step == 0, 0.0, count.clamp(0.0, 15.0))


def read_exactly(pool, slots, B):
    out = []
    for h in range(pool.shape[1]):
        tile = pool[:, h].reshape(pool.shape[0], -1)
        half = tile.shape[1] // B - 4                                       # bytes of a row's values
        data = tile[:, :B * half].reshape(-1, half)[slots]
        pair = tile[:, B * half:].reshape(-1, 4)[slots].contiguous().view(torch.float16).double()
        n = torch.empty(len(slots), 2 * half, dtype=torch.float64, device=pool.device)
        n[:, 0::2], n[:, 1::2] = (data % 16).double(), torch.div(data, 16, rounding_mode="floor").double()
        out.append(pair[:, 1:] + n * pair[:, :1])
    return torch.stack(out, 1)                                              # [rows, H, D]


def attended_exactly(q, k, v, scale, positions):
    """q [n, H, D] at the given positions over k, v [m, Hk, D], in 64 bits."""
    n, H, D = q.shape
    out = torch.zeros(n, H, D, dtype=torch.float64, device=q.device)
    if k.shape[0] == 0:
        return out
    hidden = torch.arange(k.shape[0], device=q.device)[None] > positions[:, None]
    for h in range(H):
        kh, vh = k[:, h * k.shape[1] // H].double(), v[:, h * k.shape[1] // H].double()
        w = (q[:, h].double() @ kh.T).mul_(scale).masked_fill_(hidden, -math.inf)
        w = w.sub_(w.max(1, keepdim=True).values).exp_()
        out[:, h] = (w @ vh) / w.sum(1, keepdim=True)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        out = []
        place = s["positions"].double().index_select(0, s["pair_axis"].long())
        z = torch.polar(torch.ones_like(place), place * s["inv_freq"].view(-1, 1)).T.unsqueeze(1)
        R = case["rotary_dim"]
        for x, w in ((s["q"], s["q_weight"]), (s["key"], s["k_weight"])):
            x = x.double()
            if w is not None:
                x = x / (x.pow(2).sum(-1, keepdim=True) / case["head_dim"] + 1e-6).sqrt() * w.double()
            i = torch.arange(R // 2, device=x.device)
            re, im = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + R // 2)
            y = torch.complex(x[..., re], x[..., im]) * z
            x = x.clone()
            x[..., re], x[..., im] = y.real, y.imag
            out.append(x)
        return tuple(out)
    if op == "write":
        return stored_exactly(s["key"]), stored_exactly(s["value"])
    if op == "gather":
        return tuple(read_exactly(s[k], s["slots"], case["block_size"]) for k in ("k_cache", "v_cache"))
    lens = lengths(case)
    out = []
    if op == "decode":
        B = case["block_size"]
        for i, n in enumerate(lens):
            t = torch.arange(n, device=DEV)
            slots = s["tables"][i].long()[t // B] * B + t % B
            k, v = (read_exactly(s[c], slots, B) for c in ("k_cache", "v_cache"))
            out.append(attended_exactly(s["q"][i:i + 1], k, v, s["scale"], torch.tensor([n], device=DEV)))
        return torch.cat(out)
    q0, k0 = starts(lens), starts([n + case["cached"] for n in lens])
    for i, n in enumerate(lens):
        out.append(attended_exactly(s["q"][q0[i]:q0[i + 1]], s["key"][k0[i]:k0[i + 1]], s["value"][k0[i]:k0[i + 1]],
                                    s["scale"], torch.arange(n, device=DEV) + case["cached"]))
    return torch.cat(out)
