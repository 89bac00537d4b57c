"""Measured cases of decoding with drafted tokens over the fp16 paged cache.

One step of it: queries and keys of the drafted tokens are rotated by their positions, and keys and
values written to their slots (``rope_and_cache``); the drafts, a chain or a tree, attend over the
cached context and over their own ancestors (``paged_attention_tree``); the target model's
distributions decide which drafts stay (``verify_draft``); and the kept ones' rows move to the places
that follow the context, in every layer (``move_accepted``).

A case is a dict of plain values; ``run`` computes its operator in plain torch operations, or with
``own`` through the package's binding.  A pool is fp16 [blocks, heads, B, D], and token slot ``n`` is
row ``n % B`` of block ``n // B``.  A sequence's drafts are numbered from 0 (the root, which is no
draft but the last certain token) on, parents before children.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


def listed():
    return [
        # the one new token of each of 64 sequences: latency counts
        {"name": "append_step_64", "op": "append", "tokens": 64, "heads": 40, "kv_heads": 40, "head_dim": 128,
         "rotary_dim": 128, "interleaved": False, "norm": False, "stretch": 1.0, "max_pos": 2048, "block_size": 16},
        # sixteen drafts of each of 64 sequences, half of each head turned in neighbouring pairs
        {"name": "append_drafts", "op": "append", "tokens": 1024, "heads": 64, "kv_heads": 8, "head_dim": 128,
         "rotary_dim": 64, "interleaved": True, "norm": False, "stretch": 1.0, "max_pos": 32768, "block_size": 32},
        # a prompt batch of an odd number of tokens, normalised heads, wavelengths stretched for long contexts
        {"name": "append_prompt", "op": "append", "tokens": 16411, "heads": 40, "kv_heads": 8, "head_dim": 128,
         "rotary_dim": 128, "interleaved": False, "norm": True, "stretch": 8.0, "max_pos": 1000000, "block_size": 16},
        # eight drafts of one 2048-token sequence: the smallest step
        {"name": "tree_one", "op": "tree", "seqs": 1, "lo": 2048, "hi": 2048, "lens": 1, "nodes": 8, "fewest": 8,
         "branch": 3, "heads": 40, "kv_heads": 40, "head_dim": 128, "block_size": 16},
        # the 64-sequence batch of contexts from 128 to 2048 with up to sixteen drafts each
        {"name": "tree_batch", "op": "tree", "seqs": 64, "lo": 128, "hi": 2048, "lens": 2, "nodes": 16, "fewest": 5,
         "branch": 3, "heads": 40, "kv_heads": 40, "head_dim": 128, "block_size": 16},
        # long ragged contexts, eight query heads to a cached head, chains of drafts
        {"name": "tree_long_grouped", "op": "tree", "seqs": 32, "lo": 8192, "hi": 32768, "lens": 3, "nodes": 12,
         "fewest": 12, "branch": 1, "heads": 64, "kv_heads": 8, "head_dim": 128, "block_size": 32},
        # wide trees over mid-length contexts, heads of 64
        {"name": "tree_wide", "op": "tree", "seqs": 16, "lo": 1024, "hi": 8192, "lens": 4, "nodes": 64, "fewest": 33,
         "branch": 4, "heads": 32, "kv_heads": 8, "head_dim": 64, "block_size": 16},
        # a chain of four drafts of one sequence, looked up rather than drawn: they have no distributions
        {"name": "verify_one", "op": "verify", "seqs": 1, "nodes": 5, "fewest": 5, "trees": 5, "branch": 1,
         "vocab": 32000, "draft": False},
        # chains of seven drafts of 64 sequences, rows of an odd length
        {"name": "verify_batch", "op": "verify", "seqs": 64, "nodes": 8, "fewest": 4, "trees": 6, "branch": 1,
         "vocab": 50257, "draft": True},
        # trees of drafts, refused siblings leave their share to the next, a large vocabulary
        {"name": "verify_trees", "op": "verify", "seqs": 128, "nodes": 16, "fewest": 9, "trees": 7, "branch": 3,
         "vocab": 131072, "draft": True},
        # one sequence's kept drafts, all layers
        {"name": "move_one", "op": "move", "seqs": 1, "nodes": 16, "trees": 8, "layers": 40, "heads": 8,
         "head_dim": 128, "block_size": 16},
        # the kept drafts of 64 sequences, all layers
        {"name": "move_batch", "op": "move", "seqs": 64, "nodes": 16, "trees": 9, "layers": 40, "heads": 40,
         "head_dim": 128, "block_size": 16},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "tree", "tree", "verify", "move"])
    head_dim = rng.choice([64, 128, 128])
    block_size = rng.choice([4, 8, 16, 16, 32])
    kv_heads = rng.choice([1, 2, 5, 8, 12, 40])
    group = rng.choice([1, 1, 2, 3, 4, 7, 8]) if kv_heads < 40 else 1
    seed = rng.randrange(1 << 20)
    if op == "append":
        rotary = rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4])
        return {"op": op, "tokens": spread(1, 12000), "heads": kv_heads * min(group, 40 // kv_heads),
                "kv_heads": kv_heads, "head_dim": head_dim, "rotary_dim": rotary, "interleaved": rng.random() < 0.3,
                "norm": rng.random() < 0.5, "stretch": rng.choice([1.0, 1.0, 4.0, 32.0]), "max_pos": spread(64, 1000000),
                "block_size": block_size}
    if op == "tree":
        nodes = spread(1, 64)
        hi = max(nodes, spread(1, 32768))
        pairs = hi * kv_heads * group * nodes
        most = max(1, min(100, (1 << 29) // pairs, (1 << 22) // (hi * kv_heads)))
        return {"op": op, "seqs": spread(1, most), "lo": max(nodes, hi // rng.choice([1, 2, 8])), "hi": hi, "lens": seed,
                "nodes": nodes, "fewest": rng.choice([1, nodes]), "branch": rng.choice([1, 2, 4, 64]),
                "heads": kv_heads * group, "kv_heads": kv_heads, "head_dim": head_dim, "block_size": block_size}
    if op == "verify":
        vocab, nodes = spread(100, 131072), spread(1, 32)
        most = max(1, min(256, (1 << 28) // (vocab * nodes)))
        return {"op": op, "seqs": spread(1, most), "nodes": nodes, "fewest": rng.choice([1, nodes]), "trees": seed,
                "branch": rng.choice([1, 1, 2, 4, 8]), "vocab": vocab, "draft": rng.random() < 0.6}
    return {"op": op, "seqs": spread(1, 64), "nodes": spread(2, 32), "trees": seed, "layers": spread(1, 40),
            "heads": kv_heads, "head_dim": head_dim, "block_size": block_size}


def lengths(case):
    """(context lengths, the drafts in them counted; drafts) of the case's sequences, the longest context at a
    place of its own."""
    r = random.Random(case["lens"])
    got = [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    got[r.randrange(len(got))] = case["hi"]
    return got, [r.randint(case["fewest"], case["nodes"]) for _ in got]


def forest(r, counts, branch):
    """Parents of each sequence's nodes (-1: the root), at most `branch` children to a node, rather deep than wide."""
    out = []
    for n in counts:
        parents, children = [-1], [0]
        for j in range(1, n):
            free = [i for i in range(j) if children[i] < branch]
            p = free[int(len(free) * math.sqrt(r.random()))]
            parents.append(p)
            children[p] += 1
            children.append(0)
        out.append(parents)
    return out


def starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


def inverse_frequencies(case):
    """Radians per position of each pair.  Where the context is stretched, wavelengths of 1/32 of 8192 positions
    and less stay, those over 8192 are `stretch` times as long, and between them it goes over."""
    pairs = case["rotary_dim"] // 2
    inv = 10000.0 ** (-np.arange(pairs) / pairs)
    turns = 8192 * inv / (2 * math.pi)
    keep = np.clip((turns - 1) / 31, 0, 1)
    return inv * (keep + (1 - keep) / case["stretch"])


def magnitude(case):
    return 1 + 0.1 * math.log(case["stretch"])


# ---- what a program has in hand ---------------------------------------------------------------

def gauss(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float16)


def on_gpu(x, dtype):
    return torch.tensor(x, dtype=dtype, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    op, B, D = case["op"], case.get("block_size"), case.get("head_dim")
    if op == "append":
        T, H, Hk = case["tokens"], case["heads"], case["kv_heads"]
        # the projection's output: queries, keys and values of a token side by side
        qkv = gauss(g, T, H + 2 * Hk, D)
        s["q"], s["key"], s["value"] = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        s["q_weight"] = (1 + 0.2 * gauss(g, D)) if case["norm"] else None
        s["k_weight"] = (1 + 0.2 * gauss(g, D)) if case["norm"] else None
        s["positions"] = torch.randint(0, case["max_pos"], (T,), generator=g, device=DEV, dtype=torch.int32)
        inv = inverse_frequencies(case)
        s["inv_freq"] = on_gpu(inv, torch.float64)
        # the same as parts of a turn per position, in units of 2^-64 turns
        s["frequencies"] = on_gpu([int(f / (2 * math.pi) * 2.0 ** 64) for f in inv], torch.int64)
        N = -(-T // B) + 9
        s["k_cache"] = torch.zeros(N, Hk, B, D, dtype=torch.float16, device=DEV)
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        t = torch.arange(T, device=DEV)
        s["slots"] = torch.randperm(N, generator=g, device=DEV)[t // B] * B + t % B
    elif op == "tree":
        lens, counts = lengths(case)
        H, Hk = case["heads"], case["kv_heads"]
        blocks = [-(-n // B) for n in lens]
        N = sum(blocks) + 5
        order = torch.randperm(N, generator=g, device=DEV).to(torch.int32)
        col = torch.arange(max(blocks), device=DEV)
        have = col[None] < on_gpu(blocks, torch.int64)[:, None]
        first = on_gpu(starts(blocks)[:-1], torch.int64)
        s["tables"] = torch.where(have, order[(first[:, None] + col[None]).clamp(max=N - 1)], -1).to(torch.int32)
        s["ctx"] = on_gpu(lens, torch.int32)
        for name in ("k_cache", "v_cache"):
            pool = torch.cat([gauss(g, min(4096, N - i), Hk, B, D) for i in range(0, N, 4096)])
            # slots behind a sequence's end hold what is not a number
            at = torch.arange(max(blocks) * B, device=DEV)
            past = (at[None] >= s["ctx"][:, None]) & have.repeat_interleave(B, 1)
            pool[s["tables"].long().repeat_interleave(B, 1)[past], :, (at % B)[None].expand(len(lens), -1)[past]] = math.nan
            s[name] = pool
        s["q"] = gauss(g, sum(counts), H, D)
        s["query_start"] = on_gpu(starts(counts), torch.int32)
        s["parents"] = forest(random.Random(seed), counts, case["branch"])
        words = (case["nodes"] + 31) // 32
        mask = np.zeros((sum(counts), words), np.uint32)
        row = 0
        for parents in s["parents"]:
            for j, p in enumerate(parents):
                if p >= 0:
                    mask[row + j] = mask[row + p]
                mask[row + j, j // 32] |= np.uint32(1 << j % 32)
            row += len(parents)
        s["mask"] = on_gpu(mask.view(np.int32), torch.int32)
        s["scale"] = 1 / math.sqrt(D)
    elif op == "verify":
        r = random.Random(seed)
        S, V = case["seqs"], case["vocab"]
        counts = [r.randint(case["fewest"], case["nodes"]) for _ in range(S)]
        trees = forest(r, counts, case["branch"])
        s["query_start"] = on_gpu(starts(counts), torch.int32)
        s["parents"] = on_gpu(sum(trees, []), torch.int32)
        first = on_gpu(np.repeat(starts(counts)[:-1], counts), torch.int64)
        rows = (first + s["parents"].clamp(min=0)).long()
        T = sum(counts)
        # the draft's distributions are near the target's, and its drafts are drawn from them
        logits = torch.randn(T, V, generator=g, device=DEV) * 4
        s["target"] = logits.softmax(-1)
        logits += torch.randn(T, V, generator=g, device=DEV) * 0.7
        draft = logits.softmax(-1)
        del logits
        at = torch.rand(T, generator=g, device=DEV, dtype=torch.float64)
        s["tokens"] = torch.cat([(draft[rows[i:i + 64]].double().cumsum(-1) <= at[i:i + 64, None]).sum(-1).clamp(max=V - 1)
                                 for i in range(0, T, 64)]).to(torch.int32)
        s["draft"] = draft if case["draft"] else None
        s["uniforms"] = torch.rand(T, generator=g, device=DEV)
    else:
        r = random.Random(seed)
        S, n, L, H = case["seqs"], case["nodes"], case["layers"], case["heads"]
        per = (n + B - 1) // B + 1                                              # blocks that hold a sequence's drafts
        N = S * per + 3
        pools = torch.empty(L, 2, N, H, B, D, dtype=torch.float16, device=DEV)
        for i in range(L):
            pools[i] = gauss(g, 2, N, H, B, D)
        s["pools"] = pools
        s["k_caches"], s["v_caches"] = [x[0] for x in pools], [x[1] for x in pools]
        place = torch.randperm(N, generator=g, device=DEV)[:S * per].view(S, per)
        off = torch.randint(0, B, (S, 1), generator=g, device=DEV) + torch.arange(n, device=DEV)
        s["slots"] = (place.gather(1, off // B) * B + off % B).flatten()
        s["query_start"] = on_gpu(np.arange(S + 1) * n, torch.int32)
        # the kept drafts lie behind the places that they go to, so that a second pass changes nothing
        kept = [r.randint(1, min(8, (n + 1) // 2)) for _ in range(S)]
        path = np.full((S, 8), -1, np.int32)
        for i, k in enumerate(kept):
            path[i, :k] = [0] + sorted(r.sample(range(k, n), k - 1))
        s["path"], s["path_len"] = on_gpu(path, torch.int32), on_gpu(kept, torch.int32)
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


def plain_append(s):
    c = s["case"]
    angle = (s["positions"].double()[:, None] * s["inv_freq"])[:, None]        # [T, 1, pairs]
    cos, sin = (angle.cos() * magnitude(c)).float(), (angle.sin() * magnitude(c)).float()
    blk, row = s["slots"] // c["block_size"], s["slots"] % c["block_size"]
    s["k_cache"][blk, :, row] = rotated(s["key"], s["k_weight"], cos, sin, c["interleaved"])
    s["v_cache"][blk, :, row] = s["value"]
    return rotated(s["q"], s["q_weight"], cos, sin, c["interleaved"]), s["k_cache"], s["v_cache"]


def softmax_of(x, live):
    """Softmax over the last axis of the live places; a row without any is zeros."""
    x = torch.where(live, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = (x - torch.where(m == -math.inf, 0.0, m)).exp()
    return e / e.sum(-1, keepdim=True).clamp(min=1e-30)


def plain_tree(s):
    c, tables, ctx = s["case"], s["tables"], s["ctx"]
    B, H, Hk, D, n = c["block_size"], c["heads"], c["kv_heads"], c["head_dim"], c["nodes"]
    S = ctx.shape[0]
    i = torch.arange(n, device=ctx.device)
    count = s["query_start"][1:] - s["query_start"][:-1]
    real = i[None] < count[:, None]                                             # [S, n]
    at = (s["query_start"][:-1, None] + i[None]).clamp(max=s["q"].shape[0] - 1).long()
    t = torch.arange(tables.shape[1] * B, device=ctx.device)
    j = t[None] - (ctx - count)[:, None]                                        # [S, L]: which draft, negative in the context
    word = s["mask"][at].gather(2, (j.clamp(0, n - 1) // 32)[:, None].expand(-1, n, -1))
    seen = (word >> (j.clamp(0, n - 1) % 32)[:, None] & 1).bool() | (j < 0)[:, None]
    seen &= (t[None] < ctx[:, None])[:, None]                                   # [S, n, L]
    blk, row = tables.long()[:, t // B].clamp(min=0), (t % B).expand(S, -1)
    q = s["q"][at].float().view(S, n, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).reshape(S, Hk, -1, D)
    k = s["k_cache"][blk, :, row].float().permute(0, 2, 3, 1)                   # [S, Hk, D, L]
    x = (q @ k * s["scale"]).view(S, Hk, H // Hk, n, -1)
    del k
    p = softmax_of(x, seen[:, None, None]).view(S, Hk, -1, t.shape[0])
    del x
    v = s["v_cache"][blk, :, row].float().permute(0, 2, 1, 3)                   # [S, Hk, L, D]
    v = torch.where((t[None] < ctx[:, None])[:, None, :, None], v, 0.0)
    return (p @ v).view(S, Hk, H // Hk, n, D).permute(0, 3, 1, 2, 4).reshape(S, n, H, D)[real].half()


ONE = 1 << 60


def part_of(a, b):
    """floor(a b / 2^60) of whole numbers up to 2^60."""
    mask = (1 << 30) - 1
    a1, a0, b1, b0 = a >> 30, a & mask, b >> 30, b & mask
    return a1 * b1 + (a1 * b0 + a0 * b1 + (a0 * b0 >> 30) >> 30)


def whole(p):
    """floor(p 2^60): fp32 values up to 1, as whole numbers, whose sums do not depend on an order."""
    return (p.double() * float(ONE)).long()


def plain_verify(s):
    """Which drafts stay, in one ascending pass over the nodes of all sequences at once: `left` is what refused
    siblings leave of the current node's distribution, `share` its sum."""
    c = s["case"]
    start, n = s["query_start"].long(), c["nodes"]
    count, S = start[1:] - start[:-1], c["seqs"]
    top = s["target"].shape[0] - 1
    cur, size = torch.zeros_like(count), torch.ones_like(count)
    path = torch.full((S, n), -1, dtype=torch.int32, device=cur.device)
    path[:, 0] = 0
    left, share = whole(s["target"][start[:-1]]), torch.full_like(count, ONE)
    u = whole(s["uniforms"])
    for j in range(1, n):
        at = (start[:-1] + j).clamp(max=top)
        tried = (j < count) & (s["parents"][at] == cur)
        x = s["tokens"][at].long()[:, None]
        has = left.gather(1, x)[:, 0]
        if c["draft"]:
            q = whole(s["draft"][start[:-1] + cur])
            ok = tried & (part_of(part_of(share, q.gather(1, x)[:, 0]), u[at]) < has)
            after = (left - part_of(share[:, None], q)).clamp(min=0)
            rest = after.sum(-1)
        else:
            ok = tried & (part_of(share, u[at]) < has)
            after = left.scatter(1, x, 0)
            rest = (share - has).clamp(min=0)
        no = tried & ~ok
        left, share = torch.where(no[:, None], after, left), torch.where(no, rest, share)
        left = torch.where(ok[:, None], whole(s["target"][at]), left)
        share = torch.where(ok, ONE, share)
        cur = torch.where(ok, j, cur)
        path.scatter_(1, torch.where(ok, size, 0)[:, None], torch.where(ok, j, 0)[:, None].int())
        size = size + ok
    total = left.sum(-1)
    # nothing left (the target gives nothing that the draft does not): the node's own distribution
    left = torch.where((total == 0)[:, None], whole(s["target"][start[:-1] + cur]), left)
    aim = part_of(left.sum(-1), u[start[:-1]])
    token = (left.cumsum(-1) <= aim[:, None]).sum(-1)
    return path, size.int(), token.int()


def plain_move(s):
    B = s["case"]["block_size"]
    slots, path, pools = s["slots"].view(s["case"]["seqs"], -1), s["path"].long(), s["pools"]
    i = torch.arange(path.shape[1], device=path.device)[None].expand_as(path)
    i = torch.where(i < s["path_len"][:, None], i, 0)
    src = slots.gather(1, torch.where(i > 0, path, 0)).flatten()
    dst = slots.gather(1, i).flatten()
    pools[:, :, dst // B, :, dst % B] = pools[:, :, src // B, :, src % B]
    return pools


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from paged_kv_cache_73_gb300 import binding as pkv
        if op == "append":
            q = pkv.rope_and_cache(s["q"], s["key"], s["value"], s["positions"], s["frequencies"], s["k_cache"],
                                   s["v_cache"], s["slots"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                   interleaved=c["interleaved"], rotary_scale=magnitude(c))
            return q, s["k_cache"], s["v_cache"]
        if op == "tree":
            return pkv.paged_attention_tree(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["ctx"],
                                            s["query_start"], s["scale"], c["block_size"], c["nodes"],
                                            tree_mask=s["mask"])
        if op == "verify":
            return pkv.verify_draft(s["target"], s["tokens"], s["parents"], s["query_start"], s["uniforms"],
                                    c["nodes"], draft_probs=s["draft"])
        pkv.move_accepted(s["k_caches"], s["v_caches"], s["slots"], s["query_start"], s["path"], s["path_len"])
        return s["pools"]
    if op == "append":
        return plain_append(s)
    if op == "tree":
        return plain_tree(s)
    if op == "verify":
        return plain_verify(s)
    return plain_move(s)


def work(case):
    """Bytes: inputs once, outputs once; of the verified distributions the row that the next token is drawn from
    (of the draft's too).  Flops: the products over all cached tokens in attention, a few operations a value
    elsewhere."""
    op = case["op"]
    if op == "verify":
        n = case["seqs"] * case["vocab"] * (2 if case["draft"] else 1)
        return {"bytes": 4 * n + 24 * case["seqs"] * case["nodes"], "flops": 4 * n}
    D, H = case["head_dim"], case["heads"]
    if op == "append":
        n = case["tokens"] * (H + 2 * case["kv_heads"]) * D
        return {"bytes": 4 * n + 12 * case["tokens"], "flops": 8 * n}
    if op == "tree":
        lens, counts = lengths(case)
        pairs = sum(c * n for c, n in zip(lens, counts))
        return {"bytes": 4 * sum(lens) * case["kv_heads"] * D + 4 * sum(counts) * H * D, "flops": 4 * pairs * H * D}
    rows = case["seqs"] * max(1, min(8, (case["nodes"] + 1) // 2) // 2) * case["layers"] * 2 * H
    return {"bytes": rows * 4 * D, "flops": rows}


# ---- the definitions in 64 bits -----------------------------------------------------------------------

def turned_exactly(s, x, w):
    c = s["case"]
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / c["head_dim"] + 1e-6).sqrt() * w.double()
    z = torch.polar(torch.full_like(s["inv_freq"], magnitude(c)).expand(c["tokens"], -1),
                    s["positions"].double().view(-1, 1) * s["inv_freq"]).unsqueeze(1)
    i = torch.arange(c["rotary_dim"] // 2, device=x.device)
    re, im = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + c["rotary_dim"] // 2)
    y = torch.complex(x[..., re], x[..., im]) * z
    x = x.clone()
    x[..., re], x[..., im] = y.real, y.imag
    return x


def laid_out(pool, slots, x):
    """A pool's values in 64 bits with rows x at the slots."""
    N, H, B, D = pool.shape
    out = pool.double().transpose(1, 2).reshape(N * B, H, D)
    out[slots] = x.double()
    return out.view(N, B, H, D).transpose(1, 2)


def ancestors(parents):
    out = torch.zeros(len(parents), len(parents), dtype=torch.bool)
    for i in range(len(parents)):
        j = i
        while j >= 0:
            out[i, j] = True
            j = parents[j]
    return out.to(DEV)


def attended_exactly(q, k, v, scale, tree):
    """q [n, H, D] over k, v [m, Hk, D], whose last n are its own, in 64 bits."""
    n, H, D = q.shape
    m, Hk = k.shape[:2]
    hidden = torch.zeros(n, m, dtype=torch.bool, device=q.device)
    hidden[:, m - n:] = ~tree
    out = torch.zeros(n, H, D, dtype=torch.float64, device=q.device)
    for h in range(Hk):
        mine = slice(h * (H // Hk), (h + 1) * (H // Hk))
        kh, vh = k[:, h].double(), v[:, h].double()
        w = (q[:, mine].double() @ kh.T).mul_(scale).masked_fill_(hidden[:, None], -math.inf)
        w = w.sub_(w.max(-1, keepdim=True).values).exp_()
        out[:, mine] = (w @ vh) / w.sum(-1, keepdim=True)
    return out


def verified_exactly(p, q, tokens, parents, u):
    """One sequence: (the path's nodes, the next token)."""
    path, at, rest, mass = [0], 0, p[0].double(), 1.0
    for j in range(1, len(tokens)):
        if parents[j] != at:
            continue
        x = tokens[j]
        chance = float(rest[x]) / mass if mass > 0 else 0.0
        if u[j] * (1.0 if q is None else float(q[at, x])) < chance:
            path.append(j)
            at, rest, mass = j, p[j].double(), 1.0
        elif q is None:
            mass -= float(rest[x])
            rest = rest.clone()
            rest[x] = 0.0
        else:
            rest = torch.relu(rest - mass * q[at].double())
            mass = float(rest.sum())
    if float(rest.sum()) == 0:
        rest = p[at].double()
    running = rest.cumsum(0)
    return path, int(torch.searchsorted(running, running[-1] * u[0], right=True))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "append":
        return (turned_exactly(s, s["q"], s["q_weight"]),
                laid_out(s["k_cache"], s["slots"], turned_exactly(s, s["key"], s["k_weight"])),
                laid_out(s["v_cache"], s["slots"], s["value"]))
    if op == "tree":
        (lens, counts), B, out = lengths(case), case["block_size"], []
        q0 = starts(counts)
        for i, n in enumerate(lens):
            t = torch.arange(n, device=DEV)
            blk = s["tables"][i].long()[t // B]
            out.append(attended_exactly(s["q"][q0[i]:q0[i + 1]], s["k_cache"][blk, :, t % B], s["v_cache"][blk, :, t % B],
                                        s["scale"], ancestors(s["parents"][i])))
        return torch.cat(out)
    if op == "verify":
        q0 = s["query_start"].tolist()
        tokens, parents, u = s["tokens"].tolist(), s["parents"].tolist(), s["uniforms"].tolist()
        paths = np.full((case["seqs"], case["nodes"]), -1, np.int32)
        size, token = [], []
        for i in range(case["seqs"]):
            a, b = q0[i], q0[i + 1]
            path, x = verified_exactly(s["target"][a:b], None if s["draft"] is None else s["draft"][a:b], tokens[a:b],
                                       parents[a:b], u[a:b])
            paths[i, :len(path)] = path
            size.append(len(path))
            token.append(x)
        return paths, np.array(size, np.int32), np.array(token, np.int32)
    # rows as they lie token after token, one sequence after the other
    L, _, N, H, B, D = s["pools"].shape
    rows = s["pools"].transpose(3, 4).reshape(L, 2, N * B, H, D)
    slots, path, size = s["slots"].tolist(), s["path"].tolist(), s["path_len"].tolist()
    for i, k in enumerate(size):
        for j in range(1, k):
            a, b = slots[i * case["nodes"] + path[i][j]], slots[i * case["nodes"] + j]
            rows[:, :, b] = rows[:, :, a]
    return rows.view(L, 2, N, B, H, D).transpose(3, 4).double()
