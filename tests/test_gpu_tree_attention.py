"""paged_attention_tree on the GPU against the fp64 oracle on the same pools.

Tolerance per value, derived, with a = sum p |v|: the output's fp16 rounding is 2^-11 |o| (2^-25 below the normals).
Weights are rounded to fp16 and summed as rounded, 2^-11 of each: 2^-11 (a + |o|); those under 2^-32 of the row's
largest are lost, n 2^-32 of the largest |v| at most.  A logit of D products in fp32, the tensor cores cutting
off each of D / 16 sums at its last bit, is off by (D / 8) 2^-23 of sum |q k|, its scaling by 2^-23 of itself, the
exponential by 2^-22 relative: dx of the weights each, so 2 dx a.  Sums over n keys lose n 2^-27 a."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import drafts as od
from paged_kv_cache_73_gb300 import binding as pkv

pytestmark = pytest.mark.gpu


def parents_of(rng, n, wide=False):
    return [-1] + [0 if wide else int(rng.integers(max(0, j - 4), j)) for j in range(1, n)]


def make(seed, lens, counts, H, Hk, D, B, extra=3, q_scale=1.0, trees=None):
    """Pools whose slots outside the contexts are NaN; masks of random trees."""
    rng = np.random.default_rng(seed)
    blocks = [-(-n // B) for n in lens]
    N = sum(blocks) + extra
    ids = rng.permutation(N).astype(np.int32)
    tables = np.full((len(lens), max(1, max(blocks))), -1, np.int32)
    at = 0
    live = np.zeros((N, B), bool)
    for s, b in enumerate(blocks):
        tables[s, :b] = ids[at:at + b]
        at += b
        t = np.arange(lens[s])
        live[tables[s][t // B], t % B] = True
    pools = []
    for _ in range(2):
        pool = rng.standard_normal((N, Hk, B, D)).astype(np.float16)
        pool.transpose(0, 2, 1, 3)[~live] = np.nan
        pools.append(pool)
    q = (rng.standard_normal((sum(counts), H, D)) * q_scale).astype(np.float16)
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    trees = [parents_of(rng, n) if n else [] for n in counts] if trees is None else trees
    return dict(q=q, k=pools[0], v=pools[1], tables=tables, lens=np.array(lens, np.int32), start=start, parents=trees,
                seen=[od.ancestors(p) for p in trees], B=B)


def words_of(c, words):
    out = np.zeros((c["q"].shape[0], words * 32), bool)
    for s, seen in enumerate(c["seen"]):
        q0, n = c["start"][s], len(seen)
        out[q0:q0 + n, :n] = seen
    return (out.reshape(out.shape[0], words, 32) << np.arange(32, dtype=np.uint32)).sum(-1).astype(np.uint32).view(np.int32)


def call(c, dev, scale=None, mask=True, most=None, **kw):
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)
    most = max(1, int(np.diff(c["start"]).max())) if most is None else most
    m = t(words_of(c, max(1, -(-most // 32)))) if mask else None
    scale = c["q"].shape[2] ** -0.5 if scale is None else scale
    return pkv.paged_attention_tree(kw.pop("q", None) if "q" in kw else t(c["q"]), t(c["k"]), t(c["v"]), t(c["tables"]),
                                    t(c["lens"]), t(c["start"]), scale, c["B"], most, tree_mask=m, **kw)


def tolerance(c, want, scale):
    T, H, D = c["q"].shape
    group = H // c["k"].shape[1]
    tol = np.zeros_like(want)
    for s, n_ctx in enumerate(c["lens"]):
        q0, n = c["start"][s], c["start"][s + 1] - c["start"][s]
        if n == 0 or n_ctx == 0:
            continue
        k = oa.gather_sequence(c["k"], c["tables"][s], n_ctx)
        v = oa.gather_sequence(c["v"], c["tables"][s], n_ctx)
        for i in range(n):
            live = np.concatenate([np.ones(n_ctx - n, bool), c["seen"][s][i]])
            if not live.any():
                continue
            for h in range(H):
                q = c["q"][q0 + i, h].astype(np.float64)
                kk, vv = k[live][:, h // group], v[live][:, h // group]
                x = scale * kk @ q
                p = np.exp(x - x.max())
                p /= p.sum()
                a = p @ np.abs(vv)
                size = (np.abs(kk) @ np.abs(q)).max() * scale
                dx = D / 8 * 2.0 ** -23 * size + 2.0 ** -23 * np.abs(x).max() + 2.0 ** -22
                o = np.abs(want[q0 + i, h])
                tol[q0 + i, h] = (2.0 ** -11 * o + 2.0 ** -25 + 2.0 ** -11 * (a + o) + 2 * dx * a
                                  + n_ctx * (2.0 ** -27 * a + 2.0 ** -32 * np.abs(vv).max(0)) + 2.0 ** -20 * a)
    return tol


def check(c, dev, scale=None, **kw):
    scale = c["q"].shape[2] ** -0.5 if scale is None else scale
    with np.errstate(invalid="ignore"):
        want = od.tree_attention(c["q"], c["k"], c["v"], c["tables"], c["lens"], c["start"], c["seen"], scale)
    got = call(c, dev, scale, **kw).cpu().numpy().astype(np.float64)
    code = pkv.device_error()
    assert code == 0, pkv.DEV_CODES[code]
    used = ~np.isnan(want)
    err, tol = np.abs(got - want)[used], tolerance(c, want, scale)[used]
    assert np.isfinite(got[used]).all() and (err <= tol).all(), float((err / np.maximum(tol, 1e-30)).max())
    return got


LENS = [1, 2, 5, 15, 16, 17, 33, 63, 64, 65, 70, 127, 128, 129, 300]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [4, 8, 16, 32])
def test_ragged_lengths(cuda_device, D, B):
    check(make(D + B, LENS, [min(n, 1 + 5 * i % 13) for i, n in enumerate(LENS)], 3, 3, D, B), cuda_device)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 16, 40])
def test_grouped_heads(cuda_device, D, group):
    check(make(group + D, [7, 90, 300], [7, 1, 9], 2 * group, 2, D, 16), cuda_device)


@pytest.mark.parametrize("nodes,group", [(31, 1), (32, 1), (33, 2), (64, 1), (65, 4), (128, 1), (129, 1), (200, 2), (300, 1)])
def test_many_nodes(cuda_device, nodes, group):
    check(make(nodes, [nodes, nodes + 70, nodes + 200], [nodes, nodes // 2, nodes], group, 1, 64, 16), cuda_device)


@pytest.mark.parametrize("seqs,ctx,nodes,H,Hk", [(1, 2048, 8, 8, 8), (1, 5000, 3, 4, 1), (3, 1500, 16, 16, 2), (100, 400, 2, 2, 1),
                                                 (2, 3000, 40, 4, 1), (1, 4000, 1, 2, 2)])
def test_split_contexts(cuda_device, seqs, ctx, nodes, H, Hk):
    lens = [max(nodes, ctx - 37 * i % ctx) for i in range(seqs)]
    check(make(seqs + ctx, lens, [nodes] * seqs, H, Hk, 128, 16), cuda_device)


def test_without_a_mask_drafts_are_a_chain(cuda_device):
    counts = [1, 9, 40, 0, 130]
    c = make(31, [1, 200, 40, 20, 130], counts, 4, 2, 64, 8, trees=[list(range(-1, n - 1)) for n in counts])
    a, b = check(c, cuda_device, mask=False), check(c, cuda_device)
    used = slice(0, sum(counts))
    assert np.array_equal(a[used], b[used])


def test_masks_that_leave_nothing_or_any_node(cuda_device):
    rng = np.random.default_rng(32)
    c = make(32, [20, 20, 90, 100], [20, 20, 40, 70], 2, 1, 64, 16)
    c["seen"] = [rng.random((n, n)) < 0.5 for n in (20, 20, 40, 70)]    # also later nodes, and not oneself
    c["seen"][0][3] = False
    c["seen"][1][:] = False
    got = check(c, cuda_device)
    assert (got[3] == 0).all() and (got[20:40] == 0).all()


def test_bits_past_the_nodes_do_not_matter(cuda_device):
    c = make(33, [30, 60], [5, 37], 2, 2, 64, 16)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(cuda_device)
    words = words_of(c, 3).view(np.uint32)
    args = [t(c[n]) for n in ("q", "k", "v", "tables", "lens", "start")] + [0.125, 16, 64]
    want = pkv.paged_attention_tree(*args, tree_mask=t(words.view(np.int32)))
    noisy = words.copy()
    noisy[:5, 0] |= np.uint32(0xffffffe0)
    noisy[:5, 1:] = 0xffffffff
    noisy[5:, 1] |= np.uint32(0xffffffe0)
    noisy[5:, 2] = 0xabcdef01
    assert torch.equal(want, pkv.paged_attention_tree(*args, tree_mask=t(noisy.view(np.int32))))


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("nodes,lens", [(6, [6, 100]), (40, [40, 333])])
def test_what_is_not_seen_may_hold_anything(cuda_device, value, nodes, lens):
    """One node's key and value are not finite: rows that do not see it are as if it were finite, rows that
    do get what the definition gives."""
    c = make(nodes + 34, lens, [nodes, nodes], 2, 1, 64, 8, trees=[parents_of(np.random.default_rng(5), nodes, wide=True)] * 2)
    for row in c["seen"]:
        row[5, 4] = True                                                # node 5 sees node 4 as well
    clean = check(c, cuda_device)
    for s, ctx in enumerate(lens):
        t = ctx - nodes + 4
        blk, r = c["tables"][s][t // 8], t % 8
        c["v"][blk, 0, r, 3] = value
        c["v"][blk, 0, r, 62] = -value
    got = call(c, cuda_device).cpu().numpy().astype(np.float64)
    assert pkv.device_error() == 0
    for s in range(2):
        for i in range(nodes):
            row, want = got[s * nodes + i], clean[s * nodes + i].copy()
            if i in (4, 5):
                want[:, 3], want[:, 62] = value, -value
            assert np.array_equal(row, want, equal_nan=True), (s, i)
    for s, ctx in enumerate(lens):
        t = ctx - nodes + 4
        c["k"][c["tables"][s][t // 8], 0, t % 8, :] = value
    got = call(c, cuda_device).cpu().numpy().astype(np.float64)
    for s in range(2):
        for i in range(nodes):
            if i not in (4, 5):
                assert np.array_equal(got[s * nodes + i], clean[s * nodes + i])


def test_infinite_values_in_the_context_reach_all(cuda_device):
    c = make(35, [150], [3], 2, 1, 64, 16)
    c["v"][c["tables"][0][2], 0, 5, 7] = np.inf
    got = call(c, cuda_device).cpu().numpy()
    assert np.isinf(got[:, :, 7]).all() and np.isfinite(np.delete(got, 7, axis=2)).all()


def test_a_row_that_sees_only_infinite_logits(cuda_device):
    c = make(36, [40], [2], 1, 1, 64, 16)
    c["q"][0, 0, :] = 60000.0
    c["q"][1, 0, :] = 0.0
    got = call(c, cuda_device, scale=4.0).cpu().numpy().astype(np.float64)
    want = od.tree_attention(c["q"], c["k"], c["v"], c["tables"], c["lens"], c["start"], c["seen"], 4.0)
    assert np.abs(got - want).max() <= 2.0 ** -9 * 4        # one key takes all, or all alike; |v| below 4 or so


@pytest.mark.parametrize("ctx", [40, 3000])                 # one part, and many
def test_infinite_logits(cuda_device, ctx):
    """A key of -inf in the context has no weight, one of +inf (exp(inf - inf)) makes its row a NaN; a draft's reach the
    rows that see it alone."""
    nodes = 6
    c = make(44, [ctx], [nodes], 2, 1, 64, 16, trees=[[-1, 0, 0, 1, 1, 2]])
    c["q"][:] = np.abs(c["q"]) + np.float16(0.125)          # logits of such a key have one sign
    at = lambda t: (c["tables"][0][t // 16], 0, t % 16)
    c["k"][at(7)] = -np.inf
    got = call(c, cuda_device).cpu().numpy().astype(np.float64)
    assert pkv.device_error() == 0
    keep = np.arange(ctx) != 7
    k, v = (oa.gather_sequence(c[n], c["tables"][0], ctx)[keep] for n in ("k", "v"))
    for i in range(nodes):
        live = np.concatenate([np.ones(ctx - nodes - 1, bool), c["seen"][0][i]])
        # as above with |o| and a at most the largest |v|, and dx below 2^-15 (logits here stay under 2^5)
        most = (3 * 2.0 ** -11 + 2.0 ** -13) * np.abs(v).max()
        assert np.abs(got[i] - oa.contiguous_attention(c["q"][i], np.repeat(k[live], 2, axis=1), np.repeat(v[live], 2, axis=1), 0.125)).max() < most
    c["k"][at(ctx - nodes + 2)] = np.inf                    # node 2, which itself and its child 5 see
    row = call(c, cuda_device).cpu().numpy().astype(np.float64)
    assert np.isnan(row[[2, 5]]).all() and np.array_equal(row[[0, 1, 3, 4]], got[[0, 1, 3, 4]])
    c["k"][at(9)] = np.inf
    assert np.isnan(call(c, cuda_device).cpu().numpy()).all()
    # nothing but keys without weight: as a row that sees nothing
    c = make(45, [6], [6], 2, 1, 64, 16)
    c["q"][:], c["k"][:] = 1, -np.inf
    assert (call(c, cuda_device).cpu().numpy() == 0).all() and pkv.device_error() == 0


@pytest.mark.parametrize("nodes,ctx,H,Hk,D", [(700, 700, 2, 2, 64), (1100, 1500, 2, 1, 128)])
def test_prompt_chunks(cuda_device, nodes, ctx, H, Hk, D):
    """Hundreds of new tokens, as a chain without a mask and as a tree."""
    c = make(nodes, [ctx, 50], [nodes, 3], H, Hk, D, 16, trees=[list(range(-1, nodes - 1)), [-1, 0, 1]])
    a, b = check(c, cuda_device, mask=False), check(c, cuda_device)
    assert np.array_equal(a, b)
    check(make(nodes + 1, [ctx], [nodes], H, Hk, D, 16), cuda_device)


def test_the_same_twice(cuda_device):
    """Parts are cut and joined in one order: a call repeats itself bit for bit, whatever ran in between."""
    cs = [make(46, [2048], [8], 8, 8, 128, 16), make(47, [900, 77, 3, 1500], [12, 5, 3, 40], 8, 2, 128, 16),
          make(48, [1000] * 9, [33] * 9, 8, 2, 64, 16)]
    n = max(pkv.paged_attention_tree_workspace_size(len(c["lens"]), c["q"].shape[0], 64, *c["q"].shape[1:2], c["k"].shape[1], 128,
                                                    c["tables"].shape[1], 16) for c in cs)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=cuda_device)
    want = [call(c, cuda_device, workspace=ws).clone() for c in cs]
    for order in ((2, 0, 1), (0, 0, 2), (1, 2, 0)):
        for i in order:
            assert torch.equal(call(cs[i], cuda_device, workspace=ws), want[i])


def test_an_output_at_half_a_sector(cuda_device):
    c = make(49, [300, 20], [9, 3], 4, 2, 64, 16)
    want = call(c, cuda_device)
    buf = torch.full((12 * 4 * 64 + 16,), 7.0, dtype=torch.float16, device=cuda_device)
    out = buf[8:-8].view(12, 4, 64)                          # 16 bytes past a 32-byte boundary
    assert torch.equal(call(c, cuda_device, out=out), want) and (buf[:8] == 7).all() and (buf[-8:] == 7).all()


@pytest.mark.parametrize("q_scale", [0.0, 2.0 ** -20, 30.0])
def test_queries_of_any_size(cuda_device, q_scale):
    check(make(37, [300, 5], [9, 5], 4, 2, 128, 16, q_scale=q_scale), cuda_device)


def test_rising_logits_move_the_maximum(cuda_device):
    c = make(38, [1500, 700], [4, 30], 2, 2, 64, 16)
    c["tables"][0, :94] = np.sort(c["tables"][0, :94])
    c["k"][..., 0] = np.linspace(-40, 40, c["k"].shape[0])[:, None, None].astype(np.float16)
    c["q"][..., 0] = 3
    live = np.isnan(c["v"][..., 0])
    c["k"][live] = np.nan
    check(c, cuda_device)


def test_strided_queries_and_given_buffers(cuda_device):
    c = make(39, [100, 33], [8, 5], 4, 2, 64, 16)
    wide = torch.randn(13, 8, 64, device=cuda_device).half()
    wide[:, :4] = torch.from_numpy(c["q"]).to(cuda_device)
    want = call(c, cuda_device)
    out = torch.full((13, 4, 64), 7.0, dtype=torch.float16, device=cuda_device)
    n = pkv.paged_attention_tree_workspace_size(2, 13, 8, 4, 2, 64, c["tables"].shape[1], 16)
    ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device=cuda_device)
    got = call(c, cuda_device, q=wide[:, :4], out=out, workspace=ws)
    assert got is out and torch.equal(out, want)
    if n:
        with pytest.raises(pkv.PkvError) as e:
            call(c, cuda_device, workspace=ws[:n - 16])
        assert e.value.status == pkv.PKV_ERR_WORKSPACE


def test_rows_in_no_sequence_are_left(cuda_device):
    c = make(40, [50, 60], [3, 5], 2, 2, 64, 16)
    want = call(c, cuda_device)
    q = torch.zeros(12, 2, 64, dtype=torch.float16, device=cuda_device)
    q[:8] = torch.from_numpy(c["q"]).to(cuda_device)
    c2 = dict(c, q=np.zeros((12, 2, 64), np.float16))
    out = torch.full((12, 2, 64), 7.0, dtype=torch.float16, device=cuda_device)
    call(c2, cuda_device, q=q, out=out)
    assert torch.equal(out[:8], want) and (out[8:] == 7).all() and pkv.device_error() == 0


def test_bad_blocks_lengths_and_ranges(cuda_device):
    c = make(41, [40, 300, 30], [4, 4, 4], 2, 2, 64, 16)
    want = call(c, cuda_device)
    tables = c["tables"].copy()
    tables[1, 2], tables[0, 3:] = c["k"].shape[0], 10 ** 6  # past the context: never looked at
    got = call(dict(c, tables=tables), cuda_device)
    assert pkv.device_error() == 1 and pkv.device_error() == 0
    assert torch.equal(got[:4], want[:4]) and torch.equal(got[8:], want[8:])
    # the bad block's tokens have no weight
    keep = np.r_[0:32, 48:300]
    kk, vv = (oa.gather_sequence(c[n], c["tables"][1], 300)[keep] for n in ("k", "v"))
    for i in range(4):
        live = np.r_[np.ones(280, bool), c["seen"][1][i]]
        o = oa.contiguous_attention(c["q"][4 + i], kk[live], vv[live], 0.125)
        assert np.abs(got[4 + i].cpu().numpy() - o).max() < 2e-3
    for bad, code in ((dict(lens=[40, tables.shape[1] * 16 + 1, 30]), 2), (dict(lens=[40, -1, 30]), 2), (dict(lens=[40, 3, 30]), 6),
                      (dict(start=[0, 4, 8, 13]), 6)):
        out = torch.full((12, 2, 64), 7.0, dtype=torch.float16, device=cuda_device)
        call(dict(c, **{k: np.array(v, np.int32) for k, v in bad.items()}), cuda_device, out=out, most=5, mask=False)
        assert pkv.device_error() == code and pkv.device_error() == 0
        assert (out[8:] == 7).all() if "start" in bad else (out[4:8] == 7).all()
    # more nodes than max_query_len
    out = torch.full((12, 2, 64), 7.0, dtype=torch.float16, device=cuda_device)
    call(dict(c, start=np.array([0, 2, 10, 12], np.int32)), cuda_device, out=out, most=4, mask=False)
    assert pkv.device_error() == 6 and (out[2:10] == 7).all() and (out[10:] != 7).any()


def test_a_block_twice_and_offsets_past_32_bits(cuda_device):
    B, Hk, D = 32, 8, 128
    N = (1 << 32) // (Hk * B * D) + 9
    c = make(42, [500], [6], 16, Hk, D, B)
    big = [torch.empty(N, Hk, B, D, dtype=torch.float16, device=cuda_device) for _ in range(2)]
    tables = c["tables"].copy()
    tables[0, 3] = tables[0, 9]                              # the same block at two places
    c["tables"] = tables
    want = check(c, cuda_device)
    moved = np.where(tables >= 0, N - 1 - tables, -1).astype(np.int32)
    for pool, name in zip(big, "kv"):
        pool[torch.from_numpy(N - 1 - np.arange(c[name].shape[0])).to(cuda_device)] = torch.from_numpy(c[name]).to(cuda_device)
    t = lambda x: torch.from_numpy(x).to(cuda_device)
    got = pkv.paged_attention_tree(t(c["q"]), big[0], big[1], t(moved), t(c["lens"]), t(c["start"]), D ** -0.5, B, 6,
                                   tree_mask=t(words_of(c, 1)))
    assert np.array_equal(got.cpu().numpy().astype(np.float64), want)


def test_two_streams_at_once_and_a_captured_call(cuda_device):
    cs = [make(43 + i, [900, 77 + i], [12, 5], 8, 2, 128, 16) for i in range(2)]
    want = [call(c, cuda_device) for c in cs]
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(cuda_device)
    args = [[t(c[n]) for n in ("q", "k", "v", "tables", "lens", "start")] + [128 ** -0.5, 16, 12] for c in cs]
    masks = [t(words_of(c, 1)) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            outs[i].append(pkv.paged_attention_tree(*args[i], tree_mask=masks[i], stream=st))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in outs[i])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = pkv.paged_attention_tree(*args[0], tree_mask=masks[0])
    args[0][0].copy_(args[1][0])
    for a, b in zip(args[0][1:3], args[1][1:3]):
        a[:b.shape[0]].copy_(b[:a.shape[0]])
    args[0][3].copy_(args[1][3])
    args[0][4].copy_(args[1][4])
    masks[0].copy_(masks[1])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[1]) and pkv.device_error() == 0


def test_refusals(cuda_device):
    c = make(50, [50, 60], [3, 5], 4, 2, 64, 16)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(cuda_device)
    q, k, v, tab, lens, start = [t(c[n]) for n in ("q", "k", "v", "tables", "lens", "start")]
    ok = [q, k, v, tab, lens, start, 0.125, 16, 5]
    for i, bad in ((0, q.float()), (0, q[:, :3]), (1, k[:2]), (1, k.cpu()), (3, tab.long()), (4, lens[:1]), (5, start[:2]), (6, 0.0),
                   (6, -1.0), (7, 8)):
        with pytest.raises(pkv.PkvError):
            pkv.paged_attention_tree(*ok[:i], bad, *ok[i + 1:])
    for kw in (dict(tree_mask=torch.zeros(7, 1, dtype=torch.int32, device=cuda_device)),
               dict(tree_mask=torch.zeros(8, 0, dtype=torch.int32, device=cuda_device)), dict(out=q[:5].contiguous())):
        with pytest.raises(pkv.PkvError):
            pkv.paged_attention_tree(*ok, **kw)


def test_more_sequences_than_are_looked_up_at_a_time(cuda_device):
    """9000 sequences of few tokens, some without any or with a length that is refused."""
    rng = np.random.default_rng(60)
    lens = rng.integers(1, 40, 9000)
    counts = np.minimum(lens, rng.integers(0, 4, 9000))
    c = make(61, lens.tolist(), counts.tolist(), 2, 1, 64, 16)
    got = check(c, cuda_device)
    bad = c["lens"].copy()
    bad[4100] = -5
    out = torch.full((c["q"].shape[0], 2, 64), 7.0, dtype=torch.float16, device=cuda_device)
    call(dict(c, lens=bad), cuda_device, out=out)
    assert pkv.device_error() == (2 if counts[4100] else 0)
    out = out.cpu().numpy().astype(np.float64)
    mine = slice(c["start"][4100], c["start"][4101])
    assert (out[mine] == 7).all()
    out[mine] = got[mine]
    assert np.abs(out - got).max() < 2e-3               # cut elsewhere: other parts are joined
