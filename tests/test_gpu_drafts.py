"""verify_draft and move_accepted on the GPU: whole numbers, so equal to the oracle; and a run of the whole set."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import drafts as od
from paged_kv_cache_73_gb300 import binding as pkv

pytestmark = pytest.mark.gpu


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def make(seed, counts, V, branch=2, sharp=3.0, noise=0.7):
    rng = np.random.default_rng(seed)
    T = sum(counts)
    logits = rng.standard_normal((T, V)) * sharp
    target, draft = softmax(logits), softmax(logits + noise * rng.standard_normal((T, V)))
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    parents, tokens = [], np.zeros(T, np.int32)
    for s, n in enumerate(counts):
        p = [-1] * min(n, 1) + [int(rng.integers(max(0, j - branch), j)) for j in range(1, n)]
        parents += p
        for j in range(1, n):
            q = draft[start[s] + p[j]].astype(np.float64)
            tokens[start[s] + j] = rng.choice(V, p=q / q.sum())
    return dict(target=target, draft=draft, tokens=tokens, parents=np.array(parents, np.int32), start=start,
                u=rng.random(T, dtype=np.float32))


def call(c, dev, max_path, with_draft=True, **kw):
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)
    return pkv.verify_draft(t(c["target"]), t(c["tokens"]), t(c["parents"]), t(c["start"]), t(c["u"]), max_path,
                            draft_probs=t(c["draft"]) if with_draft else None, **kw)


def check(c, dev, max_path, with_draft=True):
    path, size, token = (x.cpu().numpy() for x in call(c, dev, max_path, with_draft))
    assert pkv.device_error() == 0
    sizes = []
    for s in range(len(size)):
        a, b = c["start"][s], c["start"][s + 1]
        if a == b:
            assert size[s] == 0 and token[s] == -1 and (path[s] == -1).all()
            continue
        want, x = od.verify(c["target"][a:b], c["draft"][a:b] if with_draft else None, c["tokens"][a:b], c["parents"][a:b],
                            c["u"][a:b], max_path)
        assert path[s, :size[s]].tolist() == want and (path[s, size[s]:] == -1).all() and token[s] == x
        sizes.append(len(want))
    return sizes


@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 127, 1000, 4099])
def test_against_oracle(cuda_device, V, with_draft):
    check(make(V, [1, 2, 5, 0, 9, 16, 3, 3], V), cuda_device, 16, with_draft)


@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("branch", [1, 3, 40])
def test_trees(cuda_device, branch, with_draft):
    sizes = check(make(branch, [12] * 24, 200, branch=branch, sharp=2.0), cuda_device, 12, with_draft)
    assert len(set(sizes)) > 1                              # some stay, some do not


def test_many_siblings_of_a_poor_draft(cuda_device):
    """Every draft behind the root, from a distribution that hardly meets the target's: refusal after refusal."""
    c = make(5, [30] * 6, 300, sharp=1.0, noise=6.0)
    c["parents"][:] = np.where(c["parents"] >= 0, 0, -1)
    check(c, cuda_device, 4)
    check(c, cuda_device, 4, with_draft=False)


def test_many_nodes_and_short_paths(cuda_device):
    c = make(6, [1024, 700], 40, branch=1, noise=0.01)      # long chains that nearly all stay
    for most in (1, 2, 33, 1024):
        check(c, cuda_device, most)


@pytest.mark.parametrize("V", [50257, 131072])
def test_large_vocabularies(cuda_device, V):
    check(make(V, [3, 2], V, sharp=1.0), cuda_device, 4)


def test_rows_where_the_draft_is_the_target(cuda_device):
    c = make(7, [6] * 8, 500, noise=0.0)
    c["u"][:] = np.float32(1 - 2.0 ** -24)
    assert check(c, cuda_device, 6) and check(dict(c, u=np.zeros_like(c["u"])), cuda_device, 6)


def test_one_hot_rows(cuda_device):
    """Greedy decoding: all of the target's weight on one token, which drafts meet or not."""
    c = make(8, [7] * 10, 64, branch=2)
    c["target"] = np.eye(64, dtype=np.float32)[np.random.default_rng(1).integers(0, 4, c["target"].shape[0])]
    c["tokens"] = np.random.default_rng(2).integers(0, 4, c["tokens"].shape[0]).astype(np.int32)
    sizes = check(c, cuda_device, 7, with_draft=False)
    assert max(sizes) > 1


def test_strided_and_unaligned_rows(cuda_device):
    c = make(9, [5, 6], 301)
    dev = cuda_device
    want = [x.cpu() for x in call(c, dev, 6)]
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)
    wide = torch.full((11, 2, 333), float("nan"), device=dev)
    for pt, pd in ((3, 3), (1, 2), (0, 5)):                 # the same and other places within 16 bytes
        wide[:, 0, pt:pt + 301], wide[:, 1, pd:pd + 301] = t(c["target"]), t(c["draft"])
        got = pkv.verify_draft(wide[:, 0, pt:pt + 301], t(c["tokens"]), t(c["parents"]), t(c["start"]), t(c["u"]), 6,
                               draft_probs=wide[:, 1, pd:pd + 301])
        assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want)) and pkv.device_error() == 0


def test_leaves_draft_rows_are_not_read(cuda_device):
    c = make(10, [6, 1, 4], 100, branch=1)
    leaves = [5, 6, 10]
    want = [x.cpu() for x in call(c, cuda_device, 6)]
    c["draft"][leaves] = np.nan
    got = call(c, cuda_device, 6)
    assert pkv.device_error() == 0 and all(torch.equal(a.cpu(), b) for a, b in zip(got, want))


def test_bad_nodes_are_recorded_and_left_out(cuda_device):
    c = make(11, [6, 6], 50, branch=1)
    c["u"][:] = 0                                           # all stay
    assert check(c, cuda_device, 6) == [6, 6]
    padded = dict(c, parents=c["parents"].copy())
    padded["parents"][3] = -1                               # padding: its descendants are not reached
    assert check(padded, cuda_device, 6) == [3, 6]
    for field, value, code in (("parents", 3, 9), ("parents", 99, 9), ("tokens", 50, 10), ("tokens", -1, 10)):
        bad = dict(c, **{field: c[field].copy()})
        bad[field][3] = value
        path, size, token = call(bad, cuda_device, 6)
        assert pkv.device_error() == code and pkv.device_error() == 0
        assert size.tolist() == [3, 6] and path[0].tolist() == [0, 1, 2, -1, -1, -1]
    bad = dict(c, start=np.array([0, 6, 13], np.int32))
    path, size, token = call(bad, cuda_device, 6)
    assert pkv.device_error() == 6 and size.tolist() == [6, 0] and token[1] == -1


def test_rows_that_are_no_distributions(cuda_device):
    c = make(12, [1, 1, 1, 1, 1, 1], 2000)
    for i, row in enumerate((np.nan, -0.1, 1.5, 0.0)):
        c["target"][i, 700 if i < 3 else slice(None)] = row
    c["target"][4] *= 2
    _, size, token = call(c, cuda_device, 2)
    assert pkv.device_error() == 11 and size.tolist() == [1] * 6
    token = token.tolist()
    assert token[:5] == [-1] * 5 and token[5] >= 0


@pytest.mark.parametrize("V", [3, 256, 4096])
def test_refused_tokens_of_a_row_that_sums_to_more_than_one(cuda_device, V):
    """Without draft distributions what the refused tokens leave decides, also where the row's sum is past what the
    kernel adds up to: 2.25 less 0.75 is just not too much, 2.375 less 0.75 is."""
    c = make(16, [2], V)
    c["tokens"][:] = 0
    c["u"][:] = 0.9375                                      # refuses what has 0.75
    for third, token in ((0.75, 2), (0.875, -1)):
        c["target"][:] = 0
        c["target"][:, :2], c["target"][:, 2] = 0.75, third
        path, size, got = call(c, cuda_device, 2, with_draft=False)
        assert size.tolist() == [1] and got.tolist() == [token] and pkv.device_error() == (11 if token < 0 else 0)


def test_random_numbers_at_their_ends(cuda_device):
    c = make(14, [3] * 40, 333)
    for u in (np.float32(0), np.float32(1 - 2.0 ** -24)):
        check(dict(c, u=np.full_like(c["u"], u)), cuda_device, 3)
    # 1 is none of them: it counts as the largest below, and no draft stays by chance alone
    _, size, token = call(dict(c, u=np.ones_like(c["u"])), cuda_device, 3)
    assert ((token >= 0) & (token < 333)).all() and pkv.device_error() == 0
    _, size, token = call(dict(c, u=np.full_like(c["u"], np.nan)), cuda_device, 3)
    assert pkv.device_error() == 11 and ((token >= 0) & (token < 333)).all()


def test_captured_and_on_two_streams(cuda_device):
    cs = [make(20 + i, [9, 9, 9], 3001) for i in range(2)]
    want = [[x.clone() for x in call(c, cuda_device, 9)] for c in cs]
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(cuda_device)
    args = [[t(c[n]) for n in ("target", "tokens", "parents", "start", "u")] for c in cs]
    drafts = [t(c["draft"]) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[pkv.verify_draft(*args[i], 9, draft_probs=drafts[i], stream=st) for _ in range(4)] for i, st in enumerate(streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i in range(2) for g in got[i] for a, b in zip(g, want[i]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = pkv.verify_draft(*args[0], 9, draft_probs=drafts[0])
    for a, b in zip(args[0] + [drafts[0]], args[1] + [drafts[1]]):
        a.copy_(b)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want[1]))


@pytest.mark.parametrize("seqs", [1, 20, 200, 300, 600])   # clusters of eight, eight, four, two CTAs and of one
def test_clusters_without_nodes(cuda_device, seqs):
    """A sequence without nodes, or with rows that are none, is over as soon as its cluster runs: call upon call of
    those, between sequences that have some."""
    V = 333
    c = make(15, [0, 3, 0, 0], V)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(cuda_device)
    args = [t(c[n]) for n in ("target", "tokens", "parents")]
    empty = torch.zeros(seqs + 1, dtype=torch.int32, device=cuda_device)
    mixed = empty.clone()
    mixed[seqs // 2 + 1:] = 3                               # one sequence in the middle has all three
    bad = empty.clone()
    bad[seqs // 2 + 1:] = 4                                 # or one more than there are
    u, draft = t(c["u"]), t(c["draft"])
    want, x = od.verify(c["target"], c["draft"], c["tokens"], c["parents"], c["u"], 3)
    torch.cuda.synchronize()
    for start in (empty, mixed, bad):
        got = [pkv.verify_draft(*args, start, u, 3, draft_probs=draft if i % 2 else None) for i in range(20)]
        assert pkv.device_error() == (6 if start is bad else 0)
        for i, (path, size, token) in enumerate(got):
            some = [seqs // 2] if start is mixed else []
            rest = torch.ones(seqs, dtype=torch.bool)
            rest[some] = False
            assert (size.cpu()[rest] == 0).all() and (token.cpu()[rest] == -1).all() and (path.cpu()[rest] == -1).all()
            if some and i % 2:
                n = int(size[some[0]])
                assert path[some[0], :n].tolist() == want and int(token[some[0]]) == x


@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("seqs,V", [(120, 333), (200, 333), (300, 333), (600, 333), (600, 3), (300, 1301)])
def test_many_sequences(cuda_device, seqs, V, with_draft):
    """Clusters of eight, four, two CTAs and of one; sequences without nodes among them."""
    rng = np.random.default_rng(seqs)
    sizes = check(make(seqs + V, rng.integers(0, 5, seqs).tolist(), V, branch=3, sharp=2.0), cuda_device, 4, with_draft)
    assert len(set(sizes)) > 1


@pytest.mark.parametrize("V", [3, 130, 1000, 50257])
@pytest.mark.parametrize("refusals", [1, 2, 3, 4, 5, 7])
def test_refusals_are_rounded_in_their_sum(cuda_device, refusals, V):
    """The draft's distribution misses the target's by one step of fp32 in one token, so that every refusal leaves the
    2^24-th part of that step: 2^36, 2^12 and 1 units, and with the fourth nothing, so that the token comes from
    the whole row.  (Rounding every refusal's product by itself would leave the one unit for good.)"""
    e = 2.0 ** -24
    first, few, never = np.random.default_rng(V).choice(V, 3, replace=False)
    if few < first:
        first, few = few, first                             # the token that the whole row gives lies behind
    target, draft = np.zeros((2, V), np.float32)
    target[first], target[few] = 1 - 4 * e, 4 * e
    draft[first], draft[few], draft[never] = 1 - 5 * e, 4 * e, e
    n = refusals + 1
    c = dict(target=np.tile(target, (n, 1)), draft=np.tile(draft, (n, 1)), tokens=np.full(n, never, np.int32),
             parents=np.array([-1] + [0] * refusals, np.int32), start=np.array([0, n], np.int32), u=np.full(n, 1 - e, np.float32))
    assert od.verify(c["target"], c["draft"], c["tokens"], c["parents"], c["u"], 4) == ([0], first if refusals < 4 else few)
    check(c, cuda_device, 4)
    check(dict(c, draft=c["target"]), cuda_device, 4)       # nothing is left from the first refusal on


def test_verify_refusals(cuda_device):
    c = make(13, [4], 20)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(cuda_device)
    ok = [t(c[n]) for n in ("target", "tokens", "parents", "start", "u")] + [4]
    for i, bad in ((0, ok[0].half()), (0, ok[0].t()), (0, ok[0].cpu()), (1, ok[1].long()), (1, ok[1][:3]), (2, ok[2][:2]), (4, ok[4].double()),
                   (5, 0), (5, 2000)):
        with pytest.raises(pkv.PkvError):
            pkv.verify_draft(*ok[:i], bad, *ok[i + 1:])
    with pytest.raises(pkv.PkvError):
        pkv.verify_draft(*ok, draft_probs=t(c["draft"])[:3])


# ---- the move ------------------------------------------------------------------------------------

def move_case(seed, counts, kept, L, Hk, D, B, extra=3):
    rng = np.random.default_rng(seed)
    T = sum(counts)
    N = -(-T // B) + extra
    slots = rng.permutation(N * B)[:T].astype(np.int64)
    pools = [[rng.integers(0, 65536, (N, Hk, B, D)).astype(np.uint16).view(np.float16) for _ in range(L)] for _ in range(2)]
    path = np.full((len(counts), max(1, max(kept))), -1, np.int32)
    for s, (n, k) in enumerate(zip(counts, kept)):
        if k:
            path[s, :k] = [0] + sorted(rng.choice(np.arange(1, n), k - 1, replace=False).tolist())
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return pools, slots, start, path, np.array(kept, np.int32)


def moved(case, dev):
    (ks, vs), *rest = case
    t = lambda x: torch.from_numpy(x).to(dev)
    kd, vd = [t(x.view(np.int16)).view(torch.float16) for x in ks], [t(x.view(np.int16)).view(torch.float16) for x in vs]
    pkv.move_accepted(kd, vd, *[t(x) for x in rest])
    return kd, vd


def same(case, got):
    return all(np.array_equal(a.view(torch.int16).cpu().numpy(), b.view(np.int16)) for x, y in zip(got, case[0]) for a, b in zip(x, y))


@pytest.mark.parametrize("counts,kept,L,Hk,D,B", [
    ([1], [1], 1, 1, 64, 16),
    ([8], [5], 1, 2, 128, 4),
    ([16, 3, 0, 9], [16, 2, 0, 7], 3, 5, 64, 8),
    ([20] * 7, [1, 2, 3, 9, 10, 19, 20], 70, 1, 64, 16),     # more layers than one launch takes
    ([200, 90], [150, 80], 2, 3, 128, 32),                  # more rows than are looked up at a time
    ([12], [6], 2, 300, 128, 16),                           # a token's rows longer than a CTA's threads
])
def test_move_against_oracle(cuda_device, counts, kept, L, Hk, D, B):
    case = move_case(len(counts) + L + Hk, counts, kept, L, Hk, D, B)
    got = moved(case, cuda_device)
    assert pkv.device_error() == 0
    od.move_accepted(case[0][0], case[0][1], *case[1:])
    assert same(case, got)


def test_move_leaves_out_what_is_bad(cuda_device):
    for change, code in ((lambda c: c[1].__setitem__(slice(None), -1), 0), (lambda c: c[1].__setitem__(slice(None), 10 ** 6), 3),
                         (lambda c: c[3].__setitem__((0, slice(1, 4)), [0, 1, 99]), 9), (lambda c: c[4].__setitem__(0, 5), 6),
                         (lambda c: c[2].__setitem__(1, 99), 6)):
        case = move_case(3, [9], [4], 2, 2, 64, 16)
        change(case)
        assert same(case, moved(case, cuda_device))
        assert pkv.device_error() == code and pkv.device_error() == 0


def test_move_refusals(cuda_device):
    (ks, vs), *rest = move_case(4, [5], [3], 2, 2, 64, 16)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(cuda_device)
    k, v, r = [t(x) for x in ks], [t(x) for x in vs], [t(x) for x in rest]
    for args in (([], [], *r), (k, v[:1], *r), (k, [v[0], v[1][:1]], *r), (k, v, r[0].int(), *r[1:]), (k, v, *r[:2], r[2][0], r[3]),
                 (k, v, r[0], r[1][:1], *r[2:]), ([k[0], k[1].cpu()], v, *r)):
        with pytest.raises(pkv.PkvError):
            pkv.move_accepted(*args)


# ---- the set -------------------------------------------------------------------------------------

def test_steps_with_drafts_through_the_block_manager(cuda_device):
    """Three steps of two sequences over two layers: slots, tables and what a refused draft gives back come from
    the block manager; after each step the cache holds what writing the kept tokens one by one would."""
    dev, B, H, Hk, D, L, V = cuda_device, 8, 6, 2, 64, 2, 97
    rng = np.random.default_rng(60)
    bm = pkv.BlockManager(64, B, rng.permutation(64))
    inv = 10000.0 ** (-np.arange(D // 2) / (D // 2))
    freq = pkv.rope_frequencies(inv, dev)
    half = lambda *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float16)).to(dev)
    pools = [[torch.full((64, Hk, B, D), float("nan"), dtype=torch.float16, device=dev) for _ in range(L)] for _ in range(2)]
    # every token's projections, by (sequence, token's own number): what a model would compute for it
    history = [[], []]
    def project(n):
        return [half(n, H + 2 * Hk, D) for _ in range(L)]
    def append(seqs, qkvs, positions, slots):
        out = []
        for l in range(L):
            x = qkvs[l]
            out.append(pkv.rope_and_cache(x[:, :H], x[:, H:H + Hk], x[:, H + Hk:], positions, freq, pools[0][l], pools[1][l], slots))
        return out
    for s, n in enumerate((13, 30)):                        # prompts
        slots = torch.from_numpy(bm.add_seq(s, n)).to(dev)
        qkv = project(n)
        append([s], qkv, torch.arange(n, dtype=torch.int32, device=dev), slots)
        history[s] = [[x[i] for x in qkv] for i in range(n)]
    for step in range(3):
        counts = [int(rng.integers(4, 9)), int(rng.integers(2, 20))]
        parents = [[-1] + [int(rng.integers(max(0, j - 3), j)) for j in range(1, n)] for n in counts]
        start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        mask, depths = pkv.tree_masks(sum(parents, []), start, dev)
        before = [bm.block_table(s)[1] for s in range(2)]
        slots = []
        for s, n in enumerate(counts):
            got, copies = bm.extend(s, n)
            assert len(copies) == 0
            slots.append(got)
        slots = torch.from_numpy(np.concatenate(slots)).to(dev)
        tables, lens = bm.block_tables([0, 1], 16)
        qkv = project(sum(counts))
        base = torch.from_numpy(np.repeat(before, counts).astype(np.int32)).to(dev)
        qs = append([0, 1], qkv, base + depths, slots)
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)
        for l in range(L):
            out = pkv.paged_attention_tree(qs[l], pools[0][l], pools[1][l], t(tables), t(lens), t(start), D ** -0.5, B, max(counts),
                                           tree_mask=mask)
            want = od.tree_attention(qs[l].cpu().numpy(), pools[0][l].cpu().numpy(), pools[1][l].cpu().numpy(), tables, lens, start,
                                     [od.ancestors(p) for p in parents], D ** -0.5)
            assert np.abs(out.cpu().numpy() - want).max() < 4e-3
        c = make(61 + step, counts, V)
        c["parents"] = np.array(sum(parents, []), np.int32)
        path, size, token = call(c, dev, max(counts))
        pkv.move_accepted(pools[0], pools[1], slots, t(start), path, size)
        assert pkv.device_error() == 0
        path, size = path.cpu().numpy(), size.cpu().numpy()
        for s in range(2):
            bm.truncate(s, counts[s] - int(size[s]))
            history[s] += [[x[start[s] + j] for x in qkv] for j in path[s, :size[s]]]
            # the cache, read through the table, against the tokens' rows written one after another
            table, n = bm.block_table(s)
            assert n == before[s] + size[s] == len(history[s])
            for l in range(L):
                rows = torch.stack([h[l] for h in history[s]])
                _, k = pkv.qk_norm_rope(rows[:, :H].contiguous(), rows[:, H:H + Hk].contiguous(), torch.arange(n, dtype=torch.int32, device=dev), freq)
                tab = np.array(table)
                for pool, x in ((pools[0][l], k), (pools[1][l], rows[:, H + Hk:])):
                    have = oa.gather_sequence(pool.cpu().numpy(), tab, n)
                    assert np.array_equal(have, x.cpu().numpy().astype(np.float64))


def test_a_captured_step_of_all_four(cuda_device):
    """A step over three layers as one graph, its products' output and the appended rows read by the next call without
    a wait between them; replayed with other inputs in the same buffers, it gives what the calls one by one give."""
    dev, B, H, Hk, D, L, V = cuda_device, 16, 8, 2, 128, 3, 501
    counts, ctx = [9, 1, 17, 4], [700, 33, 17, 2100]
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    T, blocks = int(start[-1]), -(-max(ctx) // B)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)
    freq = pkv.rope_frequencies(10000.0 ** (-np.arange(D // 2) / (D // 2)), dev)
    N = len(counts) * blocks + 2

    def inputs(seed):
        rng = np.random.default_rng(seed)
        tables = rng.permutation(N)[:len(counts) * blocks].reshape(len(counts), blocks).astype(np.int32)
        parents = [[-1] + [int(rng.integers(max(0, j - 3), j)) for j in range(1, n)] for n in counts]
        mask, depths = pkv.tree_masks(sum(parents, []), start, dev)
        base = np.repeat(np.array(ctx) - counts, counts).astype(np.int32)
        slots = [int(tables[s, (ctx[s] - n + i) // B]) * B + (ctx[s] - n + i) % B for s, n in enumerate(counts) for i in range(n)]
        c = make(seed, counts, V)
        return dict(qkv=t(rng.standard_normal((L, T, H + 2 * Hk, D)).astype(np.float16)), tables=t(tables), mask=mask,
                    positions=t(base) + depths, slots=t(np.array(slots, np.int64)), parents=t(np.array(sum(parents, []), np.int32)),
                    pools=t(rng.standard_normal((2, L, N, Hk, B, D)).astype(np.float16)),
                    **{n: t(c[n]) for n in ("target", "draft", "tokens", "u")})

    lens, begin = t(np.array(ctx, np.int32)), t(start)

    def step(x):
        ks, vs = [list(p) for p in x["pools"]]
        outs = []
        for l in range(L):
            y = x["qkv"][l]
            q = pkv.rope_and_cache(y[:, :H], y[:, H:H + Hk], y[:, H + Hk:], x["positions"], freq, ks[l], vs[l], x["slots"])
            outs.append(pkv.paged_attention_tree(q, ks[l], vs[l], x["tables"], lens, begin, D ** -0.5, B, max(counts), tree_mask=x["mask"]))
        kept = pkv.verify_draft(x["target"], x["tokens"], x["parents"], begin, x["u"], 17, draft_probs=x["draft"])
        pkv.move_accepted(ks, vs, x["slots"], begin, kept[0], kept[1])
        return [*outs, *kept, x["pools"]]

    want = [[y.clone() for y in step(inputs(seed))] for seed in (70, 71, 72)]
    x = inputs(70)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(x)
    for seed in (71, 72, 70):
        for name, y in inputs(seed).items():
            x[name].copy_(y)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[seed - 70])), seed
    assert pkv.device_error() == 0
