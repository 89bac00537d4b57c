"""The oracle of drafted tokens against facts fixed outside it, and the host helpers against the oracle."""
import numpy as np
import pytest
import torch

from oracle import drafts as od
from oracle.block_manager import BlockManager as OracleManager
from paged_kv_cache_73_gb300 import _build
from paged_kv_cache_73_gb300 import binding as pkv


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return pkv.load()


def random_parents(rng, n):
    return [-1] + [int(rng.integers(0, j)) for j in range(1, n)]


def test_a_chains_attention_is_causal():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 6, 2, 8)), rng.standard_normal((4, 2, 4, 8)), rng.standard_normal((4, 2, 4, 8))
    table, n, ctx = np.array([[2, 0, 3]]), 6, 11
    got = od.tree_attention(q[0], k, v, table, [ctx], [0, n], [od.ancestors([-1, 0, 1, 2, 3, 4])], 0.3)
    keys = np.concatenate([k[b].transpose(1, 0, 2) for b in table[0]])[:ctx]
    vals = np.concatenate([v[b].transpose(1, 0, 2) for b in table[0]])[:ctx]
    for i in range(n):
        m = ctx - n + i + 1
        want = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(q[0, i])[:, None], torch.from_numpy(keys[:m]).transpose(0, 1),
            torch.from_numpy(vals[:m]).transpose(0, 1), scale=0.3)[:, 0].numpy()
        assert np.allclose(got[i], want, atol=1e-12)


def test_siblings_do_not_see_each_other():
    seen = od.ancestors([-1, 0, 0, 2, 1])
    assert seen.tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 0, 1, 1, 0], [1, 1, 0, 0, 1]]


@pytest.mark.parametrize("with_draft", [True, False])
def test_kept_and_drawn_tokens_are_the_targets(with_draft):
    """Two drafts behind the root (drawn from q, or fixed) and the next token: over a fine grid of all random
    numbers the first token that follows the root has exactly the target's probability."""
    p, q = np.array([0.5, 0.25, 0.125, 0.125], np.float32), np.array([0.125, 0.375, 0.375, 0.125], np.float32)
    grid = (np.arange(16) + 0.5) / 16
    share = np.zeros(4)
    pairs = [(x, y, float(q[x] * q[y])) for x in range(4) for y in range(4)] if with_draft else [(2, 0, 1.0)]
    target = np.stack([p, np.eye(4, dtype=np.float32)[0], np.eye(4, dtype=np.float32)[0]])
    draft = np.stack([q, q, q]) if with_draft else None
    for x, y, chance in pairs:
        for u1 in grid:
            for u2 in grid:
                for u0 in grid:
                    path, tok = od.verify(target, draft, [0, x, y], [-1, 0, 0], [u0, u1, u2], 3)
                    first = tok if len(path) == 1 else (x, y)[path[1] - 1]
                    share[first] += chance / 16 ** 3
    # the grid's step bounds what the borders between outcomes can move
    assert np.abs(share - p).max() < 3 / 16 / 4
    assert abs(share.sum() - 1) < 1e-9


def test_a_draft_like_the_target_always_stays():
    p = np.array([0.25, 0.5, 0.25], np.float32)
    path, tok = od.verify(np.stack([p, p, p]), np.stack([p, p, p]), [0, 2, 1], [-1, 0, 1], [0.5, 0.999, 0.999], 8)
    assert path == [0, 1, 2] and tok == 1
    assert od.verify(np.stack([p, p, p]), np.stack([p, p, p]), [0, 2, 1], [-1, 0, 1], [0.5, 0.9, 0.9], 2)[0] == [0, 1]


@pytest.mark.parametrize("refusals", [1, 2, 3, 4, 6])
def test_what_refusals_take_is_rounded_once(refusals):
    """p = 1 - 2^-22 and q = p - 2^-24 on token 0: with C_1 = 1 and C_k+1 = C_k + M_k, floor(C_k q) leaves 2^36, 2^12, 1 and
    0 units of 2^-60, worked out by hand; the rest of the row is covered by q."""
    e = 2.0 ** -24
    p, q = np.array([1 - 4 * e, 4 * e, 0], np.float32), np.array([1 - 5 * e, 4 * e, e], np.float32)
    n = refusals + 1
    path, token = od.verify(np.stack([p] * n), np.stack([q] * n), [2] * n, [-1] + [0] * refusals, [1 - e] * n, 4)
    assert path == [0] and token == (0 if refusals < 4 else 1)


def test_a_row_that_leaves_nothing_falls_back_on_the_target():
    p, q = np.array([0.25, 0.75], np.float32), np.array([0.5, 1.0], np.float32)   # q covers p: nothing is left
    path, tok = od.verify(p[None].repeat(2, 0), q[None].repeat(2, 0), [0, 0], [-1, 0], [0.3, 0.9], 4)
    assert path == [0] and tok == 1


def test_move_reads_before_it_writes():
    pool = np.arange(2 * 1 * 4 * 1, dtype=np.float16).reshape(2, 1, 4, 1)
    k, v = pool.copy(), -pool
    od.move_accepted([k], [v], [1, 2, 3, 4, 5], [0, 5], [[0, 2, 3, -1]], [3])
    assert k.ravel().tolist() == [0, 1, 3, 4, 4, 5, 6, 7] and (v == -k).all()


def test_tree_masks_match_the_oracle():
    rng = np.random.default_rng(2)
    counts = [1, 0, 33, 64, 5, 70]
    parents = [random_parents(rng, n) for n in counts if n]
    start = np.concatenate([[0], np.cumsum(counts)])
    masks, depths = pkv.tree_masks(sum(parents, []), start, device="cpu")
    assert masks.shape == (sum(counts), 3)
    bits = (masks.numpy().view(np.uint32)[:, :, None] >> np.arange(32, dtype=np.uint32) & 1).reshape(sum(counts), -1).astype(bool)
    row = 0
    for par in parents:
        seen, n = od.ancestors(par), len(par)
        assert (bits[row:row + n, :n] == seen).all() and not bits[row:row + n, n:].any()
        assert (depths.numpy()[row:row + n] == seen.sum(1) - 1).all()
        row += n


def test_tree_masks_refuse_bad_trees():
    for parents, start in (([-1, 1], [0, 2]), ([-1, 2, 0], [0, 3]), ([-1], [0, 2]), ([-1], [1, 1])):
        with pytest.raises(pkv.PkvError):
            pkv.tree_masks(parents, start, device="cpu")


def test_tree_masks_look_at_all_starts_before_any_parent(lib):
    """The parents end at query_start's last entry: a start before it that is larger, or a decreasing one behind, is refused
    without reading past them (what lies there would be refused in another way)."""
    past = np.full(64, 99, np.int32)
    past[0] = -1
    for start in ([0, 40, 1], [0, 1, 60, 1], [0, 1, -5, 1], [-1, 1]):
        st, masks = np.array(start, np.int32), np.full((64, 4), 7, np.int32)
        assert lib.pkv_tree_masks(past.ctypes.data, st.ctypes.data, len(st) - 1, 4, masks.ctypes.data, None) == pkv.PKV_ERR_INVALID_ARG
        assert b"nodes from" in lib.pkv_last_error() and (masks == 7).all(), lib.pkv_last_error()
    with pytest.raises(pkv.PkvError):
        pkv.tree_masks([-1], [0, 40, 1], device="cpu")


@pytest.mark.parametrize("B", [4, 16])
def test_truncate_matches_the_oracle(B):
    rng = np.random.default_rng(B)
    mine, theirs = pkv.BlockManager(40, B), OracleManager(40, B)
    for s in range(3):
        assert mine.add_seq(s, 3 * s + 2).tolist() == theirs.add_seq(s, 3 * s + 2)
    mine.fork(2, 3), theirs.fork(2, 3)
    for _ in range(200):
        s = int(rng.integers(0, 4))
        if rng.random() < 0.5:
            n = int(rng.integers(0, 9))
            try:
                want = theirs.extend(s, n)
            except MemoryError:
                with pytest.raises(pkv.PkvOutOfBlocks):
                    mine.extend(s, n)
                continue
            got = mine.extend(s, n)
            assert got[0].tolist() == want[0] and [tuple(p) for p in got[1].tolist()] == want[1]
        else:
            n = int(rng.integers(0, theirs.block_table(s)[1]))
            mine.truncate(s, n), theirs.truncate(s, n)
        assert mine.block_table(s) == theirs.block_table(s)
        assert mine.stats()[0] == theirs.num_free() and mine.ref_histogram(8).tolist() == theirs.ref_histogram(8)


def test_truncate_refuses():
    bm = pkv.BlockManager(4, 4)
    bm.add_seq(1, 6)
    for args, status in (((2, 1), pkv.PKV_ERR_NOT_FOUND), ((1, 6), pkv.PKV_ERR_INVALID_ARG), ((1, -1), pkv.PKV_ERR_INVALID_ARG)):
        with pytest.raises(pkv.PkvError) as e:
            bm.truncate(*args)
        assert e.value.status == status
    assert bm.block_table(1)[1] == 6


# ---- refusals of the device entry points, on the host ----------------------------------------------

def rope(lib, **kw):
    a = dict(q=16, k=16, v=16, qw=None, kw=None, eps=1e-6, pos=16, axes=1, fr=16, ax=None, R=64, inter=0, rs=1.0, T=2, H=4,
             Hk=2, D=64, qs=256, ks=128, vs=128, qo=16, qos=256, kc=16, vc=16, slots=16, B=16, N=4)
    a.update(kw)
    return lib.pkv_rope_and_cache(*[a[n] for n in ("q k v qw kw eps pos axes fr ax R inter rs T H Hk D qs ks vs qo qos kc "
                                                   "vc slots B N").split()], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), pkv.PKV_OK), (dict(T=-1), pkv.PKV_ERR_INVALID_ARG), (dict(D=96), pkv.PKV_ERR_UNSUPPORTED),
    (dict(B=12), pkv.PKV_ERR_UNSUPPORTED), (dict(R=24), pkv.PKV_ERR_UNSUPPORTED), (dict(R=128), pkv.PKV_ERR_UNSUPPORTED),
    (dict(N=0), pkv.PKV_ERR_INVALID_ARG), (dict(rs=float("nan")), pkv.PKV_ERR_INVALID_ARG),
    (dict(slots=None), pkv.PKV_ERR_INVALID_ARG), (dict(kc=24), pkv.PKV_ERR_INVALID_ARG), (dict(v=None), pkv.PKV_ERR_INVALID_ARG),
    (dict(vs=120), pkv.PKV_ERR_INVALID_ARG), (dict(ks=132), pkv.PKV_ERR_INVALID_ARG), (dict(qos=264), pkv.PKV_ERR_INVALID_ARG),
    (dict(eps=-1.0), pkv.PKV_ERR_INVALID_ARG), (dict(axes=9), pkv.PKV_ERR_UNSUPPORTED),
])
def test_rope_and_cache_refuses(lib, kw, status):
    assert rope(lib, **kw) == status


def tree(lib, **kw):
    a = dict(q=16, qs=256, k=16, v=16, tab=16, lens=16, start=16, mask=None, words=0, S=2, T=4, most=2, H=4, Hk=2, D=64,
             N=8, maxb=4, scale=0.125, B=16, out=16, ws=None, wsb=0)
    a.update(kw)
    return lib.pkv_paged_attention_tree(*[a[n] for n in ("q qs k v tab lens start mask words S T most H Hk D N maxb scale B out "
                                                         "ws wsb").split()], None)


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), pkv.PKV_OK), (dict(T=0), pkv.PKV_OK), (dict(most=0), pkv.PKV_OK), (dict(H=3), pkv.PKV_ERR_INVALID_ARG),
    (dict(D=80), pkv.PKV_ERR_UNSUPPORTED), (dict(B=64), pkv.PKV_ERR_UNSUPPORTED), (dict(scale=0.0), pkv.PKV_ERR_INVALID_ARG),
    (dict(scale=float("inf")), pkv.PKV_ERR_INVALID_ARG), (dict(mask=16), pkv.PKV_ERR_INVALID_ARG),
    (dict(mask=16, words=1, most=33), pkv.PKV_ERR_INVALID_ARG), (dict(q=24), pkv.PKV_ERR_INVALID_ARG),
    (dict(qs=248), pkv.PKV_ERR_INVALID_ARG), (dict(qs=260), pkv.PKV_ERR_INVALID_ARG), (dict(start=None), pkv.PKV_ERR_INVALID_ARG),
    (dict(maxb=1 << 28), pkv.PKV_ERR_UNSUPPORTED), (dict(out=None), pkv.PKV_ERR_INVALID_ARG),
    (dict(S=70000), pkv.PKV_ERR_UNSUPPORTED),
])
def test_paged_attention_tree_refuses(lib, kw, status):
    assert tree(lib, **kw) == status


def verify(lib, **kw):
    a = dict(t=16, d=None, tok=16, par=16, start=16, u=16, S=2, T=4, V=100, ts=100, ds=0, most=4, path=16, size=16, nxt=16)
    a.update(kw)
    return lib.pkv_verify_draft(*[a[n] for n in "t d tok par start u S T V ts ds most path size nxt".split()], None)


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), pkv.PKV_OK), (dict(V=0), pkv.PKV_ERR_INVALID_ARG), (dict(most=0), pkv.PKV_ERR_INVALID_ARG),
    (dict(most=1025), pkv.PKV_ERR_UNSUPPORTED), (dict(ts=99), pkv.PKV_ERR_INVALID_ARG), (dict(d=16, ds=99), pkv.PKV_ERR_INVALID_ARG),
    (dict(u=None), pkv.PKV_ERR_INVALID_ARG), (dict(path=None), pkv.PKV_ERR_INVALID_ARG), (dict(T=0, start=None), pkv.PKV_ERR_INVALID_ARG),
    (dict(V=1 << 25, ts=1 << 25), pkv.PKV_ERR_UNSUPPORTED),
])
def test_verify_draft_refuses(lib, kw, status):
    assert verify(lib, **kw) == status


def move(lib, **kw):
    import ctypes
    a = dict(k=(16, 32), v=(48, 64), L=2, slots=16, start=16, path=16, size=16, S=2, T=8, most=4, Hk=2, D=64, B=16, N=4)
    a.update(kw)
    arr = lambda x: None if x is None else (ctypes.c_void_p * len(x))(*x)
    return lib.pkv_move_accepted(arr(a["k"]), arr(a["v"]), *[a[n] for n in "L slots start path size S T most Hk D B N".split()], None)


@pytest.mark.parametrize("kw", [dict(k=(16, 16)), dict(v=(48, 48)), dict(v=(48, 16)), dict(k=(64, 32))])
def test_move_accepted_refuses_a_pool_twice(lib, kw):
    """Layers that share their cache, or keys that are the values: its rows would be moved twice."""
    assert move(lib, **kw) == pkv.PKV_ERR_INVALID_ARG and b"twice" in lib.pkv_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), pkv.PKV_OK), (dict(L=0), pkv.PKV_ERR_INVALID_ARG), (dict(k=None), pkv.PKV_ERR_INVALID_ARG),
    (dict(v=(48, 8)), pkv.PKV_ERR_INVALID_ARG), (dict(D=32), pkv.PKV_ERR_UNSUPPORTED), (dict(B=2), pkv.PKV_ERR_UNSUPPORTED),
    (dict(path=None), pkv.PKV_ERR_INVALID_ARG), (dict(most=0), pkv.PKV_ERR_INVALID_ARG), (dict(N=0), pkv.PKV_ERR_INVALID_ARG),
])
def test_move_accepted_refuses(lib, kw, status):
    assert move(lib, **kw) == status
