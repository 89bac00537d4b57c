"""Paged decode attention over the four-bit cache against the fp64 oracle on the same pools.

Tolerance per value, derived.  With P = sum p = 1 after normalisation, span = the largest scale times 15
over the context (every stored value lies within it), a = sum p |v|: the fp16 rounding of the output is
2^-11 |o| (2^-25 below the normals); each weight's rounding, 2^-11 of it, meets at most 8 steps of its
row: 2^-11 * 8/15 * span; the logits' fp32 error dx (2^-23 times the sum of |terms|, and 2^-22 from exp2)
moves the weights by that much relative: dx * 2 a."""
import numpy as np
import pytest
import torch

from oracle import int4_cache as o4
from paged_kv_cache_73_gb300 import binding as pkv

pytestmark = pytest.mark.gpu


def make(seed, lens, H, Hk, D, B, dev, row_scale=None, q_scale=1.0, extra=3):
    """Random pools: only the sequences' rows are ordinary; every other slot's scale is NaN."""
    rng = np.random.default_rng(seed)
    blocks = [-(-n // B) for n in lens]
    N = sum(blocks) + extra
    ids = rng.permutation(N).astype(np.int32)
    maxb = max(1, max(blocks))
    tables = np.full((len(lens), maxb), -1, np.int32)
    pools = []
    at = 0
    for s, b in enumerate(blocks):
        tables[s, :b] = ids[at:at + b]
        at += b
    for _ in range(2):
        rows = rng.standard_normal((N * B, Hk, D))
        if row_scale is not None:
            rows = row_scale(rng, rows)
        pool = o4.empty_pool(N, Hk, B, D)
        n, sc, z = o4.quantise_rows(np.clip(rows, -65504, 65504).astype(np.float16).reshape(N, B, Hk, D).transpose(0, 2, 1, 3))
        pool[:, :, :B * D // 2] = (n[..., 0::2] | (n[..., 1::2] << 4)).reshape(N, Hk, -1)
        live = np.zeros((N, B), bool)
        for s, ln in enumerate(lens):
            for t in range(ln):
                live[tables[s, t // B], t % B] = True
        meta = np.stack([sc, z], -1)                          # [N, Hk, B, 2]
        meta[~live[:, None, :].repeat(Hk, 1)] = np.nan
        pool[:, :, B * D // 2:] = meta.reshape(N, Hk, -1).view(np.uint8)
        pools.append(pool)
    q = (rng.standard_normal((len(lens), H, D)) * q_scale).astype(np.float16)
    return q, pools[0], pools[1], tables, np.array(lens, np.int32)


def run(case, scale, B, dev, **kw):
    return pkv.paged_attention_decode_int4(*(torch.from_numpy(x).to(dev) for x in case), scale, B, **kw)


def tolerance(case, want, scale, B):
    q, kc, vc, tables, lens = case
    group = q.shape[1] // kc.shape[1]
    v = o4.pool_values(vc, B)
    meta = np.ascontiguousarray(vc[:, :, B * q.shape[2] // 2:]).view(np.float16).reshape(vc.shape[0], vc.shape[1], B, 2)
    k = o4.pool_values(kc, B)
    kmeta = np.ascontiguousarray(kc[:, :, B * q.shape[2] // 2:]).view(np.float16).reshape(vc.shape[0], vc.shape[1], B, 2)
    tol = np.zeros_like(want)
    for s, n in enumerate(lens):
        if n == 0:
            continue
        t = np.arange(n)
        blk, row = tables[s][t // B], t % B
        vs, sc = v[blk, :, row], meta[blk, :, row][..., 0].astype(np.float64)       # [n, Hk, D], [n, Hk]
        ks, km = k[blk, :, row], kmeta[blk, :, row].astype(np.float64)
        for h in range(q.shape[1]):
            qh = q[s, h].astype(np.float64)
            x = scale * ks[:, h // group] @ qh
            p = np.exp(x - x.max())
            p /= p.sum()
            a = p @ np.abs(vs[:, h // group])
            # |terms| of a logit: whole numbers up to 15 times |q|, the zero point times |sum q|'s terms
            terms = abs(scale) * np.abs(qh).sum() * (15 * km[:, h // group, 0] + np.abs(km[:, h // group, 1])).max()
            dx = 2.0 ** -23 * 4 * terms + 2.0 ** -21
            step = (p * sc[:, h // group]).sum()
            tol[s, h] = (2.0 ** -11 * np.abs(want[s, h]) + 2.0 ** -25 + 2.0 ** -11 * 8 * step
                         + 2 * dx * (a + 2.0 ** -11 * 8 * step) + 2.0 ** -20 * (15 * step + a))
    return tol


def check(case, B, dev, scale=None, **kw):
    scale = case[0].shape[2] ** -0.5 if scale is None else scale
    want = o4.paged_decode_attention(*case, scale, B)
    got = run(case, scale, B, dev, **kw).cpu().numpy().astype(np.float64)
    code = pkv.device_error()
    assert code == 0, pkv.DEV_CODES[code]
    err, tol = np.abs(got - want), tolerance(case, want, scale, B)
    assert np.isfinite(got).all() and (err <= tol).all(), float((err / np.maximum(tol, 1e-30)).max())
    return got


LENS = [0, 1, 2, 7, 15, 16, 17, 31, 32, 33, 63, 127, 128, 129, 130, 257, 500]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [4, 8, 16, 32])
def test_ragged_lengths(cuda_device, D, B):
    check(make(D + B, LENS, 3, 3, D, B, cuda_device), B, cuda_device)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 9, 16, 17, 40])
def test_grouped_heads(cuda_device, D, group):
    check(make(group + D, [1, 40, 300], 2 * group, 2, D, 16, cuda_device), 16, cuda_device)


@pytest.mark.parametrize("seqs,ctx,H,Hk", [(1, 2048, 8, 8), (1, 5000, 4, 1), (3, 1500, 64, 8), (160, 700, 2, 1)])
def test_split_contexts(cuda_device, seqs, ctx, H, Hk):
    lens = [ctx - 37 * i % ctx for i in range(seqs)]
    check(make(seqs + ctx, lens, H, Hk, 128, 16, cuda_device), 16, cuda_device)


def _mixed(rng, rows):
    rows = rows * 10.0 ** rng.uniform(-3.5, 1.5, rows.shape[:2] + (1,))
    rows[::5] = rows[::5, :, :1]                            # flat rows: scale 0
    return rows + rng.choice([0, 0, 3.0], rows.shape[:2] + (1,))


def test_rows_of_many_sizes(cuda_device):
    check(make(21, [900, 33, 260], 4, 2, 128, 16, cuda_device, row_scale=_mixed), 16, cuda_device)


@pytest.mark.parametrize("size", [2.0 ** -13, 2.0 ** 9])
def test_tiny_and_large_values(cuda_device, size):
    # tiny: the scales are subnormal fp16 numbers; large: logits far apart, one token takes all
    check(make(22, [400, 70], 2, 2, 64, 8, cuda_device, row_scale=lambda r, x: x * size), 8, cuda_device)


@pytest.mark.parametrize("q_scale", [0.0, 2.0 ** -20, 30.0])
def test_queries_of_any_size(cuda_device, q_scale):
    check(make(23, [300, 5], 4, 2, 128, 16, cuda_device, q_scale=q_scale), 16, cuda_device)


def test_negative_and_zero_scale(cuda_device):
    case = make(24, [200, 3], 2, 2, 64, 16, cuda_device)
    check(case, 16, cuda_device, scale=-0.3)
    check(case, 16, cuda_device, scale=0.0)


def test_rising_logits_move_the_maximum(cuda_device):
    def ramp(rng, rows):
        rows *= 0.05
        rows[:, :, 0] += np.linspace(0, 60, rows.shape[0])[:, None]
        return rows
    # the pool's rows rise with the block number: sorted tables give a context whose logits rise by 240
    _, kc, vc, tables, _ = make(25, [63 * 16], 2, 2, 64, 16, cuda_device, row_scale=ramp)
    q = np.zeros((1, 2, 64), np.float16)
    q[..., 0] = 4
    check((q, kc, vc, np.sort(tables, axis=1), np.array([1000], np.int32)), 16, cuda_device)


def test_bad_blocks_and_lengths_are_recorded(cuda_device):
    case = list(make(26, [40, 300, 30], 2, 2, 64, 16, cuda_device))
    want = o4.paged_decode_attention(*case, 0.125, 16)
    tables = case[3].copy()
    tables[1, 2], tables[0, 3:] = case[1].shape[0], 10 ** 6  # past the context: never looked at
    case[3] = tables
    got = run(case, 0.125, 16, cuda_device).cpu().numpy().astype(np.float64)
    assert pkv.device_error() == 1 and pkv.device_error() == 0
    tol = tolerance((case[0][[0, 2]], case[1], case[2], tables[[0, 2]], case[4][[0, 2]]), want[[0, 2]], 0.125, 16)
    assert (np.abs(got[[0, 2]] - want[[0, 2]]) <= tol).all() and np.isfinite(got).all()
    case[4] = np.array([40, tables.shape[1] * 16 + 1, -1], np.int32)
    got = run(case, 0.125, 16, cuda_device)
    assert pkv.device_error() == 2 and not got[1:].any()


def test_captured_replayed_and_other_stream(cuda_device):
    case = make(27, [700, 1900, 12], 8, 2, 128, 16, cuda_device)
    dev = [torch.from_numpy(x).to(cuda_device) for x in case]
    n = pkv.paged_attention_int4_workspace_size(3, 8, 2, 128, case[3].shape[1], 16)
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device=cuda_device)
    out = torch.zeros_like(dev[0])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        pkv.paged_attention_decode_int4(*dev, 0.1, 16, out=out, workspace=ws)
    dev[4][0] = 650                                         # the lengths are read at replay
    g.replay()
    with torch.cuda.stream(st):
        g.replay()
        direct = pkv.paged_attention_decode_int4(*dev, 0.1, 16)
    torch.cuda.synchronize()
    assert pkv.device_error() == 0 and torch.equal(out, direct)
    case = case[:4] + (np.array([650, 1900, 12], np.int32),)
    want = o4.paged_decode_attention(*case, 0.1, 16)
    assert (np.abs(out.cpu().numpy() - want) <= tolerance(case, want, 0.1, 16)).all()


def test_workspace_and_shapes_refused(cuda_device):
    case = make(28, [700, 1900], 8, 2, 128, 16, cuda_device)
    dev = [torch.from_numpy(x).to(cuda_device) for x in case]
    n = pkv.paged_attention_int4_workspace_size(2, 8, 2, 128, case[3].shape[1], 16)
    with pytest.raises(pkv.PkvError) as e:
        pkv.paged_attention_decode_int4(*dev, 0.1, 16, workspace=torch.empty(n - 64, dtype=torch.uint8, device=cuda_device))
    assert e.value.status == pkv.PKV_ERR_WORKSPACE
    for bad in (dict(q=dev[0][:, :7].contiguous()), dict(q=dev[0][..., :64].contiguous()), dict(context_lens=dev[4][:1]),
                dict(out=dev[0][:, :4].contiguous()), dict(block_size=8)):
        a = dict(q=dev[0], k_cache=dev[1], v_cache=dev[2], block_tables=dev[3], context_lens=dev[4], scale=0.1, block_size=16)
        with pytest.raises(pkv.PkvError):
            pkv.paged_attention_decode_int4(**{**a, **bad})


def test_no_sequences(cuda_device):
    case = make(29, [5], 2, 2, 64, 16, cuda_device)
    dev = [torch.from_numpy(x).to(cuda_device) for x in case]
    assert pkv.paged_attention_decode_int4(dev[0][:0], dev[1], dev[2], dev[3][:0], dev[4][:0], 0.1, 16).shape[0] == 0


def test_a_pool_past_4_gib(cuda_device):
    # offsets past 32 bits: the sequence's blocks are the last of a pool of 5 GB
    case = make(30, [200], 40, 40, 128, 32, cuda_device, extra=0)
    n = (5 << 30) // (40 * 32 * 68)
    big = [torch.zeros(n, *case[1].shape[1:], dtype=torch.uint8, device=cuda_device) for _ in range(2)]
    k = case[1].shape[0]
    for b, pool in zip(big, case[1:3]):
        b[n - k:] = torch.from_numpy(pool).to(cuda_device)
    tables = torch.from_numpy(case[3] + (n - k)).to(cuda_device)
    got = pkv.paged_attention_decode_int4(torch.from_numpy(case[0]).to(cuda_device), *big, tables,
                                          torch.from_numpy(case[4]).to(cuda_device), 0.1, 32)
    assert pkv.device_error() == 0
    want = o4.paged_decode_attention(*case, 0.1, 32)
    assert (np.abs(got.cpu().numpy() - want) <= tolerance(case, want, 0.1, 32)).all()


@pytest.mark.parametrize("H,Hk", [(3, 3), (4, 1)])
def test_many_sequences(cuda_device, H, Hk):
    # more sequences than the joining kernel's threads, a third of them empty
    rng = np.random.default_rng(31)
    lens = [int(x) for x in rng.choice([0, 1, 40, 300], 300)]
    check(make(31, lens, H, Hk, 64, 16, cuda_device), 16, cuda_device)


def test_two_streams_at_once(cuda_device):
    cases = [make(32 + i, [900, 33, 1500, 5], 8, 8 >> (2 * i), 128, 16, cuda_device) for i in range(2)]
    dev = [[torch.from_numpy(x).to(cuda_device) for x in c] for c in cases]
    alone = [pkv.paged_attention_decode_int4(*d, 0.1, 16) for d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dev]
    got = [[pkv.paged_attention_decode_int4(*d, 0.1, 16, stream=st) for d, st in zip(dev, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
    assert all(torch.equal(g, a) for pair in got for g, a in zip(pair, alone))


@pytest.mark.parametrize("H,Hk", [(8, 1), (2, 2)])
def test_error_does_not_grow_with_the_context(cuda_device, H, Hk):
    # A rounding's error is uniform within half a step, 2^-11 of the value at most: 2^-11 / sqrt(3) of it in
    # the 2-norm.  The output has one; each weight has one of its own (with a lone head 2^-11 less), which
    # meets s (n - 8) of its row: the 2-norm of p s (n - 8) over the tokens against the output's.  A fifth
    # more for the spread of 512 or 128 values' norms, 2^-16 for fp32.
    case = make(33, [40000], H, Hk, 64, 16, cuda_device)
    q, kc, vc, tables, lens = case
    want = o4.paged_decode_attention(*case, 0.125, 16)
    got = run(case, 0.125, 16, cuda_device).cpu().numpy().astype(np.float64)
    assert pkv.device_error() == 0
    t = np.arange(40000)
    blk, row = tables[0][t // 16], t % 16
    k, v = (o4.pool_values(x, 16)[blk, :, row] for x in (kc, vc))
    meta = np.ascontiguousarray(vc[:, :, 16 * 32:]).view(np.float16).reshape(vc.shape[0], Hk, 16, 2)[blk, :, row]
    sc, zero = meta[..., 0].astype(np.float64), meta[..., 1].astype(np.float64)
    part = 0.0
    for h in range(H):
        g = h * Hk // H
        x = 0.125 * k[:, g] @ q[0, h].astype(np.float64)
        p = np.exp(x - x.max())
        p /= p.sum()
        part += ((p[:, None] * (v[:, g] - zero[:, g, None] - 8 * sc[:, g, None])) ** 2).sum()
    part /= (want ** 2).sum()
    rounding = 2.0 ** -11 / 3 ** 0.5
    limit = 1.2 * rounding * (1 + (part if H > Hk else 0)) ** 0.5 + 2.0 ** -16
    off = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert off <= limit, (off, limit)


@pytest.mark.parametrize("lens,H,Hk,D,B", [([140000], 2, 1, 128, 16), ([0, 50000, 3, 30000], 8, 2, 64, 32),
                                           ([100] * 40 + [60000], 4, 1, 128, 16), ([20000], 40, 1, 64, 16)])
def test_streams_cut_into_many_parts(cuda_device, lens, H, Hk, D, B):
    # a stream over a thousand warps; beside empty and short ones; many heads on one
    check(make(34, lens, H, Hk, D, B, cuda_device), B, cuda_device)


@pytest.mark.parametrize("H,Hk", [(2, 2), (6, 2), (12, 1), (40, 2)])
@pytest.mark.parametrize("D,B", [(64, 4), (128, 8), (128, 16), (64, 32)])
def test_bad_blocks_have_no_weight(cuda_device, H, Hk, D, B):
    # scattered bad blocks, whole chunks of them, the first, the last, every one of a sequence; one short
    # sequence without any and a long one that many warps share
    rng = np.random.default_rng(D + B + H)
    case = make(D + B + H, [300, 70, 5, 33, 4000, 31], H, Hk, D, B, cuda_device)
    q, kc, vc, tables, lens = case
    blocks = [-(-int(n) // B) for n in lens]
    bad = [rng.random(b) < 0.2 for b in blocks]
    bad[0][0] = bad[1][-1] = True
    bad[2][:] = False
    bad[3][:] = True
    bad[4][500 // B:3000 // B] = True
    broken, kept, left = tables.copy(), np.full_like(tables, -1), []
    for s, b in enumerate(bad):
        broken[s, :blocks[s]][b] = rng.choice([-1, -7, kc.shape[0], 2 ** 31 - 1], b.sum())
        good = tables[s, :blocks[s]][~b]
        kept[s, :len(good)] = good
        left.append(int(lens[s]) - B * int(b.sum()) + (b[-1] and B * blocks[s] - int(lens[s])))
    fair = (q, kc, vc, kept, np.array(left, np.int32))
    want = o4.paged_decode_attention(*fair, 0.2, B)
    got = run((q, kc, vc, broken, lens), 0.2, B, cuda_device).cpu().numpy().astype(np.float64)
    assert pkv.device_error() == 1 and pkv.device_error() == 0
    assert (np.abs(got - want) <= tolerance(fair, want, 0.2, B)).all() and not got[3].any()
