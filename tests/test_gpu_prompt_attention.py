"""Prompt attention (packed, causal, grouped heads) on the GPU against the fp64 oracle.

Tolerance per value, derived, with a = sum p |v| of the row: the output's fp16 rounding 2^-11 |o| (2^-25
below the normals); each weight's fp16 rounding, 2^-11 of it in the numerator and in the sum:
2^-11 (a + |o|); weights below fp16's normals, 2^-25 of the largest weight each: n 2^-25 max |v|; the
logits' fp32 error (D products, 2^-21 of their sum of sizes) and exp2's (2^-21), twice in the quotient."""
import numpy as np
import pytest
import torch

from oracle import int4_cache as o4
from paged_kv_cache_73_gb300 import binding as pkv

pytestmark = pytest.mark.gpu


def make(seed, news, past, H, Hk, D, q_scale=1.0):
    rng = np.random.default_rng(seed)
    past = [past] * len(news) if isinstance(past, int) else past
    qs = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    ks = np.concatenate([[0], np.cumsum([a + b for a, b in zip(news, past)])]).astype(np.int32)
    q = (rng.standard_normal((qs[-1], H, D)) * q_scale).astype(np.float16)
    k, v = (rng.standard_normal((ks[-1], Hk, D)).astype(np.float16) for _ in range(2))
    return q, k, v, qs, ks


def run(case, scale, dev, **kw):
    q, k, v, qs, ks = (torch.from_numpy(x).to(dev) for x in case)
    return pkv.prompt_attention(q, k, v, qs, scale, int(np.diff(case[3]).max()), key_start=ks, **kw)


def want_and_tol(case, scale):
    q, k, v, qs, ks = case
    want = o4.prompt_attention(q, k, v, qs, ks, scale)
    tol = np.zeros_like(want)
    group = q.shape[1] // k.shape[1]
    for s in range(len(qs) - 1):
        kk, vv = k[ks[s]:ks[s + 1]].astype(np.float64), v[ks[s]:ks[s + 1]].astype(np.float64)
        n, m = qs[s + 1] - qs[s], ks[s + 1] - ks[s]
        if n == 0:
            continue
        hide = np.arange(m)[None] > (m - n + np.arange(n))[:, None]
        for h in range(q.shape[1]):
            qq = q[qs[s]:qs[s + 1], h].astype(np.float64)
            x = np.where(hide, -np.inf, scale * qq @ kk[:, h // group].T)
            p = np.exp(x - x.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            a = p @ np.abs(vv[:, h // group])
            dx = 2.0 ** -21 * (scale * np.abs(qq) @ np.abs(kk[:, h // group]).T).max(1, keepdims=True) + 2.0 ** -21
            o = np.abs(want[qs[s]:qs[s + 1], h])
            tol[qs[s]:qs[s + 1], h] = (2.0 ** -11 * (2 * o + a) + 2.0 ** -25 + 2 * dx * a
                                       + m * 2.0 ** -25 * np.abs(vv).max())
    return want, tol


def check(case, dev, scale=None):
    scale = case[0].shape[2] ** -0.5 if scale is None else scale
    got = run(case, scale, dev).cpu().numpy().astype(np.float64)
    code = pkv.device_error()
    assert code == 0, pkv.DEV_CODES[code]
    want, tol = want_and_tol(case, scale)
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-30)).max())


NEWS = [1, 2, 63, 64, 65, 127, 128, 129, 0, 200, 257, 300]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hk", [(2, 2), (2, 1), (3, 1), (10, 2), (8, 2)])
def test_ragged_prompts(cuda_device, D, H, Hk):
    check(make(D + H, NEWS, 0, H, Hk, D), cuda_device)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 2)])
def test_chunks_over_cached_context(cuda_device, D, H, Hk):
    check(make(D + H + 1, NEWS, [0, 5, 64, 1, 63, 130, 7, 400, 9, 33, 2, 129], H, Hk, D), cuda_device)


@pytest.mark.parametrize("D,H,Hk", [(128, 24, 24), (64, 30, 6)])
def test_more_tiles_than_run_at_once(cuda_device, D, H, Hk):
    # CTAs take over tiles: 29 tiles a head, some sequences without any
    check(make(D + H + 2, [130, 1, 0, 600, 64, 3, 300, 0, 257, 129, 5, 700], [0, 0, 3, 100, 1, 70, 0, 9, 5, 0, 0, 64], H, Hk, D),
          cuda_device)


def test_output_at_a_16_byte_boundary(cuda_device):
    q, k, v, qs, ks = (torch.from_numpy(x).to(cuda_device) for x in make(16, [200], 0, 2, 1, 128))
    buf = torch.zeros(200 * 2 * 128 + 8, dtype=torch.float16, device=cuda_device)
    out = buf[8:].view(200, 2, 128)
    assert out.data_ptr() % 32 == 16
    pkv.prompt_attention(q, k, v, qs, 0.1, 200, out=out)
    assert torch.equal(out, pkv.prompt_attention(q, k, v, qs, 0.1, 200)) and not buf[:8].any()


def test_one_query_each_over_long_contexts(cuda_device):
    check(make(5, [1] * 5, [0, 62, 63, 64, 1000], 4, 2, 128), cuda_device)


def test_long_prompts(cuda_device):
    check(make(6, [1500, 3], 0, 2, 1, 128), cuda_device)
    check(make(7, [1111], 700, 1, 1, 64), cuda_device)


@pytest.mark.parametrize("q_scale", [0.0, 40.0])
def test_flat_and_peaked_softmax(cuda_device, q_scale):
    check(make(8, [300, 70], 100, 2, 1, 128, q_scale), cuda_device)


def test_rising_logits_move_the_maximum(cuda_device):
    q, k, v, qs, ks = make(9, [900], 0, 2, 1, 64)
    k[:, :, 0] = np.linspace(0, 60, 900)[:, None]
    q[:, :, 0] = 8
    check((q, k, v, qs, ks), cuda_device)


@pytest.mark.parametrize("H,Hk", [(1, 1), (2, 1)])
def test_keys_and_values_that_are_not_seen(cuda_device, H, Hk):
    # rows of other sequences, and of the own one after a query, hold NaNs and infinities
    news, past = [100, 300, 64, 40], [0, 30, 7, 100]
    case = make(10, news, past, H, Hk, 128)
    clean = run(case, 0.1, cuda_device)
    q, k, v, qs, ks = (x.copy() for x in case)
    for x in (k, v):
        x[ks[1] - 1], x[ks[2] - 20], x[ks[2] - 2], x[ks[3]] = np.nan, np.inf, -np.inf, np.nan
    got = run((q, k, v, qs, ks), 0.1, cuda_device)
    assert pkv.device_error() == 0
    same = np.ones(qs[-1], bool)
    same[qs[1] - 1] = False                                  # the last query of sequence 0 sees its own key
    same[qs[2] - 20:qs[2]] = False
    same[qs[3]:] = False                                     # every query of the last sequence sees its first key
    assert torch.equal(got[torch.from_numpy(same)], clean[torch.from_numpy(same)])
    # values alone: the queries that see an infinity get it, and a NaN where two meet
    v2 = case[2].copy()
    v2[ks[2] - 20, 0, 3], v2[ks[2] - 2, 0, 3], v2[ks[2] - 5, 0, 9] = np.inf, -np.inf, np.nan
    got = run((case[0], case[1], v2, qs, ks), 0.1, cuda_device).float()
    rows = got[qs[2] - 30:qs[2], 0].cpu().numpy()
    assert (rows[10:28, 3] == np.inf).all() and np.isnan(rows[28:, 3]).all() and np.isfinite(rows[:10]).all()
    assert np.isnan(rows[25:, 9]).all() and np.isfinite(rows[:25, 9]).all()


def test_padding_rows_left_and_strided_views(cuda_device):
    q, k, v, qs, ks = make(11, [40, 200], 0, 4, 2, 128)
    pad = 9
    qkv = torch.zeros(240 + pad, 8, 128, dtype=torch.float16, device=cuda_device)
    qkv[:240, :4], qkv[:240, 4:6], qkv[:240, 6:] = (torch.from_numpy(x).to(cuda_device) for x in (q, k, v))
    qkv[240:] = float("nan")
    out = torch.full((240 + pad, 4, 128), 5.0, dtype=torch.float16, device=cuda_device)
    start = torch.from_numpy(qs).to(cuda_device)
    pkv.prompt_attention(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], start, 0.09, 200, out=out)
    assert pkv.device_error() == 0
    assert torch.equal(out[:240], run((q, k, v, qs, ks), 0.09, cuda_device)) and (out[240:] == 5).all()


def test_bad_ranges_are_recorded(cuda_device):
    case = make(12, [50, 60, 70], 0, 2, 1, 64)
    good = run(case, 0.1, cuda_device)
    q, k, v, qs, ks = (torch.from_numpy(x).to(cuda_device) for x in case)
    out = torch.full_like(q, 3.0)
    pkv.prompt_attention(q, k, v, torch.tensor([0, 50, 110, 181], dtype=torch.int32, device=cuda_device), 0.1, 128,
                         key_start=ks, out=out)              # 71 queries, 70 keys; and past q
    assert pkv.device_error() == 6
    assert torch.equal(out[:110], good[:110]) and (out[110:] == 3).all()
    pkv.prompt_attention(q, k, v, qs, 0.1, 70, key_start=torch.tensor([-1, 50, 40, 1000], dtype=torch.int32, device=cuda_device),
                         out=out)
    assert pkv.device_error() == 6
    long = make(13, [300], 0, 2, 1, 64)
    d = [torch.from_numpy(x).to(cuda_device) for x in long]
    pkv.prompt_attention(d[0], d[1], d[2], d[3], 0.1, 128)
    assert pkv.device_error() == 6                           # the rows past the grid
    got = pkv.prompt_attention(d[0], d[1], d[2], d[3], 0.1, 1000)   # overstated: nothing lost
    assert pkv.device_error() == 0 and torch.equal(got, run(long, 0.1, cuda_device))


def test_captured_and_on_another_stream(cuda_device):
    case = make(14, [77, 300], 20, 4, 2, 128)
    q, k, v, qs, ks = (torch.from_numpy(x).to(cuda_device) for x in case)
    out = torch.zeros_like(q)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        pkv.prompt_attention(q, k, v, qs, 0.1, 300, key_start=ks, out=out)
    q.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, pkv.prompt_attention(q, k, v, qs, 0.1, 300, key_start=ks))


def test_shapes_refused(cuda_device):
    q, k, v, qs, ks = (torch.from_numpy(x).to(cuda_device) for x in make(15, [10], 0, 4, 2, 64))
    for bad in (dict(key=k[:, :1]), dict(value=v[..., :32]), dict(key_start=ks[:1]), dict(out=q[:5]), dict(q=q.float()),
                dict(query_start=qs.long()), dict(q=q[:, :3]), dict(scale=-1.0)):
        with pytest.raises(pkv.PkvError):
            pkv.prompt_attention(**{**dict(q=q, key=k, value=v, query_start=qs, scale=0.1, max_query_len=10), **bad})


def test_more_sequences_than_a_warp_holds(cuda_device):
    # 70 sequences, some empty, in three batches of lanes; few and many heads
    rng = np.random.default_rng(20)
    news = [int(x) for x in rng.choice([0, 1, 5, 64, 130, 200], 70)]
    past = [int(x) for x in rng.choice([0, 3, 64, 150], 70)]
    check(make(21, news, past, 2, 1, 64), cuda_device)
    check(make(22, [0] * 40 + [150] * 3, 0, 24, 24, 128), cuda_device)


def test_a_bad_range_in_a_later_batch_is_recorded(cuda_device):
    # sequences 40, 42 and 44 go back to row 0 and the ones between overlap: more tiles than the grid has
    starts = list(range(0, 41 * 30, 30)) + [0, 1200, 0, 1200, 0, 1200]
    q, k, v = (torch.randn(1230, 2, 64, device=cuda_device).half() for _ in range(3))
    pkv.prompt_attention(q, k, v, torch.tensor(starts, dtype=torch.int32, device=cuda_device), 0.1, 1200)
    assert pkv.device_error() == 6


def test_long_wait_for_a_long_context(cuda_device):
    # one query over 2^24 keys, about 0.2 s in which some roles wait for others.  With q = 0 each weight is
    # 1; whole values in [-1, 1] keep every partial sum below 2^24, exact in fp32: only the division and the
    # fp16 rounding remain
    m = 1 << 24
    v = (torch.arange(m, device=cuda_device, dtype=torch.int32)[:, None, None] * torch.arange(1, 65, device=cuda_device,
                                                                                             dtype=torch.int32))
    v = (v % 3 - (torch.arange(64, device=cuda_device) % 2)).half()
    k = torch.zeros_like(v)
    q = torch.zeros(1, 1, 64, dtype=torch.float16, device=cuda_device)
    start = lambda n: torch.tensor([0, n], dtype=torch.int32, device=cuda_device)
    v.clamp_(-1, 1)
    got = pkv.prompt_attention(q, k, v, start(1), 1.0, 1, key_start=start(m))
    assert pkv.device_error() == 0
    want = v.sum(0, dtype=torch.float64) / m
    assert ((got[0].double() - want).abs() <= want.abs() * (2.0 ** -11 + 2.0 ** -22) + 2.0 ** -25).all()


def test_rows_past_2_31_elements(cuda_device):
    # the last sequence's rows lie past element 2^31 of q, key, value and out
    T, H, D, n = 360000, 48, 128, 200
    big = torch.empty(T, H, D, dtype=torch.float16, device=cuda_device)
    big[T - n:] = torch.randn(n, H, D, device=cuda_device)
    out = torch.empty_like(big)
    start = torch.tensor([T - n, T], dtype=torch.int32, device=cuda_device)
    pkv.prompt_attention(big, big[:, :24], big[:, 24:], start, 0.1, n, out=out)
    small = big[T - n:].clone()
    want = pkv.prompt_attention(small, small[:, :24], small[:, 24:], start - (T - n), 0.1, n)
    assert pkv.device_error() == 0 and torch.equal(out[T - n:], want)


@pytest.mark.parametrize("news,past,H,Hk,D", [
    ([1], [5000], 4, 1, 128), ([130], [4000], 2, 2, 64), ([300, 40], [2000, 3000], 3, 1, 128),
    ([1, 1, 0, 128], [0, 9000, 70, 3], 4, 2, 64), ([700], [0], 2, 1, 128), ([64, 65], [960, 1100], 8, 2, 128)])
def test_few_tiles_over_many_keys(cuda_device, news, past, H, Hk, D):
    # the keys of a query tile are shared out to the CTAs of a cluster; some have none of a short sequence
    check(make(40 + D + H, news, past, H, Hk, D), cuda_device)


def test_few_tiles_unseen_values_and_padding(cuda_device):
    # as above with NaNs and infinities behind the queries, past the sequence, and seen by some rows
    case = make(41, [100, 60], [3000, 1500], 2, 1, 128)
    q, k, v, qs, ks = case
    clean = run(case, 0.1, cuda_device)
    k2, v2 = k.copy(), v.copy()
    for x in (k2, v2):
        x[ks[1] - 1], x[ks[2] - 30] = np.nan, -np.inf
    got = run((q, k2, v2, qs, ks), 0.1, cuda_device)
    assert pkv.device_error() == 0
    same = np.ones(qs[-1], bool)
    same[qs[1] - 1] = False
    same[qs[2] - 30:] = False
    assert torch.equal(got[torch.from_numpy(same)], clean[torch.from_numpy(same)])
    assert torch.isnan(got[qs[1] - 1]).all()
    v3 = v.copy()
    v3[ks[2] - 20, 0, 3], v3[ks[2] - 2, 0, 3], v3[ks[2] - 5, 0, 9], v3[5, 0, 70] = np.inf, -np.inf, np.nan, np.inf
    got = run((q, k, v3, qs, ks), 0.1, cuda_device).float().cpu().numpy()
    rows = got[qs[2] - 30:, 0]
    assert (rows[10:28, 3] == np.inf).all() and np.isnan(rows[28:, 3]).all() and np.isfinite(rows[:10, 3]).all()
    assert np.isnan(rows[25:, 9]).all() and np.isfinite(rows[:25, 9]).all()
    assert (got[:100, :, 70] == np.inf).all()                # seen by every query of the first sequence
    # rows behind the last sequence stay, and the call replays from a graph
    out = torch.full((170, 2, 128), 5.0, dtype=torch.float16, device=cuda_device)
    d = [torch.from_numpy(x).to(cuda_device) for x in case]
    qq = torch.cat([d[0], torch.full((10, 2, 128), float("nan"), dtype=torch.float16, device=cuda_device)])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.prompt_attention(qq, d[1], d[2], d[3], 0.1, 100, key_start=d[4], out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:160], clean) and (out[160:] == 5).all()


def test_two_streams_at_once(cuda_device):
    # shared-out keys on one stream, a full grid of D = 64 on another
    cases = [make(42, [100], [6000], 8, 2, 128), make(43, [700, 900, 300], 100, 30, 6, 64)]
    dev = [[torch.from_numpy(x).to(cuda_device) for x in c] for c in cases]
    call = lambda d, **kw: pkv.prompt_attention(d[0], d[1], d[2], d[3], 0.1, 900, key_start=d[4], **kw)
    alone = [call(d) for d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dev]
    got = [[call(d, stream=st) for d, st in zip(dev, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
    assert all(torch.equal(g, a) for pair in got for g, a in zip(pair, alone))


def test_more_queries_than_announced_are_recorded(cuda_device):
    # within the first tile and past it; only rows past the announced length's tiles are not written
    for n, announced, written in ((100, 10, 100), (128, 127, 128), (300, 200, 256)):
        q, k, v, qs, _ = (torch.from_numpy(x).to(cuda_device) for x in make(44 + n, [n], 0, 2, 1, 64))
        want = pkv.prompt_attention(q, k, v, qs, 0.1, n)
        assert pkv.device_error() == 0
        out = torch.full_like(q, 3.0)
        pkv.prompt_attention(q, k, v, qs, 0.1, announced, out=out)
        assert pkv.device_error() == 6
        assert torch.equal(out[:written], want[:written]) and (out[written:] == 3).all()


@pytest.mark.parametrize("D,H,Hk,news,past", [(64, 2, 1, [1, 70], 9000), (128, 24, 24, [300], 2000)])
def test_many_small_weights_beside_a_large_one(cuda_device, D, H, Hk, news, past):
    # Each sequence's first key takes nearly all the weight and has a value of 0: the result is what thousands
    # of weights of about 2^-27 of that key's add up to.  As want_and_tol, but a weight's fp16 rounding
    # below the normals is 2^-32 of the largest weight, and of these weights' sum no more than that is lost.
    q, k, v, qs, ks = make(45 + D, news, past, H, Hk, D)
    k *= np.float16(0.05)
    v[:] = np.abs(v)
    q[..., 0], k[..., 0] = 4, 0
    scale = D ** -0.5
    k[ks[:-1], :, 0], k[ks[:-1], :, 1:], v[ks[:-1]] = 27 * np.log(2) / (4 * scale), 0, 0
    got = run((q, k, v, qs, ks), scale, cuda_device).cpu().numpy().astype(np.float64)
    assert pkv.device_error() == 0
    want = o4.prompt_attention(q, k, v, qs, ks, scale)
    for s in range(len(news)):
        rows, keys = slice(qs[s], qs[s + 1]), slice(ks[s], ks[s + 1])
        m = ks[s + 1] - ks[s]
        dx = 2.0 ** -21 * (scale * np.abs(q[rows].astype(np.float64)).sum(-1).max() * np.abs(k[keys]).max()) + 2.0 ** -21
        o = np.abs(want[rows])
        tol = 2.0 ** -11 * 3 * o + 2.0 ** -25 + 2 * dx * o + m * 2.0 ** -32 * v[keys].max()
        assert (tol < 0.25 * o).mean() > 0.9                 # the sums are not lost in the tolerance
        err = np.abs(got[rows] - want[rows])
        assert (err <= tol).all(), float((err / tol).max())


def test_infinite_values_in_two_parts_of_a_split_item(cuda_device):
    # 128 queries over 1018 keys, shared out to eight CTAs of two key tiles each: tile 13, which some queries do
    # not see whole, is the seventh's, the keys from 896 on the eighth's.  These have logits of 160, the others of
    # 0, so that the seventh's part counts for nothing in rows that see both; an infinity of the
    # eighth's in another column than the seventh's own is still one there.
    q, k, v, qs, ks = make(46, [128], 890, 1, 1, 64)
    q[:], k[:] = 0, 0
    q[..., 0], k[896:, :, 0] = 8, 20
    v[850, 0, 3], v[897, 0, 9] = np.inf, np.inf
    got = run((q, k, v, qs, ks), 1.0, cuda_device).float().cpu().numpy()[:, 0]
    assert pkv.device_error() == 0
    assert (got[:6, 3] == np.inf).all()                      # queries 0 to 5 see keys up to 890 .. 895
    assert (got[7:, 9] == np.inf).all() and np.isfinite(got[:7, 9]).all()
    rest = [c for c in range(64) if c not in (3, 9)]
    assert np.isfinite(got[:, rest]).all()
