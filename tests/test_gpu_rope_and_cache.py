"""rope_and_cache on the GPU: rotated queries and keys against the fp64 oracle, values and untouched slots bit for bit.

Tolerance per value as for qk_norm_rope: half a step of fp16 and 2^-20 of |a| + |b| in fp32; rotary_scale adds its
own fp32 roundings (its product with the sine and cosine), another 2^-23 of both."""
import numpy as np
import pytest
import torch

from oracle import int4_cache as o4
from paged_kv_cache_73_gb300 import binding as pkv

pytestmark = pytest.mark.gpu


def make(seed, T, H, Hk, D, R, axes, B, dev, far=3000):
    rng = np.random.default_rng(seed)
    qkv = torch.from_numpy(rng.standard_normal((T, H + 2 * Hk, D)).astype(np.float16)).to(dev)
    inv = 10000.0 ** (-np.arange(R // 2) / (R // 2))
    pos = rng.integers(-3, far, (axes, T)).astype(np.int32)
    axis = rng.integers(0, axes, R // 2).astype(np.int32)
    w = [torch.from_numpy((1 + 0.3 * rng.standard_normal(D)).astype(np.float16)).to(dev) for _ in range(2)]
    N = T // B + 4
    slots = rng.permutation(N * B)[:T].astype(np.int64)
    pools = [torch.from_numpy(rng.standard_normal((N, Hk, B, D)).astype(np.float16)).to(dev) for _ in range(2)]
    return qkv, inv, pos, axis, w, slots, pools


def off(got, x, w, eps, pos, inv, axis, inter, scale):
    """(error, tolerance) of rows against the oracle's."""
    want, size = o4.norm_rope(x, None if w is None else w.cpu().numpy(), eps, pos, inv, axis, inter)
    R = 2 * len(inv)
    want[..., :R] *= scale
    size[..., :R] *= abs(scale)
    return np.abs(got.astype(np.float64) - want), 2.0 ** -11 * np.abs(want) + (2.0 ** -20 + 2.0 ** -22) * size + 2.0 ** -25


@pytest.mark.parametrize("T,H,Hk,D,R,axes,B,inter,norm,scale", [
    (1, 1, 1, 64, 64, 1, 16, False, False, 1.0),
    (3, 5, 1, 128, 128, 1, 4, False, True, 1.25),
    (7, 40, 8, 128, 128, 3, 16, False, True, 1.0),
    (9, 9, 9, 128, 32, 2, 32, True, True, 0.5),
    (2, 33, 3, 64, 16, 1, 8, False, False, 1.0),
    (5, 6, 2, 64, 48, 2, 16, True, False, -2.0),
    (6000, 2, 1, 64, 32, 1, 16, False, True, 1.0),
    (2600, 4, 2, 128, 64, 1, 32, True, False, 1.0),
    (70, 40, 40, 128, 128, 1, 16, False, False, 1.0),
])
def test_against_oracle(cuda_device, T, H, Hk, D, R, axes, B, inter, norm, scale):
    qkv, inv, pos, axis, w, slots, (kc, vc) = make(T + H + D + R, T, H, Hk, D, R, axes, B, cuda_device)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]  # views into the packed projection
    slots[::7] = -1                                          # padding tokens
    before, k0, v0 = qkv.clone(), kc.cpu().numpy(), vc.cpu().numpy()
    qw, kw = w if norm else (None, None)
    qo = pkv.rope_and_cache(q, k, v, torch.from_numpy(pos).to(cuda_device), pkv.rope_frequencies(inv, cuda_device), kc, vc,
                            torch.from_numpy(slots).to(cuda_device), qw, kw, eps=1e-5,
                            pair_axis=torch.from_numpy(axis).to(cuda_device), interleaved=inter, rotary_scale=scale)
    assert pkv.device_error() == 0 and torch.equal(before, qkv)
    err, tol = off(qo.cpu().numpy(), q.cpu().numpy(), qw, 1e-5, pos, inv, axis, inter, scale)
    assert (err <= tol).all(), float((err / tol).max())
    live = slots >= 0
    k1, v1 = kc.cpu().numpy(), vc.cpu().numpy()
    b, r = slots[live] // B, slots[live] % B
    if live.any():
        err, tol = off(k1[b, :, r], k.cpu().numpy()[live], kw, 1e-5, pos[:, live], inv, axis, inter, scale)
        assert (err <= tol).all(), float((err / tol).max())
    v0[b, :, r] = v.cpu().numpy()[live]
    k0[b, :, r] = k1[b, :, r]
    assert np.array_equal(v1.view(np.uint16), v0.view(np.uint16)) and np.array_equal(k1.view(np.uint16), k0.view(np.uint16))


def test_same_as_the_two_calls(cuda_device):
    qkv, inv, pos, axis, w, slots, (kc, vc) = make(3, 37, 8, 8, 128, 128, 1, 16, cuda_device, far=2 ** 31 - 1)
    q, k, v = qkv[:, :8], qkv[:, 8:16], qkv[:, 16:]
    p, f = torch.from_numpy(pos[0]).to(cuda_device), pkv.rope_frequencies(inv, cuda_device)
    sl = torch.from_numpy(slots).to(cuda_device)
    kc2, vc2 = kc.clone(), vc.clone()
    q2, k2 = pkv.qk_norm_rope(q, k, p, f, w[0], w[1])
    pkv.reshape_and_cache(k2, v.contiguous(), kc2, vc2, sl)
    q1 = pkv.rope_and_cache(q, k, v, p, f, kc, vc, sl, w[0], w[1])
    assert torch.equal(q1, q2) and torch.equal(kc, kc2) and torch.equal(vc, vc2)
    # in place on the packed projection
    pkv.rope_and_cache(q, k, v, p, f, kc, vc, sl, w[0], w[1], q_out=q)
    assert torch.equal(q, q2) and torch.equal(kc, kc2)


def test_values_keep_their_bits(cuda_device):
    qkv, inv, pos, axis, w, slots, (kc, vc) = make(4, 5, 2, 2, 64, 64, 1, 8, cuda_device)
    bits = torch.tensor([0x7e01, 0xfe55, 0x7c00, 0xfc00, 0x0001, 0x8000, 0x7dff], dtype=torch.int32).to(torch.int16)
    qkv.view(torch.int16)[:, 4:, :7] = bits.to(cuda_device)
    v = qkv[:, 4:]
    sl = torch.from_numpy(slots).to(cuda_device)
    pkv.rope_and_cache(qkv[:, :2], qkv[:, 2:4], v, torch.from_numpy(pos[0]).to(cuda_device),
                       pkv.rope_frequencies(inv, cuda_device), kc, vc, sl)
    assert torch.equal(vc[sl // 8, :, sl % 8].view(torch.int16), v.view(torch.int16))


def test_slots_outside_the_pool_and_bad_axes(cuda_device):
    qkv, inv, pos, axis, w, slots, (kc, vc) = make(5, 6, 2, 2, 64, 64, 1, 8, cuda_device)
    k0 = kc.clone()
    p, f = torch.from_numpy(pos[0]).to(cuda_device), pkv.rope_frequencies(inv, cuda_device)
    bad = torch.full((6,), kc.shape[0] * 8, dtype=torch.int64, device=cuda_device)
    want = pkv.qk_norm_rope(qkv[:, :2], qkv[:, 2:4], p, f)[0]
    q1 = pkv.rope_and_cache(qkv[:, :2], qkv[:, 2:4], qkv[:, 4:], p, f, kc, vc, bad)
    assert pkv.device_error() == 3 and torch.equal(kc, k0) and torch.equal(q1, want)
    axes = torch.full((32,), 1, dtype=torch.int32, device=cuda_device)
    pkv.rope_and_cache(qkv[:, :2], qkv[:, 2:4], qkv[:, 4:], p, f, kc, vc, -torch.ones_like(bad), pair_axis=axes)
    assert pkv.device_error() == 8 and pkv.device_error() == 0 and torch.equal(kc, k0)


def test_refusals(cuda_device):
    qkv, inv, pos, axis, w, slots, (kc, vc) = make(6, 4, 2, 2, 64, 64, 1, 8, cuda_device)
    p, f, sl = torch.from_numpy(pos[0]).to(cuda_device), pkv.rope_frequencies(inv, cuda_device), torch.from_numpy(slots).to(cuda_device)
    q, k, v = qkv[:, :2], qkv[:, 2:4], qkv[:, 4:]
    for args in ((q, k, v[:3], p, f, kc, vc, sl), (q, k, v, p[:3], f, kc, vc, sl), (q, k, v, p, f, kc, vc[:2], sl),
                 (q, k, v, p, f, kc, vc, sl[:2]), (q.float(), k, v, p, f, kc, vc, sl), (q, k, v, p.long(), f, kc, vc, sl),
                 (q.cpu(), k, v, p, f, kc, vc, sl), (q, k, v, p, f, kc.transpose(0, 1), vc, sl)):
        with pytest.raises(pkv.PkvError):
            pkv.rope_and_cache(*args)


def test_offsets_past_32_bits(cuda_device):
    B, Hk, D = 32, 8, 128
    N = (1 << 32) // (Hk * B * D) + 9                        # a pool of more than 2^32 values
    kc = torch.empty(N, Hk, B, D, dtype=torch.float16, device=cuda_device)
    vc = torch.empty_like(kc)
    qkv, inv, pos, axis, w, _, _ = make(7, 3, 8, 8, 128, 128, 1, 32, cuda_device)
    sl = torch.tensor([(N - 1) * B + 31, 5, (N - 2) * B], device=cuda_device)
    p, f = torch.from_numpy(pos[0]).to(cuda_device), pkv.rope_frequencies(inv, cuda_device)
    want = pkv.qk_norm_rope(qkv[:, :8], qkv[:, 8:16], p, f)[1]
    pkv.rope_and_cache(qkv[:, :8], qkv[:, 8:16], qkv[:, 16:], p, f, kc, vc, sl)
    assert torch.equal(kc[sl // B, :, sl % B], want) and torch.equal(vc[sl // B, :, sl % B], qkv[:, 16:])


def test_on_two_streams_at_once(cuda_device):
    cases = [make(8 + i, 300, 8, 2, 128, 128, 1, 16, cuda_device) for i in range(2)]
    f = pkv.rope_frequencies(cases[0][1], cuda_device)
    def run(i, kc, vc, stream=None):
        qkv, _, pos, _, w, slots, _ = cases[i]
        p, sl = torch.from_numpy(pos[0]).to(cuda_device), torch.from_numpy(slots).to(cuda_device)
        torch.cuda.synchronize()
        return pkv.rope_and_cache(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], p, f, kc, vc, sl, *w, stream=stream), p, sl
    want = []
    for i, c in enumerate(cases):
        kc, vc = [x.clone() for x in c[6]]
        want.append((run(i, kc, vc)[0], kc, vc))
    streams = [torch.cuda.Stream() for _ in cases]
    got = [run(i, *cases[i][6], stream=st) for i, st in enumerate(streams)]
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip((got[i][0], *cases[i][6]), want[i]))


def test_many_calls_on_two_streams(cuda_device):
    """Calls of different shapes on two streams, all of them issued before any is waited for."""
    shapes = [(300, 8, 2, 128, 128, 1, 16), (2000, 12, 3, 64, 32, 1, 8)]
    cases = [make(10 + i, *shape, cuda_device) for i, shape in enumerate(shapes)]
    args, want = [], []
    for (qkv, inv, pos, _, w, slots, pools), (_, H, Hk, *_) in zip(cases, shapes):
        p, sl = torch.from_numpy(pos[0]).to(cuda_device), torch.from_numpy(slots).to(cuda_device)
        f = pkv.rope_frequencies(inv, cuda_device)
        args.append(lambda kc, vc, st=None, a=(qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], p, f), b=(sl, *w):
                    pkv.rope_and_cache(*a, kc, vc, *b, stream=st))
        alone = [x.clone() for x in pools]
        want.append((args[-1](*alone), *alone))
    calls = 12
    pools = [[[x.clone() for x in c[6]] for _ in range(calls)] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for n in range(calls):
        for i, st in enumerate(streams):
            got[i].append(args[i](*pools[i][n], st))
    torch.cuda.synchronize()
    for i in range(2):
        for q, kv in zip(got[i], pools[i]):
            assert all(torch.equal(a, b) for a, b in zip((q, *kv), want[i]))
    assert pkv.device_error() == 0
