"""Rows into and out of the four-bit cache on the GPU: byte for byte the oracle's, which decides
every rounding in exact arithmetic; copy and swap of four-bit blocks bit-exact."""
import numpy as np
import pytest
import torch

from oracle import int4_cache as o4
from paged_kv_cache_73_gb300 import binding as pkv

pytestmark = pytest.mark.gpu


def _rows(rng, T, H, D):
    """Rows of many sizes: ordinary, flat, tiny (scales below the normals), huge, offset, with halves."""
    x = rng.standard_normal((T, H, D)) * 10.0 ** rng.uniform(-4, 3, (T, H, 1))
    x += rng.choice([0, 0, 0, 50.0], (T, H, 1))
    x[::7] = np.round(rng.uniform(0, 30, x[::7].shape)) / 2      # scale 1 or so: exact halves
    x[::7, :, 0], x[::7, :, 1] = 0, 15
    x[3::11] = 0.125
    x[5::13] = rng.integers(-3, 4, x[5::13].shape) * 2.0 ** -24
    return np.clip(x, -65504, 65504).astype(np.float16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [4, 8, 16, 32])
@pytest.mark.parametrize("T,H", [(1, 1), (37, 3), (1100, 1), (5, 41)])
def test_write_and_read_back(cuda_device, D, B, T, H):
    rng = np.random.default_rng(D + B + T + H)
    kv = _rows(rng, T, 2 * H, D)
    N = -(-T // B) + 3
    slots = rng.permutation(N * B)[:T].astype(np.int64)
    if T > 4:
        slots[2] = -1
    kc, vc = o4.empty_pool(N, H, B, D), o4.empty_pool(N, H, B, D)
    kd, vd = (torch.from_numpy(p.copy()).to(cuda_device) for p in (kc, vc))
    dev = torch.from_numpy(kv).to(cuda_device)
    sl = torch.from_numpy(slots).to(cuda_device)
    pkv.reshape_and_cache_int4(dev[:, :H], dev[:, H:], kd, vd, sl, B)     # strided views
    o4.store(kc, kv[:, :H], slots, B)
    o4.store(vc, kv[:, H:], slots, B)
    assert pkv.device_error() == 0
    assert np.array_equal(kd.cpu().numpy(), kc) and np.array_equal(vd.cpu().numpy(), vc)
    ko, vo = torch.full((T, H, D), 7.0, dtype=torch.float16, device=cuda_device), torch.full(
        (T, H, D), 7.0, dtype=torch.float16, device=cuda_device)
    pkv.gather_cache_int4(kd, vd, sl, B, ko, vo)
    assert pkv.device_error() == 0
    for got, pool in ((ko, kc), (vo, vc)):
        want = o4.pool_values(pool, B)[slots // B, :, slots % B].astype(np.float16)   # rounded once
        want[slots < 0] = 7.0
        assert np.array_equal(got.cpu().numpy().view(np.uint16), want.view(np.uint16))


def test_rows_that_are_not_finite_stand_for_nans(cuda_device):
    x = torch.randn(4, 3, 64, device=cuda_device).half()
    x[0, 0, 5], x[1, 1, 7], x[2, 2, 9] = float("nan"), float("inf"), float("-inf")
    kc = torch.zeros(pkv.int4_cache_shape(1, 3, 4, 64), dtype=torch.uint8, device=cuda_device)
    vc = torch.zeros_like(kc)
    sl = torch.arange(4, device=cuda_device)
    pkv.reshape_and_cache_int4(x, x, kc, vc, sl, 4)
    k, v = pkv.gather_cache_int4(kc, vc, sl, 4)
    bad = torch.zeros(4, 3, dtype=torch.bool, device=cuda_device)
    bad[0, 0] = bad[1, 1] = bad[2, 2] = True
    for y in (k, v):
        assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()


def test_bad_slots_are_recorded_and_skipped(cuda_device):
    kc = torch.zeros(pkv.int4_cache_shape(2, 2, 4, 64), dtype=torch.uint8, device=cuda_device)
    vc = torch.zeros_like(kc)
    x = torch.randn(3, 2, 64, device=cuda_device).half()
    sl = torch.tensor([1, 8, -5], device=cuda_device)
    pkv.reshape_and_cache_int4(x, x, kc, vc, sl, 4)
    assert pkv.device_error() == 3
    out = torch.full((3, 2, 64), 9.0, dtype=torch.float16, device=cuda_device)
    k, _ = pkv.gather_cache_int4(kc, vc, sl, 4, key=out)
    assert pkv.device_error() == 3
    assert (k[1:] == 9).all() and not (k[0] == 9).all()
    one = kc.clone()
    one[0, :, 32:64] = 0                                    # row 1 of block 0 and its scale and zero
    one[0, :, 4 * 32 + 4:4 * 32 + 8] = 0
    assert not one.any()


def test_no_tokens_and_refusals(cuda_device):
    kc = torch.zeros(pkv.int4_cache_shape(2, 2, 4, 64), dtype=torch.uint8, device=cuda_device)
    x = torch.zeros(3, 2, 64, dtype=torch.float16, device=cuda_device)
    sl = torch.zeros(3, dtype=torch.int64, device=cuda_device)
    pkv.reshape_and_cache_int4(x[:0], x[:0], kc, kc.clone(), sl[:0], 4)
    pkv.gather_cache_int4(kc, kc, sl[:0], 4)
    for call in (lambda: pkv.reshape_and_cache_int4(x, x, kc, kc.clone(), sl[:2], 4),
                 lambda: pkv.reshape_and_cache_int4(x, x[:, :1], kc, kc.clone(), sl, 4),
                 lambda: pkv.reshape_and_cache_int4(x, x, kc, kc.clone(), sl, 5),
                 lambda: pkv.reshape_and_cache_int4(x, x, kc, kc[:1], sl, 4),
                 lambda: pkv.gather_cache_int4(kc, kc, sl, 4, key=x[:2]),
                 lambda: pkv.gather_cache_int4(kc.float(), kc, sl, 4)):
        with pytest.raises(pkv.PkvError):
            call()


@pytest.mark.parametrize("D,B,H", [(64, 4, 1), (64, 4, 3), (128, 16, 5), (128, 32, 2)])
def test_copy_and_swap_blocks(cuda_device, D, B, H):
    g = torch.Generator(device=cuda_device)
    g.manual_seed(D + B)
    shape = pkv.int4_cache_shape(9, H, B, D)
    pools = [torch.randint(0, 256, shape, generator=g, device=cuda_device, dtype=torch.uint8) for _ in range(4)]
    want = [p.clone() for p in pools]
    pairs = torch.tensor([[1, 7], [3, 0]], device=cuda_device)
    pkv.copy_blocks_int4(pools[:2], pools[2:], pairs, B)
    for p, w in zip(pools, want):
        w[7], w[0] = w[1].clone(), w[3].clone()
        assert torch.equal(p, w)
    host = [torch.zeros(pkv.int4_cache_shape(4, H, B, D), dtype=torch.uint8).pin_memory() for _ in range(4)]
    moves = torch.tensor([[8, 1], [2, 3]], device=cuda_device)
    pkv.swap_blocks_int4(pools[:2], pools[2:], host[:2], host[2:], moves, B)
    back = torch.tensor([[1, 5], [3, 6]], device=cuda_device)
    pkv.swap_blocks_int4(host[:2], host[2:], pools[:2], pools[2:], back, B)
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
    for p, w, hp in zip(pools, want, host):
        assert torch.equal(hp[1], w[8].cpu()) and torch.equal(hp[3], w[2].cpu()) and not hp[0].any()
        w[5], w[6] = w[8].clone(), w[2].clone()
        assert torch.equal(p, w)
    pkv.copy_blocks_int4(pools[:1], pools[1:2], torch.tensor([[0, 9]], device=cuda_device), B)
    assert pkv.device_error() == 4


def test_rows_and_pools_past_32_bits(cuda_device):
    # rows past element 2^31 of key, value and the outputs; slots in the last blocks of a pool past 4 GiB
    T, H, D, B, n = 700000, 24, 128, 32, 150
    N = (5 << 30) // (H * B * (D // 2 + 4))
    kv = torch.empty(T, 2 * H, D, dtype=torch.float16, device=cuda_device)
    kv[T - n:] = torch.randn(n, 2 * H, D, device=cuda_device)
    pools = [torch.zeros(pkv.int4_cache_shape(N, H, B, D), dtype=torch.uint8, device=cuda_device) for _ in range(2)]
    slots = torch.full((T,), -1, dtype=torch.int64, device=cuda_device)
    slots[T - n:] = N * B - 1 - torch.arange(n, device=cuda_device)
    pkv.reshape_and_cache_int4(kv[:, :H], kv[:, H:], *pools, slots, B)
    outs = pkv.gather_cache_int4(*pools, slots, B)
    assert outs[0].numel() > 1 << 31
    small = [torch.zeros(pkv.int4_cache_shape(8, H, B, D), dtype=torch.uint8, device=cuda_device) for _ in range(2)]
    low, x = slots[T - n:] - (N - 8) * B, kv[T - n:].clone()
    pkv.reshape_and_cache_int4(x[:, :H], x[:, H:], *small, low, B)
    assert pkv.device_error() == 0
    assert all(torch.equal(p[N - 8:], s) and not p[:N - 8].any() for p, s in zip(pools, small))
    assert all(torch.equal(o[T - n:], s) for o, s in zip(outs, pkv.gather_cache_int4(*small, low, B)))


def test_a_slot_read_many_times(cuda_device):
    x = torch.randn(8, 2, 64, device=cuda_device).half()
    pools = [torch.zeros(pkv.int4_cache_shape(2, 2, 4, 64), dtype=torch.uint8, device=cuda_device) for _ in range(2)]
    pkv.reshape_and_cache_int4(x, x, *pools, torch.arange(8, device=cuda_device), 4)
    one = pkv.gather_cache_int4(*pools, torch.arange(8, device=cuda_device), 4)
    sl = torch.tensor([5, 5, 0, 5, 7, 0, 5], device=cuda_device)
    for got, o in zip(pkv.gather_cache_int4(*pools, sl, 4), one):
        assert torch.equal(got, o[sl])


@pytest.mark.parametrize("D,H,T", [(128, 1, 9729), (128, 2, 10001), (64, 4, 9731), (64, 1, 9728)])
def test_many_tokens_of_few_heads(cuda_device, D, H, T):
    # four tokens to a warp: the last warp's not all there, padding and bad slots beside others
    B, rng = 16, np.random.default_rng(D + H)
    kv = _rows(rng, T, 2 * H, D)
    N = -(-T // B) + 1
    slots = rng.permutation(N * B)[:T].astype(np.int64)
    slots[3::7] = -1
    slots[5] = slots[T - 1] = N * B
    kc, vc = o4.empty_pool(N, H, B, D), o4.empty_pool(N, H, B, D)
    kd, vd = (torch.from_numpy(p.copy()).to(cuda_device) for p in (kc, vc))
    dev = torch.from_numpy(kv).to(cuda_device)
    sl = torch.from_numpy(slots).to(cuda_device)
    pkv.reshape_and_cache_int4(dev[:, :H], dev[:, H:], kd, vd, sl, B)
    assert pkv.device_error() == 3
    good = np.where(slots >= N * B, -1, slots)
    o4.store(kc, kv[:, :H], good, B)
    o4.store(vc, kv[:, H:], good, B)
    assert np.array_equal(kd.cpu().numpy(), kc) and np.array_equal(vd.cpu().numpy(), vc)
    ko, vo = (torch.full((T, H, D), 7.0, dtype=torch.float16, device=cuda_device) for _ in range(2))
    pkv.gather_cache_int4(kd, vd, sl, B, ko, vo)
    assert pkv.device_error() == 3
    for got, pool in ((ko, kc), (vo, vc)):
        want = o4.pool_values(pool, B)[good // B, :, good % B].astype(np.float16)
        want[good < 0] = 7.0
        assert np.array_equal(got.cpu().numpy().view(np.uint16), want.view(np.uint16))


@pytest.mark.parametrize("D", [64, 128])
def test_halves_beside_a_tiny_minimum(cuda_device, D):
    # x - min takes more than the 24 bits of fp32: rounded to them, it lands on a half that it is not on
    rng = np.random.default_rng(D)
    x = np.zeros((400, 2, D), np.float16)
    step = 2.0 ** rng.integers(-6, 12, (400, 2, 1))
    x[...] = step * rng.integers(0, 31, x.shape) / 2
    x[..., 0], x[..., 1] = 0, 15 * step[..., 0]
    x[:, 0, 0] = -rng.integers(1, 64, 400) * 2.0 ** -24      # below 0: the values lie just past the halves
    x[:, 1, 2] = x[:, 1, 0] = 2.0 ** -24                     # above 0: just before them
    x[:, 1, 3:] = np.maximum(x[:, 1, 3:], 2.0 ** -24)
    x[0, 0, :3], x[0, 0, 3:] = [-65504, 19936, -2.0 ** -24], 0
    pools = [torch.zeros(pkv.int4_cache_shape(100, 2, 4, D), dtype=torch.uint8, device=cuda_device) for _ in range(2)]
    dev = torch.from_numpy(x).to(cuda_device)
    pkv.reshape_and_cache_int4(dev, dev.flip(1), *pools, torch.arange(400, device=cuda_device), 4)
    assert pkv.device_error() == 0
    for pool, rows in zip(pools, (x, x[:, ::-1])):
        want = o4.empty_pool(100, 2, 4, D)
        o4.store(want, rows, np.arange(400), 4)
        assert np.array_equal(pool.cpu().numpy(), want)
