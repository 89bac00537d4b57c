"""qk_norm_rope on the GPU against the oracle (fp64, angles modulo one turn in exact arithmetic).

Tolerance per value, derived: the fp16 rounding is half a step, 2^-11 of the value (2^-25 below the
normals); in fp32 the sum of squares (12 roundings of 2^-24 on its longest path), rsqrtf (2^-22), two
products, the sine and cosine (2^-22, and 2^-24 turns of the angle's own rounding = 2^-21.3) and the
last product and sum are off by less than 2^-20 of |a| + |b|."""
import numpy as np
import pytest
import torch

from oracle import int4_cache as o4
from paged_kv_cache_73_gb300 import binding as pkv

pytestmark = pytest.mark.gpu


def _inputs(seed, T, H, Hk, D, R, axes, dev, far):
    rng = np.random.default_rng(seed)
    qkv = torch.from_numpy(rng.standard_normal((T, H + 2 * Hk, D)).astype(np.float16)).to(dev)
    inv = 10000.0 ** (-np.arange(R // 2) / (R // 2))
    pos = rng.integers(-3, far, (axes, T)).astype(np.int32)
    pos[0, -1] = far
    axis = rng.integers(0, axes, R // 2).astype(np.int32)
    w = [torch.from_numpy((1 + 0.3 * rng.standard_normal(D)).astype(np.float16)).to(dev) for _ in range(2)]
    return qkv, inv, pos, axis, w


def _check(got, x, w, eps, pos, inv, axis, inter):
    want, size = o4.norm_rope(x.cpu().numpy(), None if w is None else w.cpu().numpy(), eps, pos, inv, axis, inter)
    err = np.abs(got.cpu().numpy().astype(np.float64) - want)
    tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -20 * size + 2.0 ** -25
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("T,H,Hk,D,R,axes,inter,norm", [
    (1, 1, 1, 64, 64, 1, False, True),
    (3, 5, 1, 128, 128, 1, False, True),
    (7, 40, 8, 128, 128, 3, False, True),
    (5, 7, 3, 128, 64, 2, False, True),
    (5, 9, 9, 128, 32, 3, True, True),
    (2, 33, 2, 64, 16, 1, False, False),
    (4, 3, 2, 64, 48, 2, True, True),
    (3, 12, 4, 128, 96, 1, False, True),
    (1200, 2, 1, 64, 32, 1, False, True),
])
def test_against_oracle(cuda_device, T, H, Hk, D, R, axes, inter, norm):
    qkv, inv, pos, axis, w = _inputs(T + H + D + R, T, H, Hk, D, R, axes, cuda_device, 3000)
    q, k = qkv[:, :H], qkv[:, H:H + Hk]                     # views into the packed projection
    before = qkv.clone()
    qw, kw = (w if norm else (None, None))
    qo, ko = pkv.qk_norm_rope(q, k, torch.from_numpy(pos).to(cuda_device), pkv.rope_frequencies(inv, cuda_device),
                              qw, kw, eps=1e-5, pair_axis=torch.from_numpy(axis).to(cuda_device), interleaved=inter)
    assert pkv.device_error() == 0
    assert torch.equal(before, qkv)
    _check(qo, q, qw, 1e-5, pos, inv, axis, inter)
    _check(ko, k, kw, 1e-5, pos, inv, axis, inter)


def test_one_weight_only_and_far_positions(cuda_device):
    qkv, inv, pos, axis, w = _inputs(5, 6, 4, 2, 128, 128, 1, cuda_device, 2 ** 31 - 1)
    q, k = qkv[:, :4], qkv[:, 4:6]
    qo, ko = pkv.qk_norm_rope(q, k, torch.from_numpy(pos[0]).to(cuda_device), pkv.rope_frequencies(inv, cuda_device),
                              k_weight=w[1])
    assert pkv.device_error() == 0
    # fp64 frequencies are 2^-53 off and the turns count 2^-54 of a turn: 2^31 positions on, 2^-22 turns
    for got, x, wt in ((qo, q, None), (ko, k, w[1])):
        want, size = o4.norm_rope(x.cpu().numpy(), None if wt is None else wt.cpu().numpy(), 1e-6, pos, inv,
                                  np.zeros(64, int), False)
        err = np.abs(got.cpu().numpy().astype(np.float64) - want)
        assert (err <= 2.0 ** -11 * np.abs(want) + 2.0 ** -19 * size + 2.0 ** -25).all()


def test_in_place_and_zero_rows_and_tokens(cuda_device):
    qkv, inv, pos, axis, w = _inputs(6, 70, 40, 8, 128, 128, 1, cuda_device, 100)
    qkv[3] = 0
    src = qkv.clone()
    q, k, v = qkv[:, :40], qkv[:, 40:48], qkv[:, 48:]
    fr, p = pkv.rope_frequencies(inv, cuda_device), torch.from_numpy(pos[0]).to(cuda_device)
    want = pkv.qk_norm_rope(src[:, :40], src[:, 40:48], p, fr, w[0], w[1])
    got = pkv.qk_norm_rope(q, k, p, fr, w[0], w[1], q_out=q, k_out=k)
    assert got[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, src[:, 48:])
    assert not q[3].any() and torch.isfinite(qkv.float()).all()
    e = qkv[:0]
    pkv.qk_norm_rope(e[:, :40], e[:, 40:48], p[:0], fr, w[0], w[1])
    assert pkv.device_error() == 0


def test_bad_axis_is_recorded_and_its_pair_left(cuda_device):
    qkv, inv, pos, axis, w = _inputs(7, 4, 2, 1, 64, 64, 2, cuda_device, 50)
    axis[5] = 2
    q, k = qkv[:, :2], qkv[:, 2:3]
    qo, _ = pkv.qk_norm_rope(q, k, torch.from_numpy(pos).to(cuda_device), pkv.rope_frequencies(inv, cuda_device),
                             pair_axis=torch.from_numpy(axis).to(cuda_device))
    assert pkv.device_error() == 8 and pkv.device_error() == 0
    assert torch.equal(qo[..., 5], q[..., 5]) and torch.equal(qo[..., 37], q[..., 37])


def test_captured_and_on_another_stream(cuda_device):
    qkv, inv, pos, axis, w = _inputs(8, 9, 4, 2, 128, 128, 1, cuda_device, 500)
    q, k = qkv[:, :4], qkv[:, 4:6]
    fr, p = pkv.rope_frequencies(inv, cuda_device), torch.from_numpy(pos[0]).to(cuda_device)
    qo, ko = torch.zeros(9, 4, 128, dtype=torch.float16, device=cuda_device), torch.zeros(
        9, 2, 128, dtype=torch.float16, device=cuda_device)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        pkv.qk_norm_rope(q, k, p, fr, w[0], w[1], q_out=qo, k_out=ko)
    p.add_(7)
    g.replay()
    torch.cuda.synchronize()
    _check(qo, q, w[0], 1e-6, pos[:1] + 7, inv, np.zeros(64, int), False)


@pytest.mark.parametrize("change", ["dtype", "heads", "positions", "weight", "axis"])
def test_binding_refuses(cuda_device, change):
    qkv, inv, pos, axis, w = _inputs(9, 4, 2, 1, 64, 64, 1, cuda_device, 50)
    a = dict(q=qkv[:, :2], key=qkv[:, 2:3], positions=torch.from_numpy(pos).to(cuda_device),
             frequencies=pkv.rope_frequencies(inv, cuda_device))
    a.update({"dtype": dict(q=qkv[:, :2].float()), "heads": dict(q=qkv[:, ::2]), "positions": dict(positions=a["positions"][:, :3].contiguous()),
              "weight": dict(q_weight=w[0][:32].contiguous()), "axis": dict(pair_axis=torch.zeros(5, dtype=torch.int32, device=cuda_device))}[change])
    with pytest.raises(pkv.PkvError):
        pkv.qk_norm_rope(**a)


def test_rows_past_2_31_elements(cuda_device):
    T, H, D, n = 360000, 48, 128, 50
    big = torch.zeros(T, H, D, dtype=torch.float16, device=cuda_device)
    big[T - n:] = torch.randn(n, H, D, device=cuda_device)
    pos = torch.arange(T, dtype=torch.int32, device=cuda_device)
    f = pkv.rope_frequencies([10000.0 ** (-i / 64) for i in range(64)], cuda_device)
    small = big[T - n:].clone()
    want = pkv.qk_norm_rope(small[:, :40], small[:, 40:], pos[T - n:].clone(), f)
    pkv.qk_norm_rope(big[:, :40], big[:, 40:], pos, f, q_out=big[:, :40], k_out=big[:, 40:])
    assert pkv.device_error() == 0
    assert torch.equal(big[T - n:, :40], want[0]) and torch.equal(big[T - n:, 40:], want[1])


@pytest.mark.parametrize("T,H,Hk,D,R,axes,inter,norm", [(5001, 3, 1, 128, 128, 1, False, True), (4865, 1, 1, 64, 32, 3, True, True),
                                                        (4864, 8, 8, 128, 64, 2, True, False)])
def test_many_tokens_of_few_heads(cuda_device, T, H, Hk, D, R, axes, inter, norm):
    # two tokens to a warp, the last one alone
    test_against_oracle(cuda_device, T, H, Hk, D, R, axes, inter, norm)
