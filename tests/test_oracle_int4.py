"""The four-bit cache's oracle against the definitions' own consequences, the host helper
pkv_rope_frequencies against exact arithmetic, and the new entry points' refusals (CPU)."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import int4_cache as o4
from paged_kv_cache_73_gb300 import _build
from paged_kv_cache_73_gb300 import binding as pkv


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


def test_row_stands_within_half_a_step():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((200, 64)) * 10.0 ** rng.uniform(-3, 3, (200, 1))).astype(np.float16)
    n, s, z = o4.quantise_rows(x)
    y = z.astype(np.float64)[:, None] + s.astype(np.float64)[:, None] * n
    # half a step, and where the greatest value passes 15.5 steps after the scale's rounding the rest
    span = x.max(-1).astype(np.float64) - x.min(-1)
    over = np.maximum(span - 15.5 * s.astype(np.float64), 0)
    assert (np.abs(y - x) <= s.astype(np.float64)[:, None] / 2 + over[:, None]).all()
    assert (n.min(-1) == 0).all()


def test_halves_go_to_even_and_flat_rows_are_exact():
    x = np.zeros((1, 64), np.float16)
    x[0, :5] = [15, 0.5, 1.5, 2.5, 14.5]                     # scale 1: halves to even
    n, s, z = o4.quantise_rows(x)
    assert s[0] == 1 and z[0] == 0 and n[0, :5].tolist() == [15, 0, 2, 2, 14]
    n, s, z = o4.quantise_rows(np.full((1, 64), 3.25, np.float16))
    assert s[0] == 0 and z[0] == 3.25 and not n.any()


def test_store_and_values_round_trip():
    rng = np.random.default_rng(2)
    rows = rng.standard_normal((6, 2, 64)).astype(np.float16)
    pool = o4.empty_pool(3, 2, 4, 64)
    slots = [0, 5, -1, 11, 2, 7]
    o4.store(pool, rows, slots, 4)
    vals = o4.pool_values(pool, 4)
    for t, slot in enumerate(slots):
        if slot >= 0:
            n, s, z = o4.quantise_rows(rows[t])
            want = z.astype(np.float64)[:, None] + s.astype(np.float64)[:, None] * n
            assert np.array_equal(vals[slot // 4, :, slot % 4], want)


def test_rotation_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 1, 64))
    inv = 10000.0 ** (-np.arange(32) / 32)
    pos = np.array([[0, 5, 1000000, 2147483647]])
    y, _ = o4.norm_rope(x, None, 0.0, pos, inv, np.zeros(32, int), False)
    assert np.allclose(y[0], x[0], atol=1e-15)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-12)
    z = x[:, 0, :32] + 1j * x[:, 0, 32:]
    small = z[1] * np.exp(1j * 5 * inv)
    assert np.allclose(y[1, 0, :32] + 1j * y[1, 0, 32:], small, atol=1e-12)


def test_rope_frequencies_are_turns_modulo_one(lib):
    inv = np.concatenate([10000.0 ** (-np.arange(64) / 64), [0.0, 7.0, 2 * math.pi, math.pi, -math.pi, -0.25, 1e-12]])
    got = pkv.rope_frequencies(inv, device="cpu").numpy()
    for f, g in zip(inv, got):
        want = o4.turns_of(f)
        off = (Fraction(int(g), 2 ** 64) - want) % 1
        # fp64 division by 2 pi and the removal of whole turns: three roundings of 2^-53 relative;
        # the result is a whole number of 2^-64 turns: half a unit more
        assert min(off, 1 - off) <= abs(want) * Fraction(4, 2 ** 53) + Fraction(1, 2 ** 65)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rope_frequencies_refuse(lib, bad):
    with pytest.raises(pkv.PkvError) as e:
        pkv.rope_frequencies([1.0, bad], device="cpu")
    assert e.value.status == pkv.PKV_ERR_INVALID_ARG


def _rope(lib, **kw):
    a = dict(q=16, k=16, qw=None, kw=None, eps=1e-6, pos=16, axes=1, fr=16, pa=None, R=64, inter=0, T=3, H=4, Hk=2, D=64,
             qs=256, ks=128, qo=4096, ko=4096, qos=256, kos=128)
    a.update(kw)
    return lib.pkv_qk_norm_rope(a["q"], a["k"], a["qw"], a["kw"], a["eps"], a["pos"], a["axes"], a["fr"], a["pa"],
                                a["R"], a["inter"], a["T"], a["H"], a["Hk"], a["D"], a["qs"], a["ks"], a["qo"], a["ko"],
                                a["qos"], a["kos"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), pkv.PKV_ERR_UNSUPPORTED),
    (dict(R=24), pkv.PKV_ERR_UNSUPPORTED),
    (dict(R=0), pkv.PKV_ERR_UNSUPPORTED),
    (dict(R=80), pkv.PKV_ERR_UNSUPPORTED),                 # past the head
    (dict(axes=0), pkv.PKV_ERR_INVALID_ARG),
    (dict(axes=9), pkv.PKV_ERR_UNSUPPORTED),
    (dict(T=-1), pkv.PKV_ERR_INVALID_ARG),
    (dict(Hk=0), pkv.PKV_ERR_INVALID_ARG),
    (dict(eps=-1.0), pkv.PKV_ERR_INVALID_ARG),
    (dict(eps=float("nan")), pkv.PKV_ERR_INVALID_ARG),
    (dict(pos=None), pkv.PKV_ERR_INVALID_ARG),
    (dict(fr=None), pkv.PKV_ERR_INVALID_ARG),
    (dict(q=24), pkv.PKV_ERR_INVALID_ARG),
    (dict(qw=8), pkv.PKV_ERR_INVALID_ARG),
    (dict(qs=248), pkv.PKV_ERR_INVALID_ARG),               # shorter than a token
    (dict(ks=132), pkv.PKV_ERR_INVALID_ARG),               # not a multiple of 8
    (dict(qo=16, qos=512), pkv.PKV_ERR_INVALID_ARG),       # in place with another stride
    (dict(T=0, q=None), pkv.PKV_OK),
])
def test_qk_norm_rope_refuses(lib, kw, status):
    assert _rope(lib, **kw) == status
    if status != pkv.PKV_OK:
        assert lib.pkv_last_error()


def _write(lib, **kw):
    a = dict(k=16, v=16, kc=16, vc=16, slots=16, T=2, H=2, D=64, B=16, N=4, ks=128, vs=128)
    a.update(kw)
    return lib.pkv_reshape_and_cache_int4(a["k"], a["v"], a["kc"], a["vc"], a["slots"], a["T"], a["H"], a["D"], a["B"],
                                          a["N"], a["ks"], a["vs"], None)


def _gather(lib, **kw):
    a = dict(k=16, v=16, kc=16, vc=16, slots=16, T=2, H=2, D=64, B=16, N=4)
    a.update({x: y for x, y in kw.items() if x in a})
    return lib.pkv_gather_cache_int4(a["kc"], a["vc"], a["slots"], a["k"], a["v"], a["T"], a["H"], a["D"], a["B"], a["N"],
                                     None)


@pytest.mark.parametrize("call", [_write, _gather])
@pytest.mark.parametrize("kw,status", [
    (dict(D=96), pkv.PKV_ERR_UNSUPPORTED),
    (dict(B=12), pkv.PKV_ERR_UNSUPPORTED),
    (dict(H=0), pkv.PKV_ERR_INVALID_ARG),
    (dict(N=0), pkv.PKV_ERR_INVALID_ARG),
    (dict(T=-1), pkv.PKV_ERR_INVALID_ARG),
    (dict(k=None), pkv.PKV_ERR_INVALID_ARG),
    (dict(slots=None), pkv.PKV_ERR_INVALID_ARG),
    (dict(vc=8), pkv.PKV_ERR_INVALID_ARG),
    (dict(T=0, k=None), pkv.PKV_OK),
])
def test_int4_rows_refuse(lib, call, kw, status):
    assert call(lib, **kw) == status
    if status != pkv.PKV_OK:
        assert lib.pkv_last_error()


def test_int4_write_refuses_strides(lib):
    assert _write(lib, ks=120) == pkv.PKV_ERR_INVALID_ARG
    assert _write(lib, vs=132) == pkv.PKV_ERR_INVALID_ARG


def test_int4_copy_and_swap_refuse(lib):
    assert lib.pkv_copy_blocks_int4(None, None, 1, 16, 1, 2, 64, 16, 4, None) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_copy_blocks_int4(None, None, 1, 16, 1, 2, 96, 16, 4, None) == pkv.PKV_ERR_UNSUPPORTED
    assert lib.pkv_copy_blocks_int4(None, None, 0, None, 0, 2, 64, 16, 4, None) == pkv.PKV_OK
    assert lib.pkv_swap_blocks_int4(None, None, None, None, 1, 16, 1, 2, 64, 16, 4, 4, None) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_swap_blocks_int4(None, None, None, None, 1, 16, 0, 2, 64, 16, 4, 4, None) == pkv.PKV_OK


def _decode(lib, **kw):
    a = dict(q=16, k=16, v=16, tables=16, lens=16, S=2, H=4, Hk=2, D=64, N=8, maxb=4, scale=0.125, B=16, out=16,
             ws=None, ws_bytes=0)
    a.update(kw)
    return lib.pkv_paged_attention_decode_int4(a["q"], a["k"], a["v"], a["tables"], a["lens"], a["S"], a["H"], a["Hk"],
                                               a["D"], a["N"], a["maxb"], a["scale"], a["B"], a["out"], a["ws"],
                                               a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), pkv.PKV_ERR_UNSUPPORTED),
    (dict(B=12), pkv.PKV_ERR_UNSUPPORTED),
    (dict(Hk=0), pkv.PKV_ERR_INVALID_ARG),
    (dict(Hk=3), pkv.PKV_ERR_INVALID_ARG),                 # 4 heads over 3
    (dict(S=-1), pkv.PKV_ERR_INVALID_ARG),
    (dict(S=70000), pkv.PKV_ERR_UNSUPPORTED),
    (dict(maxb=1 << 27), pkv.PKV_ERR_UNSUPPORTED),
    (dict(q=None), pkv.PKV_ERR_INVALID_ARG),
    (dict(v=8), pkv.PKV_ERR_INVALID_ARG),
    (dict(scale=float("nan")), pkv.PKV_ERR_INVALID_ARG),
    (dict(maxb=4096), pkv.PKV_ERR_WORKSPACE),              # split, and no workspace
    (dict(S=0, q=None), pkv.PKV_OK),
])
def test_decode_int4_refuses(lib, kw, status):
    assert _decode(lib, **kw) == status
    if status != pkv.PKV_OK:
        assert lib.pkv_last_error()


def test_decode_int4_oracle_groups_heads():
    rng = np.random.default_rng(4)
    kp, vp = o4.empty_pool(4, 2, 4, 64), o4.empty_pool(4, 2, 4, 64)
    rows = rng.standard_normal((2, 7, 2, 64)).astype(np.float16)
    slots = [9, 10, 11, 8, 2, 3, 1]
    for pool, x in ((kp, rows[0]), (vp, rows[1])):
        o4.store(pool, x, slots, 4)
    tables, lens = np.array([[2, 0]], np.int32), np.array([8], np.int32)
    q = rng.standard_normal((1, 6, 64)).astype(np.float16)
    out = o4.paged_decode_attention(q, kp, vp, tables, lens, 0.2, 4)
    k, v = (np.concatenate([o4.pool_values(p, 4)[2], o4.pool_values(p, 4)[0]], 1) for p in (kp, vp))
    for h in range(6):
        w = np.exp(0.2 * k[h // 3] @ q[0, h].astype(np.float64))
        assert np.allclose(out[0, h], w @ v[h // 3] / w.sum(), rtol=1e-12)


def _prompt(lib, **kw):
    a = dict(q=16, k=16, v=16, qs=16, ks=None, S=2, T=8, Tk=8, maxq=4, H=4, Hk=2, D=64, sq=256, sk=128, sv=128, scale=0.1,
             out=16)
    a.update(kw)
    return lib.pkv_prompt_attention(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["S"], a["T"], a["Tk"], a["maxq"], a["H"],
                                    a["Hk"], a["D"], a["sq"], a["sk"], a["sv"], a["scale"], a["out"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), pkv.PKV_ERR_UNSUPPORTED),
    (dict(Hk=0), pkv.PKV_ERR_INVALID_ARG),
    (dict(Hk=3), pkv.PKV_ERR_INVALID_ARG),
    (dict(T=-1), pkv.PKV_ERR_INVALID_ARG),
    (dict(Tk=0), pkv.PKV_ERR_INVALID_ARG),                 # queries without keys
    (dict(S=70000), pkv.PKV_ERR_UNSUPPORTED),
    (dict(qs=None), pkv.PKV_ERR_INVALID_ARG),
    (dict(k=40), pkv.PKV_ERR_INVALID_ARG),
    (dict(sk=64), pkv.PKV_ERR_INVALID_ARG),
    (dict(sq=260), pkv.PKV_ERR_INVALID_ARG),
    (dict(scale=0.0), pkv.PKV_ERR_INVALID_ARG),
    (dict(T=0, q=None), pkv.PKV_OK),
    (dict(S=0, q=None), pkv.PKV_OK),
])
def test_prompt_attention_refuses(lib, kw, status):
    assert _prompt(lib, **kw) == status
    if status != pkv.PKV_OK:
        assert lib.pkv_last_error()


@pytest.mark.parametrize("kw", [
    dict(T=(1 << 26) + 1),
    dict(Tk=(1 << 26) + 1),
    dict(T=1 << 26, Tk=1 << 26, maxq=1 << 26, H=65535, Hk=1, sq=65535 * 64, sk=64, sv=64),     # query tiles of all heads
])
def test_prompt_attention_refuses_what_is_too_large(lib, kw):
    assert _prompt(lib, **kw) == pkv.PKV_ERR_UNSUPPORTED and b"more than" in lib.pkv_last_error()
