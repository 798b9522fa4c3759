"""Pins of oracle/cache_ref.py by something other than itself: closed forms,
finite differences, brute force, exact rational arithmetic."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import cache_ref as C

RNG = np.random.default_rng(11)


def freqs(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


@pytest.mark.parametrize("pairs", [False, True])
def test_rotation_is_a_complex_product(pairs):
    z = RNG.standard_normal((2, 3, 5, 24))
    ang = RNG.standard_normal((2, 5, 8))
    y = C.rotate(z, ang, pairs)
    a, b = (slice(0, 16, 2), slice(1, 16, 2)) if pairs else (slice(0, 8), slice(8, 16))
    want = (z[..., a] + 1j * z[..., b]) * np.exp(1j * ang)[:, None]
    assert np.allclose(y[..., a], want.real) and np.allclose(y[..., b], want.imag)
    assert np.array_equal(y[..., 16:], z[..., 16:])


def test_scores_depend_on_the_distance_alone():
    q, k = RNG.standard_normal((2, 1, 1, 1, 16))
    f = freqs(16)
    dots = []
    for shift in (0, 1000):
        qa = C.rope_angles([[[7 + shift]]], f, [8])
        ka = C.rope_angles([[[3 + shift]]], f, [8])
        dots.append((C.rotate(q, qa, False) * C.rotate(k, ka, False)).sum())
    assert abs(dots[0] - dots[1]) < 1e-10


def test_axes_take_their_own_positions():
    pos = RNG.integers(0, 50, (3, 2, 4))
    ang = C.rope_angles(pos, [1.0, 0.5, 0.25, 2.0], [1, 2, 1])
    assert np.allclose(ang[..., 0], pos[0]) and np.allclose(ang[..., 1], pos[1] * 0.5)
    assert np.allclose(ang[..., 2], pos[1] * 0.25) and np.allclose(ang[..., 3], pos[2] * 2)


def test_norm_rows_closed_form():
    y = C.norm_rows(np.full((1, 1, 1, 8), 3.0), np.arange(8.0), 0.0)
    assert np.allclose(y, np.arange(8.0))


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("pairs", [False, True])
def test_gradients_are_those_of_differences(norm, pairs):
    x = RNG.standard_normal((2, 2, 3, 16))
    w, gy = RNG.standard_normal(16), RNG.standard_normal(x.shape)
    ang = RNG.standard_normal((2, 3, 6))
    loss = lambda x, w: (C.qk_norm_rope(x, w, ang, pairs, norm, 1e-3) * gy).sum()  # noqa: E731
    dx, dw = C.qk_norm_rope_grad(x, w, gy, ang, pairs, norm, 1e-3)
    h = 1e-6
    for at in [(0, 0, 0, 0), (1, 1, 2, 15), (0, 1, 1, 7), (1, 0, 2, 12)]:
        e = np.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-6
    if norm:
        for c in (0, 5, 15):
            e = np.zeros(16)
            e[c] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[c]) < 1e-5
    else:
        assert dw is None


def test_every_field_of_a_block_has_its_own_place():
    for d in (32, 64, 128):
        for byte in (C.key_byte, C.value_byte):
            places = [(byte(r, c, d), c % 2) for r in range(16) for c in range(d)]
            assert len(set(places)) == 16 * d
            assert min(p[0] for p in places) == 0 and max(p[0] for p in places) == 8 * d - 1


def test_quantise_against_rational_arithmetic():
    x = RNG.standard_normal((40, 32)).astype(np.float32) * np.exp2(RNG.integers(-140, 100, (40, 1))).astype(np.float32)
    x[0] = 0
    x[1, 3] = np.float32(3.4e38)
    x[2] = np.float32(2.0 ** -149)
    codes, bits = C.quantise(x)
    for row, cs, sb in zip(x, codes, bits):
        top = max(abs(Fraction(float(v))) for v in row)
        s = Fraction(float(C.bf16_value(sb[0])))
        # 1/7 and the product in fp32, then truncated: an fp32 step above top/7 at most
        assert s <= top / 7 * (1 + Fraction(1, 2 ** 23))
        assert s >= top / 7 * (1 - Fraction(1, 2 ** 7)) - Fraction(1, 2 ** 133)
        for v, c in zip(row, cs):
            if s == 0:
                assert c == 0
                continue
            t = Fraction(float(v)) / s
            near = min(range(-30, 31), key=lambda i: (abs(t - i), i % 2))
            assert c == max(-7, min(7, near))


def test_values_stay_within_half_a_scale_and_never_grow():
    x = RNG.standard_normal((500, 64)).astype(np.float32)
    codes, bits = C.quantise(x)
    y = C.dequantise(codes, bits)
    s = np.repeat(C.bf16_value(bits), 32, -1)
    assert (np.abs(y - x) <= s / 2 * (1 + 1e-12)).all()
    top = np.abs(x).reshape(500, 2, 32).max(-1)
    assert (np.abs(y).reshape(500, 2, 32).max(-1) <= top * (1 + 2.0 ** -23)).all()


def test_not_finite_blocks_read_back_as_nan():
    x = np.ones((3, 64), np.float32)
    x[0, 5], x[1, 40], x[2, 0] = np.inf, np.nan, -np.inf
    y = C.dequantise(*C.quantise(x))
    assert np.isnan(y[0, :32]).all() and np.isfinite(y[0, 32:]).all()
    assert np.isnan(y[1, 32:]).all() and np.isfinite(y[1, :32]).all()
    assert np.isnan(y[2, :32]).all()


def small_cache(d=32, Hk=2, page=32, B=2, pages=3):
    table = RNG.permutation(B * pages).reshape(B, pages)
    raw = RNG.integers(0, 256, B * pages * Hk * page // 16 * 18 * d)
    return C.Cache(raw, table, page, Hk, d)


def test_cache_keeps_what_it_is_given_and_nothing_else():
    c = small_cache()
    before = c.raw.copy()
    k, v = RNG.standard_normal((2, 2, 2, 21, 32)).astype(np.float32)
    c.write(k, v, [30, 5], [21, 7])
    for b, start, count in ((0, 30, 21), (1, 5, 7)):
        for i in range(count):
            K, V = c.token(b, start + i)
            assert np.array_equal(K, C.dequantise(*C.quantise(k[b, :, i])))
            assert np.array_equal(V, C.dequantise(*C.quantise(v[b, :, i])))
    changed = (c.raw != before).sum()
    assert 0 < changed <= (21 + 7) * 2 * 2 * 18
    assert c.token(0, 96) is None and c.token(0, -1) is None


def test_attention_is_a_mean_for_equal_keys_and_masks_by_position():
    c = small_cache()
    k = np.ones((2, 2, 40, 32), np.float32)
    v = RNG.standard_normal((2, 2, 40, 32)).astype(np.float32)
    c.write(k, v, [0, 0], [40, 40])
    q = RNG.standard_normal((2, 4, 3, 32))
    out, _, _ = C.attention(q, c, [40, 2])
    vals = np.stack([c.token(0, t)[1] for t in range(40)])
    for i in range(3):
        assert np.allclose(out[0, 0, i], vals[:38 + i, 0].mean(0))
    one = np.stack([c.token(1, t)[1] for t in range(2)])
    assert np.array_equal(out[1, 0, 0], np.zeros(32))  # before the first token
    assert np.allclose(out[1, 3, 1], one[0, 1]) and np.allclose(out[1, 3, 2], one[:, 1].mean(0))
    whole, _, _ = C.attention(q, c, [40, 0], causal=False)
    assert np.allclose(whole[0, 2, 0], vals[:, 1].mean(0)) and (whole[1] == 0).all()
