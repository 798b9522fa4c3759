"""Pins of the oracle of the operators around the attention module: gradients
against differences, 8-bit rounding against a search over all codes, closed
forms."""
import math

import numpy as np
import pytest

from oracle import layer_ref as R


def test_norm_of_a_constant_row():
    s, y = R.add_rms_norm(np.full((1, 8), 1.5), np.full((1, 8), 0.5), np.arange(8.0), 0.0, "f32")
    assert (s == 2.0).all() and np.allclose(y, np.arange(8.0), rtol=1e-15)


def test_sum_is_rounded_before_the_norm():
    s, _ = R.add_rms_norm(np.array([[256.0]]), np.array([[1.0]]), None, 1e-6, "bf16")
    assert s[0, 0] == 256.0  # a tie between 256 and 258: the even one


@pytest.mark.parametrize("weight", [True, False])
def test_norm_gradient_against_differences(weight):
    rng = np.random.default_rng(3)
    s, gy, gs = rng.normal(size=(3, 4, 16))
    w = 1 + rng.normal(size=16) if weight else None
    dx, dw = R.add_rms_norm_grad(s, gy, gs, w, 1e-3)

    def loss(s_, w_):
        return (R.add_rms_norm(s_, None, w_, 1e-3, "f32")[1] * gy).sum() + (s_ * gs).sum()
    e = 1e-6
    for i in [(0, 0), (1, 7), (3, 15)]:
        a, b = s.copy(), s.copy()
        a[i] += e
        b[i] -= e
        assert abs((loss(a, w) - loss(b, w)) / (2 * e) - dx[i]) < 1e-7
    for c in (0, 9):
        a = np.ones(16) if w is None else w.copy()
        b = a.copy()
        a[c] += e
        b[c] -= e
        assert abs((loss(s, a) - loss(s, b)) / (2 * e) - dw[c]) < 1e-7


def test_codes_are_the_nearest():
    rng = np.random.default_rng(5)
    mags = R.VALUES[:127]
    v = np.concatenate([mags, (mags[1:] + mags[:-1]) / 2, rng.uniform(0, 448, 500), 2.0 ** rng.uniform(-14, 8, 500)])
    v = np.concatenate([v, -v])
    codes = R.e4m3_code(v)
    for x, c in zip(v, codes):
        off = np.abs(R.VALUES[:127] - abs(x))
        best = np.flatnonzero(off == off.min())
        want = best[0] if len(best) == 1 or best[0] % 2 == 0 else best[1]
        assert c & 127 == want and (c >> 7) == (1 if math.copysign(1, x) < 0 else 0)


@pytest.mark.parametrize("top,byte", [(448.0, 127), (449.0, 128), (224.0, 126), (224.1, 127), (0.0, 0),
                                      (math.inf, 255), (math.nan, 255), (1.75 * 2.0 ** -119, 0),
                                      (2.0 ** -149, 0), (3.4e38, 247)])
def test_scale_bytes(top, byte):
    assert R.scale_byte(top) == byte


def test_words_and_bytes_are_each_others_reverse():
    rng = np.random.default_rng(6)
    b = rng.integers(0, 256, (5, 7)).astype(np.uint8)
    w = R.q8_words(b)
    assert w.shape == (2, 5) and (R.q8_bytes(w, 7 * 128) == b).all()
    assert (w[0, 3].view(np.uint32) >> 8 & 255) == b[3, 1] and (w[1].view(np.uint32) >> 24 == 0).all()


def test_a_value_is_off_by_at_most_half_a_step():
    rng = np.random.default_rng(7)
    x = rng.normal(size=(6, 272)) * 10.0 ** rng.uniform(-8, 8, (6, 1))
    for rows in (1, 128):
        codes, b = R.q8_write(x, rows)
        y = R.q8_read(codes, b)
        scale = np.repeat(2.0 ** (b.astype(float) - 127), 128, 1)[:, :272]
        assert (np.abs(y - x) <= np.maximum(np.abs(x) * 2.0 ** -4, scale * 2.0 ** -10)).all()


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "relu"])
def test_gated_gradients_against_differences(name):
    rng = np.random.default_rng(8)
    x, wg, wu, gh = (rng.normal(size=s) for s in ((3, 8), (8, 16), (8, 16), (3, 16)))
    _, g, u = R.gated_ff(x, wg, wu, name)
    dx, dwg, dwu = R.gated_ff_grad(x, wg, wu, g, u, gh, name)
    e = 1e-6
    for arr, grad, i in ((x, dx, (1, 5)), (wg, dwg, (2, 3)), (wu, dwu, (7, 15)), (x, dx, (0, 0))):
        was = arr[i]
        arr[i] = was + e
        up = (R.gated_ff(x, wg, wu, name)[0] * gh).sum()
        arr[i] = was - e
        down = (R.gated_ff(x, wg, wu, name)[0] * gh).sum()
        arr[i] = was
        assert abs((up - down) / (2 * e) - grad[i]) < 2e-7


def test_activations_at_known_points():
    assert R.act(0.0, "silu")[0] == 0 and R.act(0.0, "silu")[1] == 0.5
    assert abs(R.act(1.0, "gelu")[0] - 0.8413447460685429) < 1e-15
    assert abs(R.act(1.0, "gelu_tanh")[0] - 0.5 * (1 + math.tanh(math.sqrt(2 / math.pi) * 1.044715))) < 1e-15
    assert R.act(0.0, "relu")[1] == 0
