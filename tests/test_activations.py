"""The feed-forward product's activations far from zero, against fp64.

With z the exponential's argument (silu: g; gelu_tanh: 1.6 (g + 0.045 g^3), off by
4 u |z|, u = 2^-24): the exponential is off by (2 + 1.173 |z|) units of 2^-23 (bf16:
the documented bound of __expf; expf's is smaller), the division by two, the
products and the sum by three in all, so a factor of the activation is off by
(8 + 3.3 |z|) 2^-23 of itself. gelu: erfc is off by four units, its argument y by
2 u of itself, erfc by 2 y^2 times that (its logarithmic slope is below 2 y + 2 / y):
(8 + 4 y^2) 2^-23. A factor below fp32's normal range is off by up to 2^-149
besides, which g multiplies."""
import numpy as np
import pytest

from layer_helpers import ACTS, HALF, act_code, done, empty, host, own_status, upload
from oracle import layer_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    import torch
    from nystr_self_attention_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    import nystr_self_attention_gb300 as N
    own_status(N)


GATES = np.array([-104, -100, -95, -92, -90, -89, -88.5, -88, -87, -80, -60, -40, -30, -20, -14, -13, -12, -11, -10,
                  -9.5, -9, -8, -6, -4, -2, -1, -0.5, 0, 0.5, 1, 2, 4, 8, 16, 30, 60, 88, 90, 100, 104])


def relative(g, name):
    if name == "relu":
        return np.zeros_like(g)
    if name == "gelu":
        return (8 + 2 * g * g) * 2.0 ** -23
    z = g if name == "silu" else 1.5957691216057308 * (g + 0.044715 * g ** 3)
    return (8 + 3.3 * np.abs(z)) * 2.0 ** -23


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("T", [4, 100, 200])
def test_values(T, name, dtype):
    """g comes as it is: one of x's channels times one."""
    import nystr_self_attention_gb300 as N
    x, wg, wu = np.zeros((T, 16)), np.zeros((16, 40)), np.zeros((16, 40))
    x[:, 0], wg[0] = 1.0, GATES
    x[:, 1], wu[1] = 1.0, 1.0
    h = empty(T, 40, dtype)
    N.nystrom_gated_ff_fwd(upload(x, dtype), upload(wg, dtype), upload(wu, dtype), h, activation=act_code(N, name))
    done(N)
    g = R.rounded(GATES, dtype)
    with np.errstate(over="ignore"):
        want = R.act(g, name)[0]
    least = np.abs(g) * 2.0 ** -149 + 2.0 ** -149 + (2.0 ** -134 if dtype == "bf16" else 0)
    bound = (relative(g, name) + HALF[dtype]) * np.abs(want) + least
    assert (np.abs(host(h) - want) <= bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("T", [8, 136])
def test_slopes_of_large_gates(T, name, dtype):
    """dg = act'(g), du = act(g), read through the weights' gradients of an identity.
    Slopes of these gates are 0 or 1 (|g| e^-|g| is below 1e-127); the sigmoid's own
    error and the terms' are below 2^-20."""
    import nystr_self_attention_gb300 as N
    gates = np.array([-3e38, -1e30, -1e20, -4.5e19, -2e19, -1e10, -1e4, -300, 300, 1e4, 1e10, 2e19, 4.5e19, 1e20, 1e30, 3e38])
    g = R.rounded(np.repeat(gates[None], T, 0), dtype)
    one, eye, w = np.ones((T, 16)), np.eye(T), np.ones((T, 16))
    dwg, dwu = empty(T, 16, dtype), empty(T, 16, dtype)
    N.nystrom_gated_ff_bwd(upload(eye, dtype), upload(w, dtype), upload(w, dtype), upload(g, dtype), upload(one, dtype),
                           upload(one, dtype), None, dwg, dwu, activation=act_code(N, name))
    done(N)
    slope, value = (g > 0).astype(float), np.where(g > 0, g, 0.0)
    assert (np.abs(host(dwg) - slope) <= 2.0 ** -20 * slope).all()
    assert (np.abs(host(dwu) - value) <= (2.0 ** -20 + HALF[dtype]) * value).all()


def test_relu_gradients_against_differences():
    """Away from its corner: gh is 0 where a gate is nearer to 0 than the step can
    move it. The loss is of second degree there, so the difference is exact but for
    what g and u are off by, 20 u of the sums of their magnitudes (64 products summed
    in order by 8 warps, u = 2^-24), in both losses, and the like in dx itself."""
    import torch
    import nystr_self_attention_gb300 as N
    torch.manual_seed(3)
    T, d, f, e = 6, 64, 128, 2.0 ** -5
    x, wg, wu, gh = (torch.randn(s, device="cuda") for s in ((T, d), (d, f), (d, f), (T, f)))
    wg, wu = wg / 8, wu / 8
    h, g, u = (torch.empty(T, f, device="cuda") for _ in range(3))
    N.nystrom_gated_ff_fwd(x, wg, wu, h, g, u, activation=N.NYS_ACT_RELU)
    gh[g.abs() <= 2 * e * wg.abs().amax(0)] = 0.0
    assert float((gh != 0).float().mean()) > 0.8

    def loss(x_):
        N.nystrom_gated_ff_fwd(x_, wg, wu, h, activation=N.NYS_ACT_RELU)
        return float((h.double() * gh).sum())
    dx = torch.empty_like(x)
    N.nystrom_gated_ff_bwd(x, wg, wu, g, u, gh, dx, activation=N.NYS_ACT_RELU)
    eg, eu = (20 * 2.0 ** -24 * (x.abs() @ w.abs()) for w in (wg, wu))
    off = float((gh.abs() * (eg * u.abs() + eu * g.abs())).sum())
    for i in ((0, 0), (3, 17), (5, 63)):
        up, down = x.clone(), x.clone()
        up[i] += e
        down[i] -= e
        diff = (loss(up) - loss(down)) / (2 * e)
        assert abs(diff - float(dx[i])) <= 2 * off / (2 * e) + 2.0 ** -18
    done(N)
