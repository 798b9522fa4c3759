"""GPU parity of the gated feed-forward product and its gradients against the
fp64 oracle.

With whole numbers as inputs and RELU, every product and partial sum is exact in
fp32, so results have to be the oracle's, rounded once: that pins which elements
meet. Otherwise, with u = 2^-24 and A the sum of magnitudes of a product: the
matrix units take 16 products at a time into a sum that they cut off, 2 u A a
step; bf16 sums run over all K, fp32 ones over six times 64 products, whose terms
leave out 3 u A, and are then added: E = (K / 8 + 20) u A, fp32 (48 + 3 + K / 64 +
20) u A. Slopes of the activations are at most 1.13; their own error is 2^-17 of
themselves (bf16: __expf's argument, up to 30 here, at 2^-23 each) or 16 u."""
import numpy as np
import pytest

from layer_helpers import ACTS, HALF, U, act_code, done, empty, host, own_status, untouched, upload
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


def weight(w, dtype, order, pad=0):
    return upload(w, dtype, pad) if order == "in_out" else upload(w.T, dtype, pad).T


def weight_out(d, f, dtype, order, pad=0):
    return empty(d, f, dtype, pad) if order == "in_out" else empty(f, d, dtype, pad).T


SIZES = [(1, 8, 8), (1, 264, 1032), (2, 128, 64), (5, 1040, 24), (16, 520, 264), (17, 72, 776), (32, 64, 128),
         (48, 264, 136), (64, 1000, 512), (65, 136, 264), (128, 512, 1000), (129, 64, 128), (200, 1544, 72),
         (300, 264, 520), (777, 128, 1160), (1025, 392, 264), (4000, 72, 136)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("order", ["in_out", "out_in"])
@pytest.mark.parametrize("T,d,f", SIZES)
def test_whole_numbers(T, d, f, order, dtype):
    import nystr_self_attention_gb300 as N
    rng = np.random.default_rng(T + d + f)
    x, wg, wu = (rng.integers(-2, 3, s).astype(float) for s in ((T, d), (d, f), (d, f)))
    h, g, u = R.gated_ff(x, wg, wu, "relu")
    tx, tg, tu = upload(x, dtype, 16), weight(wg, dtype, order, 8), weight(wu, dtype, order, 8)
    th, tgate, tup = empty(T, f, dtype, 8), empty(T, f, dtype, 24), empty(T, f, dtype, 16)
    N.nystrom_gated_ff_fwd(tx, tg, tu, th, tgate, tup, activation=N.NYS_ACT_RELU)
    done(N)
    assert (host(tgate) == R.rounded(g, dtype)).all() and (host(tup) == R.rounded(u, dtype)).all()
    assert (host(th) == R.rounded(h, dtype)).all()
    assert untouched(th, f) and untouched(tgate, f) and untouched(tup, f)
    only = empty(T, f, dtype)
    N.nystrom_gated_ff_fwd(tx, tg, tu, only, activation=N.NYS_ACT_RELU)
    assert (host(only) == R.rounded(h, dtype)).all()

    g, u, gh = (rng.integers(-3, 4, (T, f)).astype(float) for _ in range(3))
    dx, dwg, dwu = R.gated_ff_grad(x, wg, wu, g, u, gh, "relu")
    tdx = empty(T, d, dtype, 8)
    tdg, tdu = weight_out(d, f, dtype, order, 16), weight_out(d, f, dtype, order, 16)
    args = (tx, tg, tu, upload(g, dtype, 8), upload(u, dtype), upload(gh, dtype, 16))
    N.nystrom_gated_ff_bwd(*args, tdx, tdg, tdu, activation=N.NYS_ACT_RELU)
    done(N)
    assert (host(tdx) == R.rounded(dx, dtype)).all()
    assert (host(tdg) == R.rounded(dwg, dtype)).all() and (host(tdu) == R.rounded(dwu, dtype)).all()
    assert untouched(tdx, d)
    for t in (tdg, tdu):
        assert untouched(t if order == "in_out" else t.T, f if order == "in_out" else d)
    # dx alone, the weights' gradients alone
    dx2, dg2, du2 = empty(T, d, dtype), weight_out(d, f, dtype, order), weight_out(d, f, dtype, order)
    N.nystrom_gated_ff_bwd(*args, dx2, activation=N.NYS_ACT_RELU)
    N.nystrom_gated_ff_bwd(*args, dw_gate=dg2, dw_up=du2, activation=N.NYS_ACT_RELU)
    done(N)
    assert (host(dx2) == host(tdx)).all() and (host(dg2) == host(tdg)).all() and (host(du2) == host(tdu)).all()


def product_error(A, K, dtype):
    return (K / 8 + 20) * U * A if dtype == "bf16" else (71 + K / 64) * U * A


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("T", [3, 100, 260])
def test_forward_of_any_numbers(T, name, dtype):
    import nystr_self_attention_gb300 as N
    rng = np.random.default_rng(T)
    d, f = 1032, 520
    x = R.rounded(rng.normal(size=(T, d)), dtype)
    wg, wu = (R.rounded(rng.normal(size=(d, f)) * 2 / np.sqrt(d), dtype) for _ in range(2))
    h, g, u = R.gated_ff(x, wg, wu, name)
    a = R.act(g, name)[0]
    th, tg, tu = (empty(T, f, dtype) for _ in range(3))
    N.nystrom_gated_ff_fwd(upload(x, dtype), upload(wg, dtype), upload(wu, dtype), th, tg, tu,
                           activation=act_code(N, name))
    done(N)
    eg, eu = (product_error(np.abs(x) @ np.abs(w), d, dtype) for w in (wg, wu))
    half, ea = HALF[dtype], 2.0 ** -17 if dtype == "bf16" else 16 * U
    assert (np.abs(host(tg) - g) <= eg + half * np.abs(g)).all()
    assert (np.abs(host(tu) - u) <= eu + half * np.abs(u)).all()
    bound = 1.13 * eg * (np.abs(u) + eu) + np.abs(a) * eu + (ea + half) * np.abs(h)
    assert (np.abs(host(th) - h) <= bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("T", [3, 100, 260])
def test_backward_of_any_numbers(T, name, dtype):
    """dg and du are off by their rounding to bf16 (fp32: 3 u of terms left out)
    and by the activation's error, 2^-17 or 16 u of gh u; those errors enter the
    products, whose own are as above over 2 f or T."""
    import nystr_self_attention_gb300 as N
    rng = np.random.default_rng(T + 1)
    d, f = 264, 1032
    x, g, u, gh = (R.rounded(rng.normal(size=s) * k, dtype) for s, k in
                   (((T, d), 1), ((T, f), 2), ((T, f), 1), ((T, f), 1)))
    wg, wu = (R.rounded(rng.normal(size=(d, f)) / np.sqrt(d), dtype) for _ in range(2))
    a, slope = R.act(g, name)
    dg, du = gh * u * slope, gh * a
    ea = 2.0 ** -17 if dtype == "bf16" else 16 * U
    half = HALF[dtype]
    off_g, off_u = (half + ea) * np.abs(dg) + ea * np.abs(gh * u), (half + ea) * np.abs(du) + ea * np.abs(gh * a)
    dx, dwg, dwu = R.gated_ff_grad(x, wg, wu, g, u, gh, name)
    tdx, tdg, tdu = empty(T, d, dtype), empty(d, f, dtype), empty(d, f, dtype)
    N.nystrom_gated_ff_bwd(upload(x, dtype), upload(wg, dtype), upload(wu, dtype), upload(g, dtype), upload(u, dtype),
                           upload(gh, dtype), tdx, tdg, tdu, activation=act_code(N, name))
    done(N)
    A = np.abs(dg) @ np.abs(wg).T + np.abs(du) @ np.abs(wu).T
    bound = off_g @ np.abs(wg).T + off_u @ np.abs(wu).T + product_error(A, 2 * f, dtype) + half * np.abs(dx)
    assert (np.abs(host(tdx) - dx) <= bound * 1.01).all()
    for t, want, off, dd in ((tdg, dwg, off_g, dg), (tdu, dwu, off_u, du)):
        A = np.abs(x).T @ np.abs(dd)
        bound = np.abs(x).T @ off + product_error(A, T, dtype) + half * np.abs(want)
        assert (np.abs(host(t) - want) <= bound * 1.01).all()


@pytest.mark.parametrize("name", ACTS)
def test_gradients_against_differences(name):
    """Central differences of the kernel's own forward pass in fp32: step 2^-5,
    third derivatives of act(g) u below 4 times the weights' cubes."""
    import torch
    import nystr_self_attention_gb300 as N
    torch.manual_seed(3)
    T, d, f, e = 6, 64, 128, 2.0 ** -5
    x, wg, wu, gh = (torch.randn(s, device="cuda") for s in ((T, d), (d, f), (d, f), (T, f)))
    wg, wu = wg / 8, wu / 8
    if name == "relu":
        return  # no differences across its corner
    h, g, u = (torch.empty(T, f, device="cuda") for _ in range(3))
    act = act_code(N, name)

    def loss(x_):
        N.nystrom_gated_ff_fwd(x_, wg, wu, h, g, u, activation=act)
        return float((h.double() * gh).sum())
    loss(x)
    dx = torch.empty_like(x)
    N.nystrom_gated_ff_bwd(x, wg, wu, g.clone(), u.clone(), gh, dx, activation=act)
    for i in ((0, 0), (3, 17), (5, 63)):
        up, down = x.clone(), x.clone()
        up[i] += e
        down[i] -= e
        diff = (loss(up) - loss(down)) / (2 * e)
        # e^2 / 6 of the third derivative: |gh| (4 |u| |wg|^3 + 6 |wg|^2 |wu|), summed
        third = float((gh[i[0]].abs() * (4 * (u[i[0]].abs() + 1) * wg[i[1]].abs() ** 3
                                         + 6 * wg[i[1]].abs() ** 2 * wu[i[1]].abs())).sum())
        assert abs(diff - float(dx[i])) <= e * e / 6 * third + 1e-4
    done(N)


@pytest.mark.parametrize("T", [4, 300])
def test_special_values_stay_in_their_rows(T):
    import torch
    import nystr_self_attention_gb300 as N
    rng = np.random.default_rng(1)
    x = rng.normal(size=(T, 72))
    x[2, 7] = np.nan
    w = rng.normal(size=(72, 136))
    h = empty(T, 136, "bf16")
    N.nystrom_gated_ff_fwd(upload(x, "bf16"), upload(w, "bf16"), upload(w, "bf16"), h)
    done(N)
    assert torch.isnan(h[2]).all() and not torch.isnan(h[:2]).any() and not torch.isnan(h[3:]).any()


def test_large_gates():
    """act of very negative and very positive g: no NaN, and the limits."""
    import nystr_self_attention_gb300 as N
    x = np.zeros((4, 8))
    x[:, 0] = (-1e4, -30, 30, 1e4)
    w = np.zeros((8, 8))
    w[0] = 1.0
    for dtype in ("bf16", "f32"):
        for name in ACTS:
            h = empty(4, 8, dtype)
            N.nystrom_gated_ff_fwd(upload(x, dtype), upload(w, dtype), upload(np.abs(w) * np.sign(1.0), dtype), h,
                                   activation=act_code(N, name))
            done(N)
            want = R.act(x[:, :1], name)[0] * x[:, :1]
            assert np.isfinite(host(h)).all()
            assert (np.abs(host(h) - want) <= 2.0 ** -7 * np.abs(want) + 1e-9).all()


def test_refusals_in_python():
    import torch
    import nystr_self_attention_gb300 as N
    x, w, h = (torch.zeros(s, device="cuda") for s in ((4, 64), (64, 128), (4, 128)))
    with pytest.raises(ValueError):
        N.nystrom_gated_ff_fwd(x, w, torch.zeros(128, 64, device="cuda").T, h)  # the other layout
    with pytest.raises(ValueError):
        N.nystrom_gated_ff_fwd(x, w[:32], w, h)
    with pytest.raises(ValueError):
        N.nystrom_gated_ff_fwd(x, w, w.bfloat16(), h)
    with pytest.raises(ValueError):
        N.nystrom_gated_ff_fwd(x, w, w, h, gate=h)
    with pytest.raises(ValueError):
        N.nystrom_gated_ff_fwd(x, w, w, h[:, :64])
    with pytest.raises(ValueError):
        N.nystrom_gated_ff_bwd(x, w, w, h, h, h, dw_gate=w)
    with pytest.raises(N.NystromError):
        N.nystrom_gated_ff_bwd(x, w, w, h, h, h)
    with pytest.raises(N.NystromError):
        N.nystrom_gated_ff_fwd(x, w, w, h, activation=9)
