"""GPU parity of the residual's addition with its norm, and of their gradients,
against the fp64 oracle.

Bounds, with u = 2^-24. A row's sum of squares is summed along at most 32 fused
multiply-adds of a thread, five shuffles and 16 partial sums, each off by u of
the sum: 53 u; the mean, eps and rsqrt add 1 + 1 + 4 u, and the square root
halves all but the last: r is off by at most 32 u. y adds two products and the
rounding to dtype: |y| (36 u + half). dx: r (w g - h mean(w g h)), whose mean is
a sum like the other one: M (53 + 3) u with M = mean |w g h|; in all
r (|w g| + |h| M) (64 + 56) u, plus |gs| u and the rounding. dweight: products
off by 36 u, summed along rows / groups steps of a thread, 8 groups, then at most
10 CTAs and 5 shuffles: sum |g h| (60 + rows / groups) u, with at least one row
per group: taken with rows / 100 (rows here are at most 5000 and the grid has at
least 300 groups)."""
import numpy as np
import pytest

from layer_helpers import HALF, U, done, eight, empty, host, own_status, untouched, upload
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


def inputs(rows, d, dtype, seed=1):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, d))
    r = rng.normal(size=(rows, d)) * (1 + 12 * (rng.random(d) > 0.97))
    return R.rounded(x, dtype), R.rounded(r, dtype), (1 + 0.3 * rng.normal(size=d)).astype(np.float32)


WIDTHS = [8, 64, 248, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384]


def forward_bound(y, dtype):
    return np.abs(y) * (36 * U + HALF[dtype]) + 1e-37


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_forward(d, dtype):
    import torch
    import nystr_self_attention_gb300 as N
    for rows, pad in ((1, 0), (7, 16), (700 if d < 5000 else 400, 8)):
        x, r, w = inputs(rows, d, dtype, d + rows)
        s, y = R.add_rms_norm(x, r, w, 1e-6, dtype)
        tx, tr = upload(x, dtype, pad), upload(r, dtype, 2 * pad)
        ts, ty = empty(rows, d, dtype, pad), empty(rows, d, dtype, 3 * pad)
        N.nystrom_add_rms_norm_fwd(tx, tr, torch.from_numpy(w).cuda(), ts, ty)
        done(N)
        assert (host(ts) == s).all()
        assert (np.abs(host(ty) - y) <= forward_bound(y, dtype)).all()
        assert untouched(ts, d) and untouched(ty, d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_without_its_options(dtype):
    import nystr_self_attention_gb300 as N
    x, r, _ = inputs(33, 776, dtype)
    for res, keep in ((False, False), (True, False)):
        s, y = R.add_rms_norm(x, r if res else None, None, 0.1, dtype)
        ty = empty(33, 776, dtype)
        N.nystrom_add_rms_norm_fwd(upload(x, dtype), upload(r, dtype) if res else None, None, None, ty, eps=0.1)
        done(N)
        assert (np.abs(host(ty) - y) <= forward_bound(y, dtype)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [72, 2048, 9000])
def test_in_place(d, dtype):
    import torch
    import nystr_self_attention_gb300 as N
    x, r, w = inputs(1500, d, dtype)
    s, y = R.add_rms_norm(x, r, w, 1e-6, dtype)
    tw = torch.from_numpy(w).cuda()
    for sum_over_x in (True, False):
        tx, tr = upload(x, dtype), upload(r, dtype)
        ts, ty = (tx, tr) if sum_over_x else (tr, tx)
        N.nystrom_add_rms_norm_fwd(tx, tr, tw, ts, ty)
        done(N)
        assert (host(ts) == s).all() and (np.abs(host(ty) - y) <= forward_bound(y, dtype)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 128, 144, 1024, 2064, 4096, 16384])
def test_eight_bits(d, dtype):
    """A code is the nearest to a y that is off by 36 u: half a step and that, in
    the scale of a largest value that is off by 36 u too."""
    import torch
    import nystr_self_attention_gb300 as N
    for rows, pad in ((1, 0), (5, 16), (333, 0)):
        x, r, w = inputs(rows, d, dtype, d + rows)
        s, y = R.add_rms_norm(x, r, w, 1e-6, dtype)
        q = eight(N, rows, d, pad)
        ts = empty(rows, d, dtype)
        N.nystrom_add_rms_norm_fwd(upload(x, dtype), upload(r, dtype), torch.from_numpy(w).cuda(), ts, q)
        done(N)
        assert (host(ts) == s).all()
        bytes_ = R.q8_bytes(q.scales.cpu().numpy(), d)
        blocks = bytes_.shape[1]
        assert (R.q8_words(bytes_) == q.scales.cpu().numpy()).all()  # nothing behind the last block
        for b in range(blocks):
            top = np.abs(y[:, b * 128:(b + 1) * 128]).max(1)
            lo = np.array([R.scale_byte(t * (1 - 40 * U)) for t in top])
            hi = np.array([R.scale_byte(t * (1 + 40 * U)) for t in top])
            assert ((bytes_[:, b] == lo) | (bytes_[:, b] == hi)).all()
        scale = np.repeat(2.0 ** (bytes_.astype(float) - 127), 128, 1)[:, :d]
        got = R.q8_read(q.codes.cpu().numpy(), bytes_)
        assert (np.abs(got - y) <= np.maximum(np.abs(y) * 2.0 ** -4, scale * 2.0 ** -10) + 40 * U * np.abs(y)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_backward(d, dtype):
    import torch
    import nystr_self_attention_gb300 as N
    for rows, pad in ((1, 0), (9, 8), (5000 if d < 600 else 650, 16)):
        rng = np.random.default_rng(rows + d)
        s, gs, w = inputs(rows, d, dtype, rows + d)
        gy = R.rounded(rng.normal(size=(rows, d)), dtype)
        with_gs = rows != 9
        dx, dw = R.add_rms_norm_grad(s, gy, gs if with_gs else None, w, 1e-6)
        tdx, tdw = empty(rows, d, dtype, pad), torch.full((d,), 7.0, device="cuda")
        N.nystrom_add_rms_norm_bwd(upload(s, dtype, 2 * pad), upload(gy, dtype, pad),
                                   upload(gs, dtype, 3 * pad) if with_gs else None, torch.from_numpy(w).cuda(), tdx, tdw)
        done(N)
        r = 1 / np.sqrt((s * s).mean(-1, keepdims=True) + 1e-6)
        h, wg = r * s, np.abs(w * gy)
        M = (wg * np.abs(h)).mean(-1, keepdims=True)
        bound = 120 * U * r * (wg + np.abs(h) * M) + (np.abs(gs) * U if with_gs else 0) + HALF[dtype] * np.abs(dx)
        assert (np.abs(host(tdx) - dx) <= bound).all()
        assert (np.abs(host(tdw) - dw) <= (60 + rows / 100) * U * np.abs(gy * h).sum(0)).all()
        assert untouched(tdx, d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_in_place_and_repeated(dtype):
    import torch
    import nystr_self_attention_gb300 as N
    s, gs, w = inputs(900, 1544, dtype)
    gy = R.rounded(np.random.default_rng(4).normal(size=s.shape), dtype)
    tw = torch.from_numpy(w).cuda()
    want, wdw = empty(900, 1544, dtype), torch.empty(1544, device="cuda")
    N.nystrom_add_rms_norm_bwd(upload(s, dtype), upload(gy, dtype), upload(gs, dtype), tw, want, wdw)
    for over_gy in (True, False):
        a, b, dw = upload(gy, dtype), upload(gs, dtype), torch.empty(1544, device="cuda")
        N.nystrom_add_rms_norm_bwd(upload(s, dtype), a, b, tw, a if over_gy else b, dw)
        assert torch.equal(a if over_gy else b, want) and torch.equal(dw, wdw)  # the same bits
    nodw = empty(900, 1544, dtype)
    N.nystrom_add_rms_norm_bwd(upload(s, dtype), upload(gy, dtype), upload(gs, dtype), tw, nodw)
    done(N)
    assert torch.equal(nodw, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zero_huge_and_special_rows(dtype):
    import torch
    import nystr_self_attention_gb300 as N
    x = np.zeros((5, 256))
    x[1] = 1e-30
    x[2, 3] = np.inf
    x[3, 200] = np.nan
    x[4] = 1e15
    y, q = empty(5, 256, dtype), eight(N, 5, 256)
    tx = upload(x, dtype)
    N.nystrom_add_rms_norm_fwd(tx, None, None, None, y)
    N.nystrom_add_rms_norm_fwd(tx, None, None, None, q)
    done(N)
    got, bytes_ = host(y), R.q8_bytes(q.scales.cpu().numpy(), 256)
    assert (got[0] == 0).all() and (bytes_[0] == 0).all() and (q.codes[0].cpu().numpy() == 0).all()
    assert np.allclose(got[1], 1e-27, rtol=HALF[dtype] * 2 + 1e-6)
    assert np.isnan(got[2, 3]) and (got[2, :3] == 0).all()  # 0 / inf; inf / inf
    assert np.isnan(got[3]).all() and (bytes_[3] == 255).all()
    assert bytes_[2, 0] == 255 and bytes_[2, 1] == 0
    assert np.allclose(got[4], 1.0, rtol=HALF[dtype] * 2 + 1e-6)
    out = empty(5, 256, "f32")
    N.nystrom_q8_read(q, out)
    done(N)
    assert np.isnan(host(out)[3]).all() and (host(out)[0] == 0).all() and not np.isnan(host(out)[2, 128:]).any()


def test_refusals_in_python():
    import torch
    import nystr_self_attention_gb300 as N
    x, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    y = torch.empty_like(x)
    for bad in (dict(x=x.double()), dict(x=x.T), dict(x=x.cpu()), dict(x=x.view(2, 2, 64)), dict(y=y[:, :32]),
                dict(y=y.bfloat16()), dict(w=w[:32]), dict(w=w.bfloat16()), dict(r=x[:2])):
        a = dict(dict(x=x, r=None, w=w, s=None, y=y), **bad)
        with pytest.raises(ValueError):
            N.nystrom_add_rms_norm_fwd(a["x"], a["r"], a["w"], a["s"], a["y"])
    with pytest.raises(N.NystromError):
        N.nystrom_add_rms_norm_fwd(x, x, w, y, y)
    with pytest.raises(N.NystromError):
        N.nystrom_add_rms_norm_bwd(x, y, None, w, x)
