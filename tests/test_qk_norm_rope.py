"""GPU parity of the norm and rotation of queries and keys, and of its
gradients, against the fp64 oracle.

Bounds, per element, with u = 2^-24 (half a step of fp32) and hb = 2^-8 (of
bf16). Forward: the sum of d <= 128 squares is eight fused steps and up to four
shuffle steps (12u on the sum, 6u on its root), 2^-22 = 4u the reciprocal root,
2u the mean and eps, 2u the two products: 14u on a channel of z; the angle's
sine and cosine are off by 3u (fp32) or 2^-20 = 16u (bf16); two roundings for
the rotation: 19u or 32u of |z_a| + |z_b|, taken as 24u and 40u. Backward: g
carries 5u or 18u of |g_a| + |g_b|; h 12u; the mean of w g h sums d terms with
12u and the terms' own 20u (or 33u); the last three steps 3u: taken as 64u of
r (|w| (|g_a| + |g_b|) + |h| mean(|w g| h)). A weight's gradient sums R rows in
some order: (R + 32)u of the terms' magnitudes. A bf16 result is rounded once."""
import numpy as np
import pytest

from oracle import cache_ref as C

pytestmark = pytest.mark.gpu

U, HB = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def library():
    import torch
    from nystr_self_attention_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)


def heads(rng, B, H, n, d, dtype, order, scale=1.0):
    """A [B, H, n, d] view; "packed": one slice of a wider projection."""
    import torch
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    if order == "packed":
        x = torch.from_numpy(rng.standard_normal((B, n, H + 2, d)) * scale).to(td).cuda()
        return x[:, :, 1:H + 1].transpose(1, 2)
    shape = (B, n, H, d) if order == "bnhd" else (B, H, n, d)
    x = torch.from_numpy(rng.standard_normal(shape) * scale).to(td).cuda()
    return x.transpose(1, 2) if order == "bnhd" else x


def host(t):
    return t.detach().double().cpu().numpy()


def pair_sum(z, rot, pairs):
    """|z_a| + |z_b| in the place of both members of a rotated pair."""
    m = np.abs(z)
    out = m.copy()
    for a, b in C.rope_pairs(rot, pairs):
        out[..., a] = out[..., b] = m[..., a] + m[..., b]
    return out


def case(B=2, n=5, Hq=4, Hk=2, d=64, rot=None, sections=None, pairs=False, norm=True, dtype="bf16",
         order="bhnd", far=0, eps=1e-6, weights=True, positions=True, scale=1.0):
    rot = d if rot is None else rot
    return dict(B=B, n=n, Hq=Hq, Hk=Hk, d=d, rot=rot, sections=sections or [rot // 2], pairs=pairs,
                norm=norm, dtype=dtype, order=order, far=far, eps=eps, weights=weights,
                positions=positions, scale=scale)


CASES = {
    "plain": case(),
    "fp32": case(dtype="f32", order="bnhd", n=37),
    "one_token": case(B=1, n=1, Hq=1, Hk=1),
    "no_keys": case(Hk=0, n=9),
    "d128_packed": case(d=128, Hq=7, Hk=1, n=33, order="packed"),
    "d8": case(d=8, n=70, dtype="f32"),
    "d16_pairs": case(d=16, n=40, pairs=True, dtype="f32"),
    "d32_many_heads": case(d=32, Hq=33, Hk=11, n=3, order="bnhd"),
    "d72_odd_pairs": case(d=72, rot=36, n=17, dtype="f32"),
    "d72_full": case(d=72, n=17),
    "d96_pairs_part": case(d=96, rot=30, pairs=True, n=11),
    "d104_rot2": case(d=104, rot=2, n=3, order="packed"),
    "d120_rot24": case(d=120, rot=24, n=9, dtype="f32"),
    "not_rotated": case(rot=0, n=6),
    "half_rotated": case(d=128, rot=64, n=12),
    "axes3": case(d=128, sections=[16, 24, 24], n=50, order="bnhd"),
    "axes2_pairs": case(d=64, sections=[1, 31], pairs=True, dtype="f32", n=21),
    "axes4_an_empty_one": case(d=32, sections=[5, 0, 7, 4], n=13, dtype="f32"),
    "far": case(far=2 ** 31 - 100, dtype="f32", n=30, d=128),
    "negative": case(far=-(2 ** 31), dtype="f32", n=30),
    "rotation_alone": case(norm=False, n=31, dtype="f32"),
    "rotation_alone_bf16": case(norm=False, n=31, order="bnhd"),
    "no_weights": case(weights=False, n=8, dtype="f32"),
    "counted_positions": case(positions=False, n=300, B=3),
    "small_values": case(scale=1e-6, eps=1e-12, n=7, dtype="f32"),
    "many_tokens": case(B=3, n=700, Hq=2, Hk=2, d=64, dtype="f32", order="packed"),
    "many_rows_bf16": case(B=2, n=2049, Hq=3, Hk=1, d=32, order="bnhd"),
}


def setup(c, seed=5):
    import torch
    rng = np.random.default_rng(seed)
    q = heads(rng, c["B"], c["Hq"], c["n"], c["d"], c["dtype"], c["order"], c["scale"])
    k = heads(rng, c["B"], c["Hk"], c["n"], c["d"], c["dtype"], c["order"], c["scale"]) if c["Hk"] else None
    if c["positions"]:
        pos = rng.integers(0, 100, (len(c["sections"]), c["B"], c["n"])) + c["far"]
        dev = torch.from_numpy(pos.astype(np.int32)).cuda()
    else:
        pos, dev = np.tile(np.arange(c["n"]), (len(c["sections"]), c["B"], 1)), None
    inv = 10000.0 ** (-np.arange(c["rot"] // 2) * 2.0 / max(1, c["rot"]))
    w = [(1 + 0.3 * rng.standard_normal(c["d"])).astype(np.float32) for _ in range(2)]
    wd = [torch.from_numpy(x).cuda() if c["weights"] and c["norm"] else None for x in w]
    if not c["weights"]:
        w = [np.ones(c["d"], np.float32)] * 2
    return rng, q, k, pos, dev, inv, w, wd


def args_of(N, c):
    return dict(sections=c["sections"], pairing=N.NYS_ROPE_PAIRS if c["pairs"] else N.NYS_ROPE_HALVES,
                norm=c["norm"], eps=c["eps"])


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    import torch
    import nystr_self_attention_gb300 as N
    c = CASES[name]
    _, q, k, pos, dev, inv, w, wd = setup(c)
    outs = [torch.full_like(q, float("nan")), None if k is None else torch.full_like(k, float("nan"))]
    N.nystrom_qk_norm_rope_fwd(q, k, outs[0], outs[1], dev, inv, wd[0], wd[1], **args_of(N, c))
    torch.cuda.synchronize()
    ang = C.rope_angles(pos, inv, c["sections"])
    for x, y, wt in zip((q, k), outs, w):
        if x is None:
            continue
        z = C.norm_rows(host(x), wt.astype(np.float64), c["eps"]) if c["norm"] else host(x)
        want = C.rotate(z, ang, c["pairs"])
        tol = pair_sum(z, c["rot"], c["pairs"]) * (40 if c["dtype"] == "bf16" else 24) * U
        if c["dtype"] == "bf16":
            tol = tol * (1 + HB) + HB * np.abs(want)
        err = np.abs(host(y) - want)
        assert (err <= tol).all(), f"{name}: {(err / np.maximum(tol, 1e-300)).max():.2f} of the bound"


@pytest.mark.parametrize("name", CASES)
def test_backward(name):
    import torch
    import nystr_self_attention_gb300 as N
    c = CASES[name]
    rng, q, k, pos, dev, inv, w, wd = setup(c)
    gq = heads(rng, c["B"], c["Hq"], c["n"], c["d"], c["dtype"], "bhnd")
    gk = heads(rng, c["B"], c["Hk"], c["n"], c["d"], c["dtype"], c["order"]) if k is not None else None
    dq, dk = torch.full_like(q, float("nan")), None if k is None else torch.full_like(k, float("nan"))
    dw = [torch.full((c["d"],), float("nan"), device="cuda") if c["norm"] and x is not None else None
          for x in (q, k)]
    runs = []
    for _ in range(2):
        N.nystrom_qk_norm_rope_bwd(q, k, gq, gk, dq, dk, dev, inv, wd[0], wd[1], dw[0], dw[1], **args_of(N, c))
        torch.cuda.synchronize()
        runs.append([host(t) for t in (dq, dk, *dw) if t is not None])
    assert all(np.array_equal(a, b) for a, b in zip(*runs)), "two runs differ"
    ang = C.rope_angles(pos, inv, c["sections"])
    for x, gy, dx, wt, dwt in zip((q, k), (gq, gk), (dq, dk), w, dw):
        if x is None:
            continue
        wt = wt.astype(np.float64)
        want, wantw = C.qk_norm_rope_grad(host(x), wt, host(gy), ang, c["pairs"], c["norm"], c["eps"])
        gs = pair_sum(host(gy), c["rot"], c["pairs"])
        if c["norm"]:
            xs = host(x)
            r = 1 / np.sqrt((xs * xs).mean(-1, keepdims=True) + c["eps"])
            h = np.abs(xs * r)
            tol = 64 * U * r * (np.abs(wt) * gs + h * (np.abs(wt) * gs * h).mean(-1, keepdims=True))
        else:
            tol = (40 if c["dtype"] == "bf16" else 24) * U * gs
        if c["dtype"] == "bf16":
            tol = tol * (1 + HB) + HB * np.abs(want)
        err = np.abs(host(dx) - want)
        assert (err <= tol).all(), f"{name}: dx at {(err / np.maximum(tol, 1e-300)).max():.2f} of the bound"
        if dwt is not None:
            rows = x.numel() / c["d"]
            tolw = (rows + 32) * U * (gs * h).sum(axis=(0, 1, 2))
            errw = np.abs(host(dwt) - wantw)
            assert (errw <= tolw).all(), f"{name}: dw at {(errw / tolw).max():.2f} of the bound"


def test_backward_agrees_with_differences_of_the_forward():
    """fp32 forward differences along a random direction against <dx, v> + <dw, u>:
    a step of 2^-6 leaves a second-order error of about 2^-12 of the third
    derivatives, the forward's rounding 24u sqrt(terms) / 2^-6."""
    import torch
    import nystr_self_attention_gb300 as N
    c = case(d=64, n=6, dtype="f32", sections=[10, 10, 12])
    rng, q, k, pos, dev, inv, w, wd = setup(c)
    gq, gk = heads(rng, 2, 4, 6, 64, "f32", "bhnd"), heads(rng, 2, 2, 6, 64, "f32", "bhnd")
    dq, dk, dqw, dkw = (torch.empty_like(t) for t in (q, k, *wd))
    N.nystrom_qk_norm_rope_bwd(q, k, gq, gk, dq, dk, dev, inv, wd[0], wd[1], dqw, dkw, **args_of(N, c))
    vq, vk = torch.randn_like(q), torch.randn_like(k)
    uq, uk = torch.randn_like(wd[0]), torch.randn_like(wd[1])
    h = 2.0 ** -6

    def loss(s):
        a, b = torch.empty_like(q), torch.empty_like(k)
        N.nystrom_qk_norm_rope_fwd(q + s * vq, k + s * vk, a, b, dev, inv, wd[0] + s * uq, wd[1] + s * uk,
                                   **args_of(N, c))
        return ((a.double() * gq.double()).sum() + (b.double() * gk.double()).sum()).item()

    slope = (8 * (loss(h) - loss(-h)) - (loss(2 * h) - loss(-2 * h))) / (12 * h)  # fourth order
    want = sum((a.double() * b.double()).sum().item() for a, b in
               ((dq, vq), (dk, vk), (dqw, uq), (dkw, uk)))
    size = sum((a.double() * b.double()).norm().item() for a, b in
               ((dq, vq), (dk, vk), (dqw, uq), (dkw, uk)))
    assert abs(slope - want) <= 1e-3 * size


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(dtype):
    import torch
    import nystr_self_attention_gb300 as N
    for c in (case(n=19, dtype=dtype), case(n=19, dtype=dtype, norm=False, rot=36, d=72, order="packed"),
              case(n=300, dtype=dtype, pairs=True, Hq=9, Hk=9)):
        rng, q, k, pos, dev, inv, w, wd = setup(c)
        gq, gk = (heads(rng, c["B"], H, c["n"], c["d"], dtype, "bhnd") for H in (c["Hq"], c["Hk"]))
        a, b = torch.empty_like(q), torch.empty_like(k)
        N.nystrom_qk_norm_rope_bwd(q, k, gq, gk, a, b, dev, inv, wd[0], wd[1], **args_of(N, c))
        N.nystrom_qk_norm_rope_bwd(q, k, gq, gk, gq, gk, dev, inv, wd[0], wd[1], **args_of(N, c))
        assert torch.equal(gq, a) and torch.equal(gk, b)
        N.nystrom_qk_norm_rope_fwd(q, k, a, b, dev, inv, wd[0], wd[1], **args_of(N, c))
        N.nystrom_qk_norm_rope_fwd(q, k, q, k, dev, inv, wd[0], wd[1], **args_of(N, c))
        assert torch.equal(q, a) and torch.equal(k, b)


def test_only_the_rows_are_written():
    """Outputs inside a wider buffer: what lies between the rows stays."""
    import torch
    import nystr_self_attention_gb300 as N
    rng = np.random.default_rng(3)
    q = heads(rng, 2, 3, 21, 64, "bf16", "bhnd")
    wide = torch.full((2, 21, 5, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :, 1:4, 16:80].transpose(1, 2)
    N.nystrom_qk_norm_rope_fwd(q, None, out, None, None, [0.1] * 32)
    keep = wide.clone()
    keep[:, :, 1:4, 16:80] = 7.0
    assert (keep == 7.0).all() and not (out == 7.0).all()


def test_zero_rows_and_broadcast_inputs():
    import torch
    import nystr_self_attention_gb300 as N
    x = torch.randn(1, 1, 4, 64, device="cuda")
    x[:, :, 1] = 0
    q = x.expand(3, 5, 4, 64)  # strides of zero
    out = torch.empty(3, 5, 4, 64, device="cuda")
    N.nystrom_qk_norm_rope_fwd(q, None, out, None, None, [0.1] * 32)
    want = C.rotate(C.norm_rows(host(x), 1.0, 1e-6), C.rope_angles(np.arange(4)[None, None], [0.1] * 32, [32]), False)
    assert np.abs(host(out) - want).max() <= 48 * U * np.abs(want).max() and (out[:, :, 1] == 0).all()


def test_other_stream_and_graph_replay():
    """Captured with its own workspace, replayed on new contents; an eager
    call on another stream meanwhile."""
    import torch
    import nystr_self_attention_gb300 as N
    c = case(n=40, dtype="f32")
    rng, q, k, pos, dev, inv, w, wd = setup(c)
    gq, gk = heads(rng, 2, 4, 40, 64, "f32", "bhnd"), heads(rng, 2, 2, 40, 64, "f32", "bhnd")
    dq, dk, dqw, dkw = (torch.empty_like(t) for t in (q, k, *wd))
    a, b = torch.empty_like(q), torch.empty_like(k)

    def both():
        N.nystrom_qk_norm_rope_fwd(q, k, a, b, dev, inv, wd[0], wd[1], **args_of(N, c))
        N.nystrom_qk_norm_rope_bwd(q, k, gq, gk, dq, dk, dev, inv, wd[0], wd[1], dqw, dkw, **args_of(N, c))

    both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    q.copy_(torch.randn_like(q))
    for t in (a, b, dq, dk, dqw, dkw):
        t.fill_(float("nan"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g.replay()
    e = [torch.empty_like(t) for t in (dq, dk, dqw, dkw)]
    N.nystrom_qk_norm_rope_bwd(q, k, gq, gk, e[0], e[1], dev, inv, wd[0], wd[1], e[2], e[3], **args_of(N, c),
                               stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((dq, dk, dqw, dkw), e))


def test_cached_workspace_is_refused_under_capture():
    import ctypes
    import torch
    import nystr_self_attention_gb300 as N
    lib = N.load_library()
    q = torch.randn(1, 2, 4, 64, device="cuda")
    dq, dw = torch.empty_like(q), torch.empty(64, device="cuda")
    s = N.NysStrides(0, 256, 64)
    a = N.NysQkRope(1, 4, 2, 0, 64, 64, 1, (ctypes.c_int * 4)(32), 0, 1, N.NYS_FP32, 1e-6, s, s, s, s, s, s)
    f = (ctypes.c_double * 32)(*[0.1] * 32)

    def call(stream):
        return lib.nystrom_qk_norm_rope_bwd(ctypes.byref(a), q.data_ptr(), None, q.data_ptr(), None, None, None,
                                            None, ctypes.cast(f, ctypes.c_void_p), dq.data_ptr(), None,
                                            dw.data_ptr(), None, None, 0, stream)

    assert call(torch.cuda.current_stream().cuda_stream) == N.NYS_OK
    torch.cuda.synchronize()
    first = dw.clone()
    g, codes = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(g):
        codes.append(call(torch.cuda.current_stream().cuda_stream))
        dq.zero_()
    assert codes == [N.NYS_ERR_ARG]
    assert torch.equal(first, dw)
