"""Refusals of the operators around the attention module: bad arguments give
the documented codes before anything touches CUDA. No kernel runs here."""
import ctypes

import pytest

E_ARG, E_SHAPE, E_ALIGN, E_NOMEM = -1, -2, -3, -5
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def N():
    from nystr_self_attention_gb300 import build
    build.build()
    import nystr_self_attention_gb300 as pkg
    pkg.load_library()
    return pkg


def q8(N, codes=256, scales=512, rows=4, K=256, stride=None):
    return ctypes.byref(N.NysQ8(codes, scales, rows, K, K if stride is None else stride))


BAD_Q8 = [
    (dict(codes=None), E_ARG), (dict(scales=None), E_ARG), (dict(rows=0), E_SHAPE), (dict(K=0), E_SHAPE),
    (dict(K=264), E_SHAPE), (dict(K=(1 << 20) + 16), E_SHAPE), (dict(rows=2 ** 31 - 1), E_SHAPE),
    (dict(stride=-16), E_ARG), (dict(stride=264), E_ALIGN), (dict(codes=264), E_ALIGN), (dict(scales=514), E_ALIGN),
    (dict(codes=512), E_ARG),
]


@pytest.mark.parametrize("kw,code", BAD_Q8)
def test_q8_matrices_refused_everywhere(N, kw, code):
    lib = N.load_library()
    rows, K = kw.get("rows", 4), kw.get("K", 256)
    assert lib.nystrom_q8_write(q8(N, **kw), 1024, max(K, 8), 1, 1, 1, None) == code
    assert lib.nystrom_q8_read(q8(N, **kw), 1024, max(K, 8), 1, None) == code
    good = q8(N, 2048, 4096, K=K if K > 0 else 256)
    assert lib.nystrom_q8_matmul(q8(N, **kw), good, 1024, 8, 1, None, 0, None) == code
    assert lib.nystrom_q8_matmul(good, q8(N, **kw), 1024, 1 << 20, 1, None, 0, None) == code
    if "rows" in kw or "K" in kw:
        assert N.nystrom_q8_scales_bytes(rows, K) == 0


def test_q8_write_and_read_refusals(N):
    lib = N.load_library()

    def write(x=1024, rs=256, cs=1, block=1, dtype=1, **kw):
        return lib.nystrom_q8_write(q8(N, **kw), x, rs, cs, block, dtype, None)
    assert write(x=None) == E_ARG
    assert write(dtype=2) == E_ARG
    assert write(block=64) == E_ARG
    assert write(rs=2, cs=2) == E_ARG
    assert write(rs=-256) == E_ARG
    assert write(rs=260) == E_ALIGN
    assert write(x=1032) == E_ALIGN
    assert write(x=256) == E_ARG and write(x=512) == E_ARG   # its own codes, its own scales
    assert write(rs=1, cs=8, rows=4) == E_SHAPE              # turned: rows in eights
    assert write(rs=1, cs=12, rows=8) == E_ALIGN
    assert write(stride=128, rows=2) == E_ARG                # rows of codes on top of each other

    def read(out=1024, stride=256, dtype=1, **kw):
        return lib.nystrom_q8_read(q8(N, **kw), out, stride, dtype, None)
    assert read(out=None) == E_ARG and read(dtype=7) == E_ARG
    assert read(stride=128) == E_ARG and read(stride=258) == E_ALIGN and read(out=1028) == E_ALIGN
    assert read(out=256) == E_ARG and read(out=512) == E_ARG


def test_q8_matmul_refusals(N):
    lib = N.load_library()

    def mm(out=8192, stride=64, dtype=1, ws=None, nbytes=0, Kw=256, n=64, T=4, c=1024):
        return lib.nystrom_q8_matmul(q8(N, c, 1536, T, 256), q8(N, 2048, 4096, n, Kw), out, stride, dtype, ws, nbytes,
                                     None)
    assert mm(Kw=272) == E_SHAPE
    assert mm(n=60) == E_SHAPE
    assert mm(out=None) == E_ARG and mm(dtype=2) == E_ARG
    assert mm(stride=32) == E_ARG and mm(stride=68) == E_ALIGN and mm(out=8200) == E_ALIGN
    assert mm(out=1024) == E_ARG and mm(out=4096) == E_ARG
    assert mm(ws=128, nbytes=1 << 30) == E_ALIGN
    assert mm(ws=256, nbytes=8) == E_NOMEM
    assert N.nystrom_q8_matmul_workspace_bytes(4, 64, 256, 1) > 0
    assert N.nystrom_q8_matmul_workspace_bytes(4, 64, 256, 1) % 256 == 0
    for bad in ((0, 64, 256, 1), (4, 60, 256, 1), (4, 64, 264, 1), (4, 64, 256, 2), (2 ** 31, 64, 256, 1),
                (2 ** 31 - 2000, 1 << 20, 256, 1)):
        assert N.nystrom_q8_matmul_workspace_bytes(*bad) == 0


def norm(N, **kw):
    a = dict(dict(rows=4, d=64, dtype=1, eps=1e-6, x=64, residual=64, sum=64, y=64, gs=64, dx=64), **kw)
    return ctypes.byref(N.NysAddRmsNorm(*[a[k] for k in
                                          ("rows", "d", "dtype", "eps", "x", "residual", "sum", "y", "gs", "dx")]))


BAD_NORM = [
    (dict(dtype=2), E_ARG), (dict(eps=-1.0), E_ARG), (dict(eps=NAN), E_ARG), (dict(eps=INF), E_ARG),
    (dict(rows=0), E_SHAPE), (dict(d=0), E_SHAPE), (dict(d=60), E_SHAPE), (dict(d=16392), E_SHAPE),
    (dict(sum=-64), E_ARG), (dict(y=32), E_ARG), (dict(sum=68), E_ALIGN),
]


@pytest.mark.parametrize("kw,code", BAD_NORM)
def test_norm_refusals(N, kw, code):
    lib = N.load_library()
    if kw != dict(y=32):  # an input of the backward pass: its rows may overlap
        assert lib.nystrom_add_rms_norm_bwd(norm(N, **kw), 256, 512, 1024, 16, 2048, None, None, 0, None) == code
    assert lib.nystrom_add_rms_norm_fwd(norm(N, **kw), 256, 512, 16, 1024, 2048, None, None) == code


def test_norm_pointers(N):
    lib = N.load_library()

    def fwd(x=256, r=512, w=16, s=1024, y=2048, y8=None, **kw):
        return lib.nystrom_add_rms_norm_fwd(norm(N, **kw), x, r, w, s, y, y8, None)
    assert fwd(x=None) == E_ARG and fwd(y=None) == E_ARG
    assert fwd(y8=q8(N, 4096, 8192, 4, 64)) == E_ARG       # both outputs
    assert fwd(y=None, y8=q8(N, 4096, 8192, 4, 48)) == E_SHAPE
    assert fwd(y=None, y8=q8(N, 256, 8192, 4, 64)) == E_ARG   # codes over x
    assert fwd(r=None) == E_ARG                            # a sum without a residual
    assert fwd(s=2048) == E_ARG                            # sum and y at one address
    assert fwd(s=16) == E_ARG and fwd(y=16) == E_ARG       # over the weight
    assert fwd(s=256, sum=128) == E_ARG                    # in place with another stride
    assert fwd(x=264) == E_ALIGN and fwd(w=18) == E_ALIGN

    def bwd(s=256, gy=512, gs=1024, w=16, dx=2048, dw=None, ws=None, nbytes=0, **kw):
        return lib.nystrom_add_rms_norm_bwd(norm(N, **kw), s, gy, gs, w, dx, dw, ws, nbytes, None)
    assert bwd(s=None) == E_ARG and bwd(gy=None) == E_ARG and bwd(dx=None) == E_ARG
    assert bwd(dx=256) == E_ARG                            # the sum is read again
    assert bwd(dw=16) == E_ARG and bwd(dw=18) == E_ALIGN
    assert bwd(dw=64, ws=128, nbytes=1 << 30) == E_ALIGN and bwd(dw=64, ws=256, nbytes=8) == E_NOMEM
    assert N.nystrom_add_rms_norm_workspace_bytes(N.NysAddRmsNorm(4, 64, 1, 1e-6)) % 256 == 0
    assert N.nystrom_add_rms_norm_workspace_bytes(N.NysAddRmsNorm(4, 64, 1, 1e-6)) > 0
    assert N.nystrom_add_rms_norm_workspace_bytes(N.NysAddRmsNorm(4, 60, 1, 1e-6)) == 0


def ff(N, **kw):
    a = dict(dict(T=4, d=64, f=128, act=0, layout=0, dtype=1, x=64, w=128, h=128, gate=128, up=128, dx=64, dw=128), **kw)
    return N.NysGatedFf(*[a[k] for k in ("T", "d", "f", "act", "layout", "dtype", "x", "w", "h", "gate", "up", "dx", "dw")])


BAD_FF = [
    (dict(dtype=2), E_ARG), (dict(act=4), E_ARG), (dict(act=-1), E_ARG), (dict(layout=2), E_ARG),
    (dict(T=0), E_SHAPE), (dict(d=4), E_SHAPE), (dict(f=12), E_SHAPE), (dict(d=(1 << 20) + 8), E_SHAPE),
    (dict(T=(1 << 30) + 1), E_SHAPE), (dict(T=1 << 30, d=1 << 20, f=1 << 20), E_SHAPE),
    (dict(x=-64), E_ARG), (dict(w=68), E_ALIGN), (dict(h=132), E_ALIGN),
]


@pytest.mark.parametrize("kw,code", BAD_FF)
def test_ff_refusals(N, kw, code):
    lib = N.load_library()
    p = ff(N, **kw)
    a = [256 * i for i in range(1, 10)]
    assert lib.nystrom_gated_ff_fwd(ctypes.byref(p), *a[:6], None, 0, None) == code
    assert lib.nystrom_gated_ff_bwd(ctypes.byref(p), *a[:9], None, 0, None) == code
    if code == E_SHAPE:
        assert N.nystrom_gated_ff_workspace_bytes(p, 0) == 0 and N.nystrom_gated_ff_workspace_bytes(p, 1) == 0


def test_ff_pointers(N):
    lib = N.load_library()

    def fwd(x=256, wg=512, wu=768, h=1024, g=1280, u=1536, ws=None, nbytes=0, **kw):
        return lib.nystrom_gated_ff_fwd(ctypes.byref(ff(N, **kw)), x, wg, wu, h, g, u, ws, nbytes, None)
    for k in ("x", "wg", "wu", "h", "g", "u"):
        assert fwd(**{k: None}) == E_ARG
    for k in ("x", "wg", "wu", "h", "g", "u"):
        assert fwd(**{k: 264}) == E_ALIGN
    assert fwd(h=256) == E_ARG and fwd(g=1024) == E_ARG and fwd(u=1280) == E_ARG and fwd(u=512) == E_ARG
    assert fwd(ws=128, nbytes=1 << 40) == E_ALIGN and fwd(ws=256, nbytes=8) == E_NOMEM

    def bwd(x=256, wg=512, wu=768, g=1024, u=1280, gh=1536, dx=1792, dg=2048, du=2304, ws=None, nbytes=0, **kw):
        return lib.nystrom_gated_ff_bwd(ctypes.byref(ff(N, **kw)), x, wg, wu, g, u, gh, dx, dg, du, ws, nbytes, None)
    for k in ("x", "wg", "wu", "g", "u", "gh", "dg", "du"):
        assert bwd(**{k: None}) == E_ARG
    assert bwd(dx=None, dg=None, du=None) == E_ARG
    for k in ("x", "wg", "wu", "g", "u", "gh", "dx", "dg", "du"):
        assert bwd(**{k: 264}) == E_ALIGN
    assert bwd(dx=1536) == E_ARG and bwd(dg=512) == E_ARG and bwd(du=2048) == E_ARG and bwd(dx=256) == E_ARG
    assert bwd(ws=128, nbytes=1 << 40) == E_ALIGN and bwd(ws=256, nbytes=8) == E_NOMEM
    for back in (False, True):
        assert N.nystrom_gated_ff_workspace_bytes(ff(N), back) % 256 == 0
    assert N.nystrom_gated_ff_workspace_bytes(ff(N), True) > 0
    assert N.load_library().nystrom_gated_ff_workspace_bytes(ctypes.byref(ff(N)), 2) == 0


def test_factors_rows_do_not_overlap(N):
    lib = N.load_library()
    over = [dict(a=0), dict(a=128), dict(w=0), dict(w=240)]  # bytes between rows of 256

    def mm(a=256, w=256, T=4, n=64):
        return lib.nystrom_q8_matmul(q8(N, 1024, 1536, T, 256, stride=a), q8(N, 2048, 4096, n, 256, stride=w), 8192, 64,
                                     1, None, 0, None)
    for kw in over:
        assert mm(**kw) == E_ARG
    for T in (4, 400):
        for kw in (dict(x=0), dict(x=32), dict(w=0), dict(w=64)):
            for dtype in (0, 1):
                for layout in (0, 1):
                    p = ff(N, T=T, dtype=dtype, layout=layout, **{**dict(w=128, dw=128), **kw})
                    a = [256 * i for i in range(1, 10)]
                    if layout == 1 and kw == dict(w=64):
                        continue  # rows of 64: side by side
                    assert lib.nystrom_gated_ff_fwd(ctypes.byref(p), *a[:6], None, 0, None) == E_ARG
                    assert lib.nystrom_gated_ff_bwd(ctypes.byref(p), *a, None, 0, None) == E_ARG


def test_the_stride_of_a_single_row_does_not_matter(N):
    """Any stride is taken: what is refused is the workspace."""
    lib = N.load_library()
    for stride in (-16, -5, 3, 0):
        one = dict(x=stride, h=stride, gate=stride, up=stride, dx=stride)
        a = [256 * i for i in range(1, 10)]
        for ws, nbytes, code in ((128, 1 << 30, E_ALIGN), (256, 8, E_NOMEM)):
            assert lib.nystrom_q8_matmul(q8(N, 1024, 1536, 1, 256, stride=stride), q8(N, 2048, 4096, 64, 256), 8192,
                                         stride, 1, ws, nbytes, None) == code
            p = norm(N, rows=1, **{k: stride for k in ("x", "residual", "sum", "y", "gs", "dx")})
            assert lib.nystrom_add_rms_norm_bwd(p, 256, 512, 1024, 16, 2048, 64, ws, nbytes, None) == code
            for dtype in (0, 1):
                f = ctypes.byref(ff(N, T=1, dtype=dtype, **one))
                assert lib.nystrom_gated_ff_fwd(f, *a[:6], ws, nbytes, None) == code
                assert lib.nystrom_gated_ff_bwd(f, *a, ws, nbytes, None) == code
