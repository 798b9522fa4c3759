"""Refusals of the operators around a cached attention layer: bad arguments
give the documented codes before anything touches CUDA. No kernel runs here."""
import ctypes

import pytest

E_ARG, E_SHAPE, E_ALIGN, E_NOMEM = -1, -2, -3, -5


@pytest.fixture(scope="module")
def N():
    from nystr_self_attention_gb300 import build
    build.build()
    import nystr_self_attention_gb300 as pkg
    pkg.load_library()
    return pkg


def strides(N, H, n, d):
    return N.NysStrides(H * n * d, n * d, d)


def rope(N, back=False, q=256, k=256, qo=256, ko=256, freq=True, qw=256, pos=256, dqw=None, ws=None,
         nbytes=0, sections=(32,), inv=None, st=None, **kw):
    a = dict(dict(B=2, n=8, Hq=4, Hk=2, d=64, rot=64, axes=1, pairing=0, norm=1, dtype=1, eps=1e-6), **kw)
    s = st or strides(N, a["Hq"], a["n"], a["d"])
    desc = N.NysQkRope(a["B"], a["n"], a["Hq"], a["Hk"], a["d"], a["rot"], a["axes"],
                       (ctypes.c_int * 4)(*sections), a["pairing"], a["norm"], a["dtype"], a["eps"],
                       s, s, s, s, s, s)
    f = (ctypes.c_double * 64)(*(inv or [0.5] * 64))
    lib = N.load_library()
    fp = ctypes.cast(f, ctypes.c_void_p) if freq else None
    if back:
        return lib.nystrom_qk_norm_rope_bwd(ctypes.byref(desc), q, k, qo, ko, qw, 256, pos, fp, 256, 256,
                                            dqw, None, ws, nbytes, None)
    return lib.nystrom_qk_norm_rope_fwd(ctypes.byref(desc), q, k, qw, 256, pos, fp, qo, ko, None)


BAD_ROPE = [
    (dict(q=None), E_ARG), (dict(k=None), E_ARG), (dict(qo=None), E_ARG), (dict(freq=False), E_ARG),
    (dict(dtype=2), E_ARG), (dict(pairing=2), E_ARG), (dict(norm=2), E_ARG), (dict(eps=-1.0), E_ARG),
    (dict(eps=float("nan")), E_ARG), (dict(inv=[float("inf")] + [0.1] * 63), E_ARG),
    (dict(B=0), E_SHAPE), (dict(n=0), E_SHAPE), (dict(Hq=0), E_SHAPE), (dict(Hk=-1), E_SHAPE),
    (dict(d=60), E_SHAPE), (dict(d=136), E_SHAPE), (dict(rot=63), E_SHAPE), (dict(rot=66), E_SHAPE),
    (dict(rot=-2), E_SHAPE), (dict(axes=0), E_SHAPE), (dict(axes=5), E_SHAPE),
    (dict(sections=(31,)), E_SHAPE), (dict(axes=2, sections=(33, -1)), E_SHAPE),
    (dict(B=65536, n=32768), E_SHAPE), (dict(Hq=65536), E_SHAPE),
    (dict(q=264), E_ALIGN), (dict(qo=264), E_ALIGN), (dict(k=264), E_ALIGN), (dict(qw=258), E_ALIGN),
    (dict(pos=258), E_ALIGN),
]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,code", BAD_ROPE)
def test_rope_refusals(N, kw, code, back):
    assert rope(N, back, **kw) == code


@pytest.mark.parametrize("back", [False, True])
def test_rope_refuses_strides(N, back):
    assert rope(N, back, st=N.NysStrides(2048, 512, -64)) == E_ARG
    assert rope(N, back, st=N.NysStrides(2048, 512, 68)) == E_ALIGN
    assert rope(N, back, st=N.NysStrides(2048, 512, 0)) == E_ARG  # output rows on top of each other


def test_rope_backward_workspace_and_weights(N):
    assert rope(N, True, dqw=256, ws=128, nbytes=1 << 20) == E_ALIGN
    assert rope(N, True, dqw=256, ws=256, nbytes=8) == E_NOMEM
    assert rope(N, True, dqw=256, norm=0) == E_ARG
    desc = N.NysQkRope(2, 8, 4, 2, 64, 64, 1, (ctypes.c_int * 4)(32), 0, 1, 1, 1e-6)
    assert N.nystrom_qk_norm_rope_workspace_bytes(desc) % 256 == 0
    assert N.nystrom_qk_norm_rope_workspace_bytes(desc) > 0
    desc.norm = 0
    assert N.nystrom_qk_norm_rope_workspace_bytes(desc) == 0


def cache(N, **kw):
    a = dict(dict(data=256, table=256, pages=8, max_pages=4, page=32, Hk=2, d=64), **kw)
    return N.NysKv4Cache(a["data"], a["table"], a["pages"], a["max_pages"], a["page"], a["Hk"], a["d"])


BAD_CACHE = [
    (dict(data=None), E_ARG), (dict(table=None), E_ARG), (dict(pages=0), E_SHAPE),
    (dict(max_pages=0), E_SHAPE), (dict(page=8), E_SHAPE), (dict(page=24), E_SHAPE),
    (dict(page=8192), E_SHAPE), (dict(Hk=0), E_SHAPE), (dict(d=48), E_SHAPE), (dict(d=256), E_SHAPE),
    (dict(max_pages=1 << 27), E_SHAPE), (dict(data=264), E_ALIGN), (dict(table=258), E_ALIGN),
]


def io(N, read, c, k=256, v=256, st=None, starts=None, counts=None, B=2, n=8, dtype=1):
    s = st or strides(N, 2, n, 64)
    lib = N.load_library()
    f = lib.nystrom_kv4_read if read else lib.nystrom_kv4_write
    return f(ctypes.byref(c), k, v, ctypes.byref(s), ctypes.byref(s), starts, counts, B, n, dtype, None)


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_cache_refusals(N, kw, code, read):
    assert io(N, read, cache(N, **kw)) == code


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(k=None), E_ARG), (dict(v=None), E_ARG), (dict(dtype=3), E_ARG), (dict(B=0), E_SHAPE),
    (dict(B=65536), E_SHAPE), (dict(n=0), E_SHAPE), (dict(k=264), E_ALIGN), (dict(v=248), E_ALIGN),
    (dict(starts=258), E_ALIGN), (dict(counts=257), E_ALIGN)])
def test_io_refusals(N, kw, code, read):
    assert io(N, read, cache(N), **kw) == code


def test_io_refuses_strides(N):
    assert io(N, False, cache(N), st=N.NysStrides(-8, 512, 64)) == E_ARG
    assert io(N, False, cache(N), st=N.NysStrides(1024, 512, 60)) == E_ALIGN
    assert io(N, True, cache(N), st=N.NysStrides(1024, 0, 64)) == E_ARG


def test_cache_bytes(N):
    assert N.nystrom_kv4_cache_bytes(3, 64, 8, 128) == 3 * 64 * 8 * 2 * (128 // 2 + 128 // 32 * 2)
    assert N.nystrom_kv4_cache_bytes(1, 16, 1, 32) == 576
    assert N.nystrom_kv4_cache_bytes(1, 16, 1, 96) == 0


def attn(N, c=None, q=256, out=256, st=None, lengths=256, counts=None, B=2, nq=3, Hq=4, max_length=100,
         causal=1, scale=0.0, dtype=1, ws=None, nbytes=0):
    s = st or strides(N, Hq, nq, 64)
    return N.load_library().nystrom_kv4_attn_fwd(
        ctypes.byref(c or cache(N)), q, out, ctypes.byref(s), ctypes.byref(s), lengths, counts, B, nq, Hq,
        max_length, causal, scale, dtype, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), E_ARG), (dict(out=None), E_ARG), (dict(lengths=None), E_ARG), (dict(causal=2), E_ARG),
    (dict(scale=float("inf")), E_ARG), (dict(scale=float("nan")), E_ARG), (dict(dtype=7), E_ARG),
    (dict(B=0), E_SHAPE), (dict(nq=0), E_SHAPE), (dict(Hq=3), E_SHAPE), (dict(Hq=0), E_SHAPE),
    (dict(max_length=-1), E_SHAPE), (dict(nq=1 << 29, Hq=4), E_SHAPE), (dict(q=264), E_ALIGN),
    (dict(out=264), E_ALIGN), (dict(lengths=258), E_ALIGN), (dict(counts=258), E_ALIGN),
    (dict(ws=128, nbytes=1 << 30), E_ALIGN)])
def test_attention_refusals(N, kw, code):
    assert attn(N, **kw) == code


@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_attention_refuses_caches(N, kw, code):
    assert attn(N, cache(N, **kw)) == code


def test_attention_refuses_strides_and_small_workspaces(N):
    assert attn(N, st=N.NysStrides(768, 192, -64)) == E_ARG
    assert attn(N, st=N.NysStrides(768, 192, 0)) == E_ARG
    assert attn(N, st=N.NysStrides(768, 192, 66)) == E_ALIGN
    c = cache(N, max_pages=4096, page=32, pages=8192)
    need = N.load_library().nystrom_kv4_attn_workspace_bytes(ctypes.byref(c), 1, 1, 4, 100000, 1)
    if need:
        assert attn(N, c, B=1, nq=1, max_length=100000, ws=256, nbytes=need - 1) == E_NOMEM
        assert need % 256 == 0
    assert N.load_library().nystrom_kv4_attn_workspace_bytes(ctypes.byref(cache(N, d=48)), 1, 1, 4, 8, 1) == 0


def test_new_status_code_has_a_text(N):
    assert "range" in N.nystrom_strerror(N.NYS_ERR_INDEX)


def test_binding_refuses_tensors_that_do_not_fit(N):
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 2, 4, 64)
    with pytest.raises(ValueError):
        N.nystrom_qk_norm_rope_fwd(q, q, q, q, None, [0.5] * 32)
    with pytest.raises(ValueError):
        N.NystromKv4Cache(torch.zeros(1 << 16, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.int32), 32, 2, 64)
    with pytest.raises(N.NystromError):
        N.NystromKv4Cache(torch.zeros(1 << 16, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.int32), 24, 2, 64)


def test_well_formed_calls_need_the_gpu(N):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("checks the behaviour without a GPU")
    assert rope(N) == N.NYS_ERR_UNSUPPORTED
    assert rope(N, True, dqw=256) == N.NYS_ERR_UNSUPPORTED
    assert io(N, False, cache(N)) == N.NYS_ERR_UNSUPPORTED
    assert attn(N) == N.NYS_ERR_UNSUPPORTED


def test_packed_descriptors_are_the_structures(N):
    """The binding packs them by hand: the same bytes as the C layouts."""
    from nystr_self_attention_gb300 import _binding as b
    s = [N.NysStrides(100 + 3 * i, 101 + 3 * i, 102 + 3 * i) for i in range(6)]
    rope = N.NysQkRope(1, 2, 3, 4, 5, 6, 7, (ctypes.c_int * 4)(8, 9, 10, 11), 12, 13, 14, 0.5, *s)
    packed = b._ROPE_DESC.pack(1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 0.5, *range(100, 118))
    assert bytes(rope) == packed
    cache = b.NysKv4Cache(256, 512, 1, 2, 3, 4, 5)
    assert bytes(cache) == b._KV4_DESC.pack(256, 512, 1, 2, 3, 4, 5)
    assert bytes(s[0]) == b._STRIDES.pack(100, 101, 102)


@pytest.mark.parametrize("max_pages,page,code", [(524272, 4096, None), (524273, 4096, E_SHAPE),
                                                 (134213632, 16, None), (134213633, 16, E_SHAPE)])
def test_positions_stay_clear_of_32_bits(N, max_pages, page, code):
    """max_pages * page_size up to 2^31 - 2^16: key indexes of a tile past the
    last one still fit."""
    c = cache(N, max_pages=max_pages, page=page)
    got = io(N, False, c, k=264)  # past the shape check only the alignment is wrong
    assert got == (E_ALIGN if code is None else code)


def test_pools_past_any_memory_are_refused(N):
    big = 2 ** 31 - 1
    assert N.nystrom_kv4_cache_bytes(big, 4096, 65535, 128) == 0
    assert io(N, False, cache(N, pages=big, Hk=65535, page=4096)) == E_SHAPE
    pages = 2 ** 47 // (65535 * 256 * 18 * 128)
    assert N.nystrom_kv4_cache_bytes(pages, 4096, 65535, 128) == pages * 65535 * 256 * 18 * 128
    assert N.nystrom_kv4_cache_bytes(pages + 1, 4096, 65535, 128) == 0
