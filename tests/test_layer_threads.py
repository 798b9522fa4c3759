"""Calls of different sizes from two host threads at once, and of one thread on two
streams without workspaces."""
import ctypes
import threading

import pytest

from layer_helpers import done, own_status, tdtype

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


def at_once(calls, times):
    """Codes other than 0 of `times` calls of each, each in a thread of its own."""
    start, bad = threading.Barrier(len(calls)), []

    def work(call):
        start.wait()
        for _ in range(times):
            code = call()
            if code:
                bad.append(code)
    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return bad


def norm_back(rows, d, dtype, with_gs, stream):
    """(call, outputs) on `stream`, with a workspace of its own."""
    import torch
    import nystr_self_attention_gb300 as N
    lib, code = N.load_library(), N.NYS_BF16 if dtype == "bf16" else N.NYS_FP32
    s, gy, gs = (torch.randn(rows, d, device="cuda").to(tdtype(dtype)) for _ in range(3))
    dx, dw = torch.empty_like(s), torch.empty(d, device="cuda")
    desc = N.NysAddRmsNorm(rows, d, code, 1e-6, d, d, d, d, d, d)
    need = N.nystrom_add_rms_norm_workspace_bytes(desc)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def call():
        return lib.nystrom_add_rms_norm_bwd(
            ctypes.byref(desc), s.data_ptr(), gy.data_ptr(), gs.data_ptr() if with_gs else None, None, dx.data_ptr(),
            dw.data_ptr(), ws.data_ptr(), need, stream.cuda_stream)
    return call, [dx, dw]


@pytest.mark.parametrize("dtype,sizes", [("bf16", [(8192, True), (8192, False)]), ("bf16", [(4104, False), (8192, True)]),
                                         ("f32", [(4104, False), (8192, True)]), ("bf16", [(16384, True), (8200, False)])])
def test_norm_gradients_of_two_sizes(dtype, sizes):
    import torch
    import nystr_self_attention_gb300 as N
    made = [norm_back(3, d, dtype, gs, torch.cuda.Stream()) for d, gs in sizes]
    torch.cuda.synchronize()
    want = []
    for call, outs in made:
        assert call() == N.NYS_OK
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    assert at_once([c for c, _ in made], 4000) == []
    done(N)
    assert all(torch.equal(a, b) for (_, outs), w in zip(made, want) for a, b in zip(outs, w))


def attention(B, H, n, d, m, dtype, stream):
    import torch
    import nystr_self_attention_gb300 as N
    lib, code = N.load_library(), N.NYS_BF16 if dtype == "bf16" else N.NYS_FP32
    q, k, v = (torch.randn(B, H, n, d, device="cuda").to(tdtype(dtype)) for _ in range(3))
    out, w = torch.empty_like(q), torch.randn(H, 33, device="cuda")
    need = N.nystrom_attn_workspace_bytes(B, H, n, d, m, code)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def call():
        return lib.nystrom_attn_fwd_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), w.data_ptr(), out.data_ptr(),
                                       B, H, n, d, m, 6, 33, code, ws.data_ptr(), need, stream.cuda_stream)
    return call, [out, ws]


@pytest.mark.parametrize("dtype,sizes", [("bf16", [(64, 32), (64, 64)]), ("bf16", [(64, 256), (128, 256)]),
                                         ("f32", [(88, 16), (104, 16)])])
def test_attention_of_two_sizes(dtype, sizes):
    """(d, m) of each thread."""
    import torch
    import nystr_self_attention_gb300 as N
    made = [attention(1, 1, 512, d, m, dtype, torch.cuda.Stream()) for d, m in sizes]
    torch.cuda.synchronize()
    want = []
    for call, (out, _) in made:
        assert call() == N.NYS_OK
        torch.cuda.synchronize()
        want.append(out.clone())
    assert at_once([c for c, _ in made], 1500) == []
    torch.cuda.synchronize()
    own_status(N)  # nystrom_get_status reads the last call's workspace, one of these
    assert all(torch.equal(outs[0], w) for (_, outs), w in zip(made, want))


def partial_sums(seed):
    """Calls of C entries that keep something in a workspace between their kernels:
    (call on a stream, outputs) of each."""
    import torch
    import nystr_self_attention_gb300 as N
    from layer_helpers import eight
    lib = N.load_library()
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    made = []
    a, w, out = eight(N, 200, 8192), eight(N, 264, 8192), torch.empty(200, 264, device="cuda")
    N.nystrom_q8_write(a, randn(200, 8192))
    N.nystrom_q8_write(w, randn(264, 8192))
    made.append((lambda st: lib.nystrom_q8_matmul(a.desc, w.desc, out.data_ptr(), 264, N.NYS_FP32, None, 0, st), [out],
                 (a, w)))
    T, d, f = 150, 520, 1032
    x, wg, wu, gh = randn(T, d), randn(d, f), randn(d, f), randn(T, f)
    h, gate, up = (torch.empty(T, f, device="cuda") for _ in range(3))
    ff = N.NysGatedFf(T, d, f, 0, 0, N.NYS_FP32, d, f, f, f, f, d, f)
    made.append((lambda st: lib.nystrom_gated_ff_fwd(ctypes.byref(ff), x.data_ptr(), wg.data_ptr(), wu.data_ptr(),
                                                     h.data_ptr(), gate.data_ptr(), up.data_ptr(), None, 0, st),
                 [h, gate, up], (x, wg, wu, ff)))
    kept = randn(T, f), randn(T, f)
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    made.append((lambda st: lib.nystrom_gated_ff_bwd(
        ctypes.byref(ff), x.data_ptr(), wg.data_ptr(), wu.data_ptr(), kept[0].data_ptr(), kept[1].data_ptr(),
        gh.data_ptr(), dx.data_ptr(), dwg.data_ptr(), dwu.data_ptr(), None, 0, st), [dx, dwg, dwu], (kept, gh)))
    s, gy = randn(3000, 1032), randn(3000, 1032)
    ds, dw = torch.empty_like(s), torch.empty(1032, device="cuda")
    norm = N.NysAddRmsNorm(3000, 1032, N.NYS_FP32, 1e-6, *[1032] * 6)
    made.append((lambda st: lib.nystrom_add_rms_norm_bwd(ctypes.byref(norm), s.data_ptr(), gy.data_ptr(), None, None,
                                                         ds.data_ptr(), dw.data_ptr(), None, 0, st), [ds, dw], (s, gy, norm)))
    return made


def test_two_streams_without_workspaces():
    """The library's workspace passes from one stream's call to the other's."""
    import torch
    import nystr_self_attention_gb300 as N
    made = [partial_sums(1), partial_sums(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    busy = torch.zeros(1 << 28, device="cuda")
    torch.cuda.synchronize()
    want = []
    for m in made:
        for call, outs, _ in m:
            assert call(0) == N.NYS_OK
            torch.cuda.synchronize()
            want.append([t.clone() for t in outs])
    for turn in range(12):
        for t in (t for m in made for _, outs, _ in m for t in outs):
            t.fill_(3.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[turn % 2]):
            busy.add_(1.0)
        for i in range(4):
            for m, st in zip(made, streams):
                assert m[(i + turn) % 4][0](st.cuda_stream) == N.NYS_OK
        torch.cuda.synchronize()
        got = [outs for m in made for _, outs, _ in m]
        assert all(torch.equal(a, b) for o, w in zip(got, want) for a, b in zip(o, w))
    done(N)
