"""Calls of different sizes from two host threads at once."""
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
