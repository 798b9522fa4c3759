"""Calls of the operators around the attention module as programs make them: in
graphs, on other streams, from several threads, at offsets past 32 bits, with
workspaces of their own, and in a row, as a layer uses them."""
import os
import threading

import numpy as np
import pytest

from layer_helpers import HALF, act_code, done, eight, empty, host, own_status, tdtype, upload, upload_eight
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


def norm_back(seed, rows, d, dtype):
    import torch
    import nystr_self_attention_gb300 as N
    g = torch.Generator(device="cuda").manual_seed(seed)
    s, gy, gs = (torch.randn(rows, d, generator=g, device="cuda").to(dtype) for _ in range(3))
    w = torch.randn(d, generator=g, device="cuda")

    def call(ws=None):
        dx, dw = torch.empty_like(s), torch.empty_like(w)
        N.nystrom_add_rms_norm_bwd(s, gy, gs, w, dx, dw, workspace=ws)
        return [dx, dw]
    return call, N.nystrom_add_rms_norm_workspace_bytes(
        N.NysAddRmsNorm(rows, d, N.NYS_BF16 if dtype == torch.bfloat16 else N.NYS_FP32, 1e-6))


def matmul(seed, T, n, K, dtype):
    import torch
    import nystr_self_attention_gb300 as N
    g = torch.Generator(device="cuda").manual_seed(seed)
    a, w = eight(N, T, K), eight(N, n, K)
    N.nystrom_q8_write(a, torch.randn(T, K, generator=g, device="cuda"))
    N.nystrom_q8_write(w, torch.randn(n, K, generator=g, device="cuda"), 128)

    def call(ws=None):
        out = torch.empty(T, n, dtype=dtype, device="cuda")
        N.nystrom_q8_matmul(a, w, out, workspace=ws)
        return [out]
    return call, N.nystrom_q8_matmul_workspace_bytes(
        T, n, K, N.NYS_BF16 if dtype == torch.bfloat16 else N.NYS_FP32)


def feed_forward(seed, T, d, f, dtype):
    import torch
    import nystr_self_attention_gb300 as N
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, wg, wu, gh = (torch.randn(s, generator=g, device="cuda").to(dtype) for s in ((T, d), (d, f), (d, f), (T, f)))
    desc = N.NysGatedFf(T, d, f, 0, 0, N.NYS_BF16 if dtype == torch.bfloat16 else N.NYS_FP32)
    need = max(N.nystrom_gated_ff_workspace_bytes(desc, b) for b in (False, True))

    def call(ws=None):
        h, gate, up = (torch.empty(T, f, dtype=dtype, device="cuda") for _ in range(3))
        dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
        N.nystrom_gated_ff_fwd(x, wg, wu, h, gate, up, workspace=ws)
        N.nystrom_gated_ff_bwd(x, wg, wu, gate, up, gh, dx, dwg, dwu, workspace=ws)
        return [h, gate, up, dx, dwg, dwu]
    return call, need


def some_calls(seed=0):
    import torch
    b, f = torch.bfloat16, torch.float32
    return {"norm": norm_back(seed + 1, 1200, 1032, b), "norm32": norm_back(seed + 2, 500, 4104, f),
            "q8 step": matmul(seed + 3, 3, 1544, 4096, b), "q8 split": matmul(seed + 4, 200, 264, 8192, f),
            "q8 many": matmul(seed + 5, 900, 2056, 528, b), "ff step": feed_forward(seed + 6, 5, 1032, 776, b),
            "ff": feed_forward(seed + 7, 300, 520, 1032, b), "ff32": feed_forward(seed + 8, 150, 264, 392, f)}


NAMES = ["norm", "norm32", "q8 step", "q8 split", "q8 many", "ff step", "ff", "ff32"]


def same(a, b):
    import torch
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", NAMES)
def test_the_same_call_gives_the_same_bits(name):
    call, need = some_calls()[name]
    want = call()
    import torch
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")[:max(need, 1)]
    for i in range(20):
        assert same(call(ws if i % 2 else None), want)


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(name):
    """Replayed over changed outputs, with the library's calls in between."""
    import torch
    import nystr_self_attention_gb300 as N
    call, _ = some_calls()[name]
    other, _ = some_calls(100)[name]
    want, wrong = call(), other()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        for t in got:
            t.fill_(3.0)
        graph.replay()
        assert same(other(), wrong)
        assert same(got, want)
    done(N)


@pytest.mark.parametrize("name", ["norm", "q8 step", "ff", "ff32"])
def test_two_graphs_side_by_side(name):
    import torch
    import nystr_self_attention_gb300 as N
    calls = [some_calls(s)[name][0] for s in (0, 100)]
    want = [c() for c in calls]
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([c() for _ in range(5)])
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    done(N)
    assert all(same(o, w) for out, w in zip(outs, want) for o in out)


def test_a_capture_without_a_workspace_is_refused_by_the_library():
    import ctypes
    import torch
    import nystr_self_attention_gb300 as N
    lib = N.load_library()
    s, w = torch.zeros(64, 64, device="cuda"), torch.ones(64, device="cuda")
    dx, dw = torch.empty_like(s), torch.empty_like(w)
    desc = N.NysAddRmsNorm(64, 64, N.NYS_FP32, 1e-6, 64, 64, 64, 64, 64, 64)
    x, h = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 64, device="cuda")
    ff = N.NysGatedFf(4, 64, 64, 0, 0, N.NYS_FP32, 64, 64, 64, 64, 64, 64, 64)
    w2 = torch.zeros(64, 64, device="cuda")
    graph, stream, codes = torch.cuda.CUDAGraph(), torch.cuda.Stream(), []
    with torch.cuda.graph(graph, stream=stream):
        codes.append(lib.nystrom_add_rms_norm_bwd(ctypes.byref(desc), s.data_ptr(), s.data_ptr(), None, w.data_ptr(),
                                                  dx.data_ptr(), dw.data_ptr(), None, 0, stream.cuda_stream))
        codes.append(lib.nystrom_gated_ff_fwd(ctypes.byref(ff), x.data_ptr(), w2.data_ptr(), w2.data_ptr(),
                                              h.data_ptr(), None, None, None, 0, stream.cuda_stream))
        dx.zero_()
    assert codes == [N.NYS_ERR_ARG] * 2
    done(N)


@pytest.mark.parametrize("name", NAMES)
def test_on_another_stream(name):
    """Inputs that a slow kernel of that stream still has to write."""
    import torch
    import nystr_self_attention_gb300 as N
    call, _ = some_calls()[name]
    want = call()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        busy = torch.zeros(1 << 28, device="cuda")
        for _ in range(4):
            busy.add_(1.0)
        got = [call() for _ in range(3)]
        after = [[t.clone() for t in g] for g in got]
    stream.synchronize()
    assert all(same(a, want) for a in after)
    done(N)


def test_a_stream_that_is_given():
    """stream=: not the current one; inputs written there just before."""
    import torch
    import nystr_self_attention_gb300 as N
    s = torch.cuda.Stream()
    src = torch.randn(3, 1024, device="cuda")
    w1, w2 = torch.randn(1024, 264, device="cuda"), torch.randn(1024, 264, device="cuda")
    x, h = torch.zeros_like(src), torch.zeros(3, 264, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        busy = torch.zeros(1 << 28, device="cuda")
        busy.add_(1.0)
        x.copy_(src)
    N.nystrom_gated_ff_fwd(x, w1, w2, h, stream=s)
    s.synchronize()
    want = torch.empty_like(h)
    N.nystrom_gated_ff_fwd(src, w1, w2, want)
    done(N)
    assert torch.equal(h, want)


@pytest.mark.parametrize("pair", [("q8 step", "ff step"), ("ff", "ff32"), ("norm", "q8 split")])
@pytest.mark.parametrize("own", [False, True])
def test_two_threads(pair, own):
    """On the default stream, or on one each."""
    import torch
    import nystr_self_attention_gb300 as N
    calls = [some_calls(i)[n][0] for i, n in enumerate(pair)]
    want, wrong, errors, start = [c() for c in calls], [None, None], [], threading.Barrier(2)
    torch.cuda.synchronize()

    def work(i):
        try:
            if own:
                torch.cuda.set_stream(torch.cuda.Stream())
            start.wait()
            bad = 0
            for _ in range(300):
                bad += not same(calls[i](), want[i])
            wrong[i] = bad
        except BaseException as e:  # noqa: B902
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert wrong == [0, 0]
    done(N)


def test_c_entries_without_a_workspace_from_two_threads():
    """The library's cached workspace: a call holds it until its kernels are enqueued."""
    import ctypes
    import torch
    import nystr_self_attention_gb300 as N
    lib = N.load_library()
    made = []
    for seed, (T, d, f) in enumerate([(7, 512, 520), (40, 264, 1032)]):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x, wg, wu = (torch.randn(s, generator=g, device="cuda") for s in ((T, d), (d, f), (d, f)))
        want = torch.empty(T, f, device="cuda")
        N.nystrom_gated_ff_fwd(x, wg, wu, want)
        desc = N.NysGatedFf(T, d, f, 0, 0, N.NYS_FP32, d, f, f, f, f, d, f)
        made.append((desc, x, wg, wu, want, [torch.empty_like(want) for _ in range(500)]))
    torch.cuda.synchronize()
    codes, start = [], threading.Barrier(2)

    def work(m):
        desc, x, wg, wu, _, outs = m
        start.wait()
        for h in outs:
            codes.append(lib.nystrom_gated_ff_fwd(ctypes.byref(desc), x.data_ptr(), wg.data_ptr(), wu.data_ptr(),
                                                  h.data_ptr(), None, None, None, 0, None))
    threads = [threading.Thread(target=work, args=(m,)) for m in made]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    done(N)
    assert codes == [N.NYS_OK] * 1000
    assert all(torch.equal(h, m[4]) for m in made for h in m[5])


FIRST = """
import sys, torch
import nystr_self_attention_gb300 as N
which = sys.argv[1]
torch.cuda.set_device(0)
x, w = torch.randn(8, 512, device="cuda"), torch.randn(512, 264, device="cuda")
weight, h = torch.ones(512, device="cuda"), torch.empty(8, 264, device="cuda")
q = N.NystromQ8(torch.zeros(8, 512, dtype=torch.uint8, device="cuda"), torch.zeros(1, 8, dtype=torch.int32, device="cuda"))
y = torch.empty_like(x)
out = torch.empty(8, 8, device="cuda")
def call():
    if which == "norm": N.nystrom_add_rms_norm_fwd(x, None, weight, None, y)
    elif which == "q8":
        N.nystrom_q8_write(q, x)
        N.nystrom_q8_matmul(q, q, out)
    else: N.nystrom_gated_ff_fwd(x, w, w, h)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    call()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (y, out, h)]
call()
torch.cuda.synchronize()
for a, b, n in zip(got, (y, out, h), ("norm", "q8", "ff")):
    assert n != which or torch.equal(a, b)
assert N.nystrom_get_status() == 0
"""


@pytest.mark.parametrize("which", ["norm", "q8", "ff"])
def test_a_process_s_first_call_may_be_captured(which):
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST, which], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------- one row for all, one tensor twice

def spread(t, rows):
    """A row for all rows, at a stride of 0, and its copies."""
    one = t[:1].expand(rows, t.shape[1])
    return one, one.contiguous()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(7, 264), (600, 2056), (40, 8200), (900, 1032)])
def test_norm_of_rows_that_overlap(rows, d, dtype):
    import torch
    import nystr_self_attention_gb300 as N
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, r, w = (torch.randn(n, d, generator=g, device="cuda") for n in (rows, rows, 1))
    x, r, w = x.to(tdtype(dtype)), r.to(tdtype(dtype)), w[0]
    out = []
    for one in zip(spread(x, rows), spread(r, rows)):
        s, y = torch.empty_like(x), torch.empty_like(x)
        N.nystrom_add_rms_norm_fwd(x, one[1], w, s, y)
        N.nystrom_add_rms_norm_fwd(one[0], r, w, None, y2 := torch.empty_like(x))
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        N.nystrom_add_rms_norm_bwd(one[0], x, one[1], w, dx, dw)
        dx2, dw2 = torch.empty_like(x), torch.empty_like(w)
        N.nystrom_add_rms_norm_bwd(x, one[1], one[0], w, dx2, dw2)
        out.append([s, y, y2, dx, dw, dx2, dw2])
    done(N)
    assert same(*out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [1, 128])
def test_eight_bits_of_rows_that_overlap(block, dtype):
    import torch
    import nystr_self_attention_gb300 as N
    x = torch.randn(1, 1040, device="cuda").to(tdtype(dtype))
    out = []
    for one in spread(x, 300):
        q = eight(N, 300, 1040)
        N.nystrom_q8_write(q, one, block)
        out.append([q.codes, q.scales])
    assert same(*out)
    codes = out[0][0][:1].expand(300, 1040)
    back, want = torch.empty(300, 1040, device="cuda"), torch.empty(300, 1040, device="cuda")
    N.nystrom_q8_read(N.NystromQ8(codes, out[0][1]), back)
    N.nystrom_q8_read(N.NystromQ8(*out[0]), want)
    done(N)
    assert torch.equal(back, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 20, 100, 300])
def test_gradients_of_one_row_for_all(T, dtype):
    """gh of a sum over the tokens; g and u of one token."""
    import torch
    import nystr_self_attention_gb300 as N
    d, f = 136, 264
    g = torch.Generator(device="cuda").manual_seed(T)
    x, wg, wu, gate, up, gh = (torch.randn(s, generator=g, device="cuda").to(tdtype(dtype))
                               for s in ((T, d), (d, f), (d, f), (T, f), (T, f), (T, f)))
    out = []
    for i in range(2):
        dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
        N.nystrom_gated_ff_bwd(x, wg, wu, spread(gate, T)[i], spread(up, T)[i], spread(gh, T)[i], dx, dwg, dwu)
        out.append([dx, dwg, dwu])
    done(N)
    assert same(*out)
    h = torch.empty(T, f, dtype=x.dtype, device="cuda")
    one = x[:1].expand(T, d)
    for call in (lambda: N.nystrom_gated_ff_fwd(one, wg, wu, h),
                 lambda: N.nystrom_gated_ff_bwd(one, wg, wu, gate, up, gh, None, dwg, dwu)):
        with pytest.raises(N.NystromError):
            call()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 100, 300])
def test_one_tensor_as_several_inputs(T, dtype):
    import torch
    import nystr_self_attention_gb300 as N
    d = 136
    g = torch.Generator(device="cuda").manual_seed(T)
    x, w = (torch.randn(s, generator=g, device="cuda").to(tdtype(dtype)) for s in ((T, d), (d, d)))
    out = []
    for many in (False, True):
        t = (lambda a: a.clone()) if many else (lambda a: a)
        h, dx, dwg, dwu = (torch.empty_like(a) for a in (x, x, w, w))
        N.nystrom_gated_ff_fwd(x, w, t(w), h)
        N.nystrom_gated_ff_bwd(x, w, t(w), t(x), t(x), t(x), dx, dwg, dwu)
        y, s, dn = (torch.empty_like(x) for _ in range(3))
        N.nystrom_add_rms_norm_fwd(x, t(x), None, s, y)
        N.nystrom_add_rms_norm_bwd(x, t(x), t(x), None, dn)
        q = eight(N, T // 8 * 8 or 8, 256)
        N.nystrom_q8_write(q, torch.ones(q.rows, 256, device="cuda"))
        p = eight(N, q.rows, 256)
        N.nystrom_q8_write(p, torch.ones(q.rows, 256, device="cuda"))
        o = torch.empty(q.rows, q.rows, device="cuda")
        N.nystrom_q8_matmul(q, p if many else q, o)
        out.append([h, dx, dwg, dwu, y, s, dn, o])
    done(N)
    assert same(*out)
    assert bool((out[0][-1] == 256).all())


# ------------------------------------------------------- past 32-bit offsets

def test_norm_past_32_bits():
    """140,000 rows of 16384: the last rows lie past 2^31 elements."""
    import torch
    import nystr_self_attention_gb300 as N
    rows, d = 140000, 16384
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    tail = R.rounded(np.random.default_rng(1).normal(size=(3, d)), "bf16")
    x[-3:] = upload(tail, "bf16")
    y = torch.empty_like(x)
    N.nystrom_add_rms_norm_fwd(x, None, None, None, y)
    done(N)
    _, want = R.add_rms_norm(tail, None, None, 1e-6, "bf16")
    assert (np.abs(host(y[-3:]) - want) <= np.abs(want) * (36 * 2.0 ** -24 + HALF["bf16"])).all()
    assert bool((y[:-3] == 0).all())
    gy, dx, dw = x, y, torch.empty(d, device="cuda")
    N.nystrom_add_rms_norm_bwd(x, gy, None, None, dx, dw)
    done(N)
    gx, _ = R.add_rms_norm_grad(tail, tail, None, None, 1e-6)
    # dx = r (s - h mean(s h)) cancels: off by 120 u r (|s| + |h| M), M = mean |s h|
    r = 1 / np.sqrt((tail * tail).mean(-1, keepdims=True) + 1e-6)
    M = (np.abs(tail) * np.abs(r * tail)).mean(-1, keepdims=True)
    bound = 120 * 2.0 ** -24 * r * (np.abs(tail) + np.abs(r * tail) * M) + HALF["bf16"] * np.abs(gx)
    assert (np.abs(host(dx[-3:]) - gx) <= bound).all()


def test_q8_past_32_bits():
    """1,100,000 rows of 2048 codes, and a result of 1,100,000 x 2048 values."""
    import torch
    import nystr_self_attention_gb300 as N
    rows, K, n = 1100000, 2048, 2048
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    tail = np.random.default_rng(2).integers(-4, 5, (5, K)).astype(float)
    x[-5:] = upload(tail, "bf16")
    q = eight(N, rows, K)
    N.nystrom_q8_write(q, x)
    w = np.random.default_rng(3).integers(-4, 5, (n, K)).astype(float)
    qw = eight(N, n, K)
    N.nystrom_q8_write(qw, upload(w, "f32"), 128)
    N.nystrom_q8_read(q, x)
    out = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    N.nystrom_q8_matmul(q, qw, out)
    done(N)
    assert (host(x[-5:]) == tail).all() and bool((x[:-5] == 0).all())
    assert (host(out[-5:]) == R.to_bf16(tail @ w.T)).all()
    assert bool((out[:-5] == 0).all())


def test_feed_forward_past_32_bits():
    """270,000 tokens of 8192 features."""
    import torch
    import nystr_self_attention_gb300 as N
    T, d, f = 270000, 64, 8192
    rng = np.random.default_rng(4)
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    tail = rng.integers(-2, 3, (4, d)).astype(float)
    x[-4:] = upload(tail, "bf16")
    wg, wu = (rng.integers(-2, 3, (d, f)).astype(float) for _ in range(2))
    tg, tu = upload(wg, "bf16"), upload(wu, "bf16")
    h, g, u = (torch.empty(T, f, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    N.nystrom_gated_ff_fwd(x, tg, tu, h, g, u, activation=N.NYS_ACT_RELU)
    done(N)
    want, wantg, wantu = R.gated_ff(tail, wg, wu, "relu")
    assert (host(h[-4:]) == R.to_bf16(want)).all() and bool((h[:-4] == 0).all())
    gh = torch.zeros_like(h)
    ghost = rng.integers(-1, 2, (4, f)).astype(float)
    gh[-4:] = upload(ghost, "bf16")
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(tg), torch.empty_like(tu)
    N.nystrom_gated_ff_bwd(x, tg, tu, g, u, gh, dx, dwg, dwu, activation=N.NYS_ACT_RELU)
    done(N)
    ga, ua = host(g[-4:]), host(u[-4:])
    ex, eg, eu = R.gated_ff_grad(tail, wg, wu, ga, ua, ghost, "relu", "bf16")
    assert (host(dx[-4:]) == R.to_bf16(ex)).all() and bool((dx[:-4] == 0).all())
    assert (host(dwg) == R.to_bf16(eg)).all() and (host(dwu) == R.to_bf16(eu)).all()


# ------------------------------------------------------------------ together

def test_a_layer_in_eight_bits():
    """Two sequences through a layer as it serves a prompt: the sum and norm in 8
    bits, a packed QKV projection, attention, the output projection, the sum and
    norm again, the gated product, the projection back. The oracle rounds where
    the layer does; a code next to a border may differ, which the 2-norm of a
    result feels by far less than the 2^-5 that one code step is of a value."""
    import torch
    import nystr_self_attention_gb300 as N
    from oracle import nystrom_ref as A
    B, n, H, d, m, f = 2, 128, 4, 64, 32, 520
    D, T = H * d, B * n
    rng = np.random.default_rng(9)
    x0, r0 = (R.to_bf16(rng.normal(size=(T, D))) for _ in range(2))
    w1, w2 = ((1 + 0.1 * rng.normal(size=D)).astype(np.float32) for _ in range(2))
    wqkv, wo, wg, wu, wd = (R.to_bf16(rng.normal(size=s) / np.sqrt(s[1]))
                            for s in ((3 * D, D), (D, D), (f, D), (f, D), (D, 528)))
    wd[:, f:] = 0  # K in sixteens

    def weight8(w):
        q = eight(N, *w.shape)
        N.nystrom_q8_write(q, upload(w, "bf16"), 128)
        return q
    q_qkv, q_o, q_d = weight8(wqkv), weight8(wo), weight8(wd)

    # the layer
    stream, qx = empty(T, D, "bf16"), eight(N, T, D)
    N.nystrom_add_rms_norm_fwd(upload(x0, "bf16"), upload(r0, "bf16"), torch.from_numpy(w1).cuda(), stream, qx)
    qkv = empty(T, 3 * D, "bf16")
    N.nystrom_q8_matmul(qx, q_qkv, qkv)
    heads = [t.reshape(B, n, H, d).transpose(1, 2).contiguous() for t in qkv.split(D, dim=1)]
    att = N.nystrom_attention(*heads, None, m, 6)
    merged = att.transpose(1, 2).reshape(T, D).contiguous()
    qa, o = eight(N, T, D), empty(T, D, "bf16")
    N.nystrom_q8_write(qa, merged)
    N.nystrom_q8_matmul(qa, q_o, o)
    y = empty(T, D, "bf16")
    N.nystrom_add_rms_norm_fwd(o, stream, torch.from_numpy(w2).cuda(), stream, y)
    h = torch.zeros(T, 528, dtype=torch.bfloat16, device="cuda")
    N.nystrom_gated_ff_fwd(y, upload(wg, "bf16").T, upload(wu, "bf16").T, h[:, :f])
    qh, out = eight(N, T, 528), empty(T, D, "bf16")
    N.nystrom_q8_write(qh, h)
    N.nystrom_q8_matmul(qh, q_d, out)
    done(N)

    # the oracle
    def q8(v, rows=1):
        return R.q8_read(*R.q8_write(v, rows))
    s, yn = R.add_rms_norm(x0, r0, w1, 1e-6, "bf16")
    qkv_ref = R.to_bf16(q8(yn) @ q8(wqkv, 128).T)
    hd = [t.reshape(B, n, H, d).transpose(0, 2, 1, 3) for t in np.split(qkv_ref, 3, axis=1)]
    att_ref = A.nystrom_attention(*(t.astype(np.float32) for t in hd), np.zeros((H, 0)), m, 6)
    mg = R.to_bf16(np.asarray(att_ref, np.float64).transpose(0, 2, 1, 3).reshape(T, D))
    o_ref = R.to_bf16(q8(mg) @ q8(wo, 128).T)
    s2, y2 = R.add_rms_norm(o_ref, s, w2, 1e-6, "bf16")
    h_ref = np.zeros((T, 528))
    h_ref[:, :f] = R.to_bf16(R.gated_ff(R.to_bf16(y2), wg.T, wu.T, "silu")[0])
    out_ref = R.to_bf16(q8(h_ref) @ q8(wd, 128).T)
    for got, want in ((stream, s2), (out, out_ref)):
        g = host(got)
        assert np.linalg.norm(g - want) <= 2e-2 * np.linalg.norm(want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_training_step_of_a_block(dtype):
    """z = x + r, y = norm(z), h = ff(y): gradients of x (and r), the norm's
    weight and the feed-forward's, through the kept tensors, against the oracle's
    chain. Each step rounds at most three times per value (kept, gradient, result):
    6 half steps in the 2-norm, and what the fp32 sums add."""
    import torch
    import nystr_self_attention_gb300 as N
    T, D, f = 300, 264, 520
    rng = np.random.default_rng(11)
    x, r = (R.rounded(rng.normal(size=(T, D)), dtype) for _ in range(2))
    w = (1 + 0.2 * rng.normal(size=D)).astype(np.float32)
    wg, wu = (R.rounded(rng.normal(size=(D, f)) / np.sqrt(D), dtype) for _ in range(2))
    gh, gz = R.rounded(rng.normal(size=(T, f)), dtype), R.rounded(rng.normal(size=(T, D)), dtype)
    tw, tg, tu = torch.from_numpy(w).cuda(), upload(wg, dtype), upload(wu, dtype)
    z, y, h, g, u = empty(T, D, dtype), empty(T, D, dtype), *(empty(T, f, dtype) for _ in range(3))
    N.nystrom_add_rms_norm_fwd(upload(x, dtype), upload(r, dtype), tw, z, y)
    N.nystrom_gated_ff_fwd(y, tg, tu, h, g, u, activation=N.NYS_ACT_GELU)
    dy, dwg, dwu = empty(T, D, dtype), torch.empty_like(tg), torch.empty_like(tu)
    N.nystrom_gated_ff_bwd(y, tg, tu, g, u, upload(gh, dtype), dy, dwg, dwu, activation=N.NYS_ACT_GELU)
    dx, dw = empty(T, D, dtype), torch.empty(D, device="cuda")
    N.nystrom_add_rms_norm_bwd(z, dy, upload(gz, dtype), tw, dx, dw)
    done(N)
    zr, yr = R.add_rms_norm(x, r, w, 1e-6, dtype)
    hr, gr, ur = R.gated_ff(yr, wg, wu, "gelu")
    dyr, dwgr, dwur = R.gated_ff_grad(yr, wg, wu, gr, ur, gh, "gelu")
    dxr, dwr = R.add_rms_norm_grad(zr, dyr, gz, w, 1e-6)
    bound = 6 * HALF[dtype] if dtype == "bf16" else 1e-5
    for got, want in ((h, hr), (dx, dxr), (dw, dwr), (dwg, dwgr), (dwu, dwur)):
        assert np.linalg.norm(host(got) - want) <= bound * np.linalg.norm(want)


def test_prompt_then_steps_agree():
    """Tokens one at a time, a few at a time, and all at once: the same layer. The
    forms sum K in other orders: fp32 results off by no more than its 2-norm bound."""
    import torch
    import nystr_self_attention_gb300 as N
    torch.manual_seed(5)
    T, D, f = 150, 520, 1032
    x, wg, wu = torch.randn(T, D, device="cuda"), torch.randn(D, f, device="cuda"), torch.randn(D, f, device="cuda")
    q, w = eight(N, T, D - 8), eight(N, f, D - 8)
    N.nystrom_q8_write(q, x[:, :D - 8].contiguous())
    N.nystrom_q8_write(w, wg[:D - 8].T, 128)
    whole, whole8 = torch.empty(T, f, device="cuda"), torch.empty(T, f, device="cuda")
    N.nystrom_gated_ff_fwd(x, wg, wu, whole)
    N.nystrom_q8_matmul(q, w, whole8)
    for step in (1, 20, 50, 100):
        part, part8 = torch.empty_like(whole), torch.empty_like(whole8)
        for t in range(0, T, step):
            rows = slice(t, min(t + step, T))
            N.nystrom_gated_ff_fwd(x[rows], wg, wu, part[rows])
            qs = N.NystromQ8(q.codes[rows], q.scales[:, rows].contiguous())
            N.nystrom_q8_matmul(qs, w, part8[rows])
        assert float((part - whole).norm() / whole.norm()) <= 2e-6
        assert float((part8 - whole8).norm() / whole8.norm()) <= 2e-6
    done(N)
