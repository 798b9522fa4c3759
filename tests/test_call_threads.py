"""Two host threads that call at the same time. A call of the attention over the
cache, or of the gradients with weight sums, is two kernels with a workspace
between them: whatever the threads' calls interleave to, each has the bits that
it has alone."""
import threading

import pytest

pytestmark = pytest.mark.gpu

ROUNDS = 3000


@pytest.fixture(scope="module", autouse=True)
def library():
    import torch
    from nystr_self_attention_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)


def i32(x):
    import torch
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def attention_call(seed, B, Hq, Hk, n, nq, dtype):
    """A call whose items are cut, so that its parts go through the workspace."""
    import torch
    import nystr_self_attention_gb300 as N
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = -(-n // 64)
    data = torch.zeros(N.nystrom_kv4_cache_bytes(B * pages, 64, Hk, 128), dtype=torch.uint8, device="cuda")
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
    cache = N.NystromKv4Cache(data, table, 64, Hk, 128)
    k, v = (torch.randn(B, Hk, n, 128, generator=g, device="cuda") for _ in range(2))
    N.nystrom_kv4_write(cache, k, v)
    q = torch.randn(B, Hq, nq, 128, generator=g, device="cuda").to(dtype)
    outs, lens = [torch.empty_like(q) for _ in range(ROUNDS)], i32([n] * B)
    assert N.nystrom_kv4_attn_workspace_bytes(cache, B, nq, Hq, n, N.NYS_BF16 if dtype == torch.bfloat16
                                              else N.NYS_FP32) > 0

    def call(r):
        N.nystrom_kv4_attn_fwd(cache, q, outs[r], lens, n)
        return outs[r]
    return call


def gradient_call(seed, n, dtype):
    import numpy as np
    import torch
    import nystr_self_attention_gb300 as N
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, gq, gk = (torch.randn(1, 4, n, 64, generator=g, device="cuda").to(dtype) for _ in range(4))
    dq, dk, dw = torch.empty_like(q), torch.empty_like(k), torch.empty(ROUNDS, 2, 64, device="cuda")
    inv = 10000.0 ** (-np.arange(32) / 32)

    def call(r):
        N.nystrom_qk_norm_rope_bwd(q, k, gq, gk, dq, dk, None, inv, None, None, dw[r, 0], dw[r, 1])
        return dw[r]
    return call


def calls_of(kind):
    import torch
    if kind == "attention":
        return attention_call(1, 1, 8, 2, 2000, 1, torch.bfloat16), attention_call(2, 2, 4, 4, 1500, 3, torch.float32)
    if kind == "chunks":
        return (attention_call(3, 1, 8, 1, 3000, 30, torch.bfloat16),
                attention_call(4, 1, 4, 1, 2500, 50, torch.bfloat16))
    return gradient_call(5, 300, torch.float32), gradient_call(6, 700, torch.bfloat16)


def differing(calls, streams=(None, None)):
    """Rounds, per thread, whose results are not those of the call alone."""
    import torch
    want, wrong, errors, start = [], [None, None], [], threading.Barrier(2)
    for call in calls:
        want.append(call(0).clone())
        torch.cuda.synchronize()

    def work(i):
        try:
            if streams[i] is not None:
                torch.cuda.set_stream(streams[i])
            start.wait()
            got = [calls[i](r) for r in range(ROUNDS)]
            wrong[i] = sum(not torch.equal(x, want[i]) for x in got)
        except BaseException as e:  # noqa: B902
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    return wrong


@pytest.mark.parametrize("kind", ["attention", "chunks", "gradients"])
def test_threads_on_the_default_stream(kind):
    import torch
    import nystr_self_attention_gb300 as N
    assert torch.cuda.current_stream().cuda_stream == 0
    assert differing(calls_of(kind)) == [0, 0]
    assert N.nystrom_get_status() == N.NYS_OK


@pytest.mark.parametrize("kind", ["attention", "gradients"])
def test_threads_on_streams_of_their_own(kind):
    import torch
    calls = calls_of(kind)
    torch.cuda.synchronize()
    assert differing(calls, [torch.cuda.Stream(), torch.cuda.Stream()]) == [0, 0]


@pytest.mark.parametrize("kind", ["attention", "gradients"])
def test_workspaces_of_threads_are_apart(kind, monkeypatch):
    """On the default stream: each thread has one of its own, which it keeps
    from call to call."""
    import torch
    from nystr_self_attention_gb300 import _binding
    name = "nystrom_kv4_attn_fwd" if kind == "attention" else "nystrom_qk_norm_rope_bwd"
    real, seen, errors, both = _binding.load_library(), {}, [], threading.Barrier(2)

    class Library:
        def __getattr__(self, attr):
            fn = getattr(real, attr)
            if attr != name:
                return fn

            def call(*args):  # ..., workspace, bytes, stream
                seen.setdefault(threading.get_ident(), set()).add((args[-3], args[-2]))
                return fn(*args)
            return call

    calls = calls_of(kind)
    torch.cuda.synchronize()
    monkeypatch.setattr(_binding, "_lib", Library())

    def work(i):
        try:
            calls[i](0)
            both.wait()
            calls[i](1)
            both.wait()
        except BaseException as e:  # noqa: B902
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    (a,), (b,) = seen.values()
    assert a[0] and b[0] and (a[0] + a[1] <= b[0] or b[0] + b[1] <= a[0])


@pytest.mark.parametrize("kind", ["attention", "chunks", "gradients"])
def test_threads_with_the_librarys_workspace(kind, monkeypatch):
    """The same through the C entries with no workspace given, on one stream."""
    import torch
    import nystr_self_attention_gb300 as N
    from nystr_self_attention_gb300 import _binding
    name = "nystrom_qk_norm_rope_bwd" if kind == "gradients" else "nystrom_kv4_attn_fwd"
    real = _binding.load_library()
    fn = getattr(real, name)

    class Library:
        def __getattr__(self, attr):
            if attr != name:
                return getattr(real, attr)
            return lambda *args: fn(*args[:-3], None, 0, args[-1])

    calls = calls_of(kind)
    torch.cuda.synchronize()
    monkeypatch.setattr(_binding, "_lib", Library())
    assert differing(calls) == [0, 0]
    assert N.nystrom_get_status() == N.NYS_OK
