"""Operators around the attention module behind work of their own stream that still
has to write their inputs, and ahead of work that overwrites them."""
import pytest

from layer_helpers import done, eight, own_status

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


def tensors(seed, dtype, *shapes):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda").to(dtype) for s in shapes]


def norm(rows, d, dtype):
    def call(N, x, r, gy):
        import torch
        s, y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty(d, device="cuda")
        q = eight(N, rows, d)
        N.nystrom_add_rms_norm_fwd(x, r, None, s, y)
        N.nystrom_add_rms_norm_fwd(x, r, None, None, q)
        N.nystrom_add_rms_norm_bwd(x, gy, r, None, dx, dw)
        return [s, y, q.codes, q.scales, dx, dw]
    return call, tensors(1, dtype, (rows, d), (rows, d), (rows, d))


def back_alone(rows, d, dtype):
    def call(N, x, r, gy):
        import torch
        dx, dw = torch.empty_like(x), torch.empty(d, device="cuda")
        N.nystrom_add_rms_norm_bwd(x, gy, r, None, dx, dw)
        return [dx, dw]
    return call, tensors(2, dtype, (rows, d), (rows, d), (rows, d))


def write_and_read(rows, K, dtype, turned):
    def call(N, x):
        import torch
        q, back = eight(N, rows, K), torch.empty(rows, K, device="cuda")
        N.nystrom_q8_write(q, x.T if turned else x, 128 if turned else 1)
        N.nystrom_q8_read(q, back)
        return [q.codes, q.scales, back]
    return call, tensors(3, dtype, (K, rows) if turned else (rows, K))


def matmul(T, n, K, dtype):
    def call(N, a, sa, w, sw):
        import torch
        out = torch.empty(T, n, dtype=dtype, device="cuda")
        N.nystrom_q8_matmul(N.NystromQ8(a, sa), N.NystromQ8(w, sw), out)
        return [out]
    import torch
    import nystr_self_attention_gb300 as N
    made = []
    for rows, t in zip((T, n), tensors(4, torch.float32, (T, K), (n, K))):
        q = eight(N, rows, K)
        N.nystrom_q8_write(q, t)
        made += [q.codes, q.scales]
    return call, made


def feed_forward(T, d, f, dtype, back):
    def call(N, x, wg, wu, g, u, gh):
        import torch
        if not back:
            out = [torch.empty_like(g) for _ in range(3)]
            N.nystrom_gated_ff_fwd(x, wg, wu, *out)
        else:
            out = [torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)]
            N.nystrom_gated_ff_bwd(x, wg, wu, g, u, gh, *out)
        return out
    return call, tensors(5, dtype, (T, d), (d, f), (d, f), (T, f), (T, f), (T, f))


def cases():
    import torch
    b, s = torch.bfloat16, torch.float32
    return {
        "norm": lambda: norm(300, 1040, b), "norm32": lambda: norm(77, 8208, s), "norm ring": lambda: back_alone(400, 8192, b),
        "norm groups": lambda: back_alone(900, 264, s), "write": lambda: write_and_read(300, 1040, b, False),
        "write turned": lambda: write_and_read(264, 528, s, True), "q8 step": lambda: matmul(3, 1544, 4096, b),
        "q8 split": lambda: matmul(200, 264, 8192, s), "q8 many": lambda: matmul(900, 2056, 528, b),
        **{f"ff {T} {'back' if k else 'on'} {n}": lambda T=T, k=k, t=t: feed_forward(T, 520, 1032, t, k)
           for T in (3, 100, 300) for k in (False, True) for n, t in (("bf16", b), ("f32", s))}}


NAMES = ["norm", "norm32", "norm ring", "norm groups", "write", "write turned", "q8 step", "q8 split", "q8 many"] + [
    f"ff {T} {k} {n}" for T in (3, 100, 300) for k in ("on", "back") for n in ("bf16", "f32")]


@pytest.mark.parametrize("name", NAMES)
def test_between_writers_of_its_inputs(name):
    """A kernel on the wrong stream, or set up ahead and not waiting, sees what the
    inputs held before the copies or hold after them: zeros, which give other results."""
    import torch
    import nystr_self_attention_gb300 as N
    call, src = cases()[name]()
    want = call(N, *src)
    live = [torch.zeros_like(t) for t in src]
    wrong = call(N, *live)
    stream, busy = torch.cuda.Stream(), torch.zeros(1 << 28, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(stream):
            busy.add_(1.0)
            for a, b in zip(live, src):
                a.copy_(b)
            got = call(N, *live)
            for t in live:
                t.zero_()
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    done(N)
    assert not all(torch.equal(a, b) for a, b in zip(wrong, want))
