"""Edges of the 4-bit cache's calls."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    import torch
    from nystr_self_attention_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)


def i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cache_of(B, Hk, d, page, per, seed=0):
    import torch
    import nystr_self_attention_gb300 as N
    g = torch.Generator(device="cuda").manual_seed(seed)
    data = torch.randint(0, 256, (N.nystrom_kv4_cache_bytes(B * per, page, Hk, d),), dtype=torch.uint8,
                         generator=g, device="cuda")
    table = torch.arange(B * per, dtype=torch.int32, device="cuda").view(B, per)
    return N.NystromKv4Cache(data, table, page, Hk, d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_positions_without_a_page_read_as_plus_zero(d, dtype):
    import torch
    import nystr_self_attention_gb300 as N
    c = cache_of(3, 2, d, 32, 2)
    c.block_table[1, 0] = -1
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    k, v = (torch.full((3, 2, 40, d), 5.0, dtype=t, device="cuda") for _ in range(2))
    N.nystrom_kv4_read(c, k, v, i32([50, 0, -16]))
    assert N.nystrom_get_status() == N.NYS_ERR_INDEX
    for x in (k, v):
        for rows in (x[0, :, 14:], x[1, :, :32], x[2, :, :16]):
            assert (rows == 0).all() and not torch.signbit(rows.float()).any()


FIRST = """
import sys, numpy as np, torch
import nystr_self_attention_gb300 as N
which, rows = sys.argv[1], {"chunk": 70}.get(sys.argv[1], 1)
B, Hk, d, n = 2, 2, 64, 100
g = torch.Generator(device="cuda").manual_seed(1)
data = torch.full((N.nystrom_kv4_cache_bytes(B * 4, 32, Hk, d),), 0x3F, dtype=torch.uint8, device="cuda")
cache = N.NystromKv4Cache(data, torch.arange(B * 4, dtype=torch.int32, device="cuda").view(B, 4), 32, Hk, d)
k, v = (torch.randn(B, Hk, n, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
q = torch.randn(B, 4, rows, d, generator=g, device="cuda").to(torch.bfloat16)
a, b, dw = torch.zeros_like(k), torch.zeros_like(v), torch.zeros(2, d, device="cuda")
out, lens = torch.zeros_like(q), torch.full((B,), n, dtype=torch.int32, device="cuda")
inv = 10000.0 ** (-np.arange(32) / 32)
call = {
    "write": lambda: N.nystrom_kv4_write(cache, k, v),
    "read": lambda: N.nystrom_kv4_read(cache, a, b),
    "token": lambda: N.nystrom_kv4_attn_fwd(cache, q, out, lens, 128),
    "split": lambda: N.nystrom_kv4_attn_fwd(cache, q, out, lens, 5000),
    "chunk": lambda: N.nystrom_kv4_attn_fwd(cache, q, out, lens, 128),
    "rope": lambda: N.nystrom_qk_norm_rope_fwd(k, v, a, b, None, inv),
    "gradient": lambda: N.nystrom_qk_norm_rope_bwd(k, v, v, k, a, b, None, inv, None, None, dw[0], dw[1]),
}[which]
results = (data, out, a, b, dw)
before = [t.clone() for t in results]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
replayed = [t.clone() for t in results]
for t, t0 in zip(results, before):
    t.copy_(t0)
call()
torch.cuda.synchronize()
assert N.nystrom_get_status() == N.NYS_OK
same = [torch.equal(x, y) for x, y in zip(replayed, results)]
moved = any(not torch.equal(x, y) for x, y in zip(replayed, before))
assert all(same) and moved, (same, moved)
"""


@pytest.mark.parametrize("which", ["write", "read", "token", "split", "chunk", "rope", "gradient"])
def test_a_first_call_may_be_captured(which):
    """In a process of its own, whose first call of the library's kernels is
    inside a capture: replayed, it gives what an eager call gives."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST, which], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_sizes_and_scales_that_a_call_cannot_hold_are_refused():
    """Not cut to 32 bits on their way, and a scale that vanishes in fp32 does
    not turn into the default one."""
    import torch
    import nystr_self_attention_gb300 as N
    c = cache_of(1, 2, 64, 32, 2)
    q, lens = torch.zeros(1, 4, 1, 64, device="cuda"), i32([40])
    out = torch.full_like(q, 7.0)
    for limit in (2 ** 32 + 40, 2 ** 31, -1, -2 ** 32 + 64):
        with pytest.raises((ValueError, N.NystromError)):
            N.nystrom_kv4_attn_fwd(c, q, out, lens, limit)
    for scale in (0.0, 1e-50, -1e-60, float("nan"), float("inf"), 1e39, 3e38):
        with pytest.raises((ValueError, N.NystromError)):
            N.nystrom_kv4_attn_fwd(c, q, out, lens, 64, scale=scale)
    many = torch.zeros(1, 2, 1, 64, device="cuda").expand(1, 2, 2 ** 32 + 3, 64)
    with pytest.raises((ValueError, N.NystromError)):
        N.nystrom_kv4_write(c, many, many)
    torch.cuda.synchronize()
    assert (out == 7.0).all() and N.nystrom_get_status() == N.NYS_OK
    N.nystrom_kv4_attn_fwd(c, q, out, lens, 2 ** 31 - 1, scale=1e-30)
    assert N.nystrom_get_status() == N.NYS_OK


@pytest.mark.parametrize("nq", [1, 60])
def test_offsets_past_32_bits(nq):
    """Pages beyond 4 GiB of a pool and rows 2^31 elements and more apart: the
    bits of the same call in compact memory."""
    import numpy as np
    import torch
    import nystr_self_attention_gb300 as N
    B, Hk, Hq, d, n, page = 3, 2, 4, 128, 200, 16
    per = -(-n // page)
    page_bytes = N.nystrom_kv4_cache_bytes(1, page, Hk, d)
    pages = (5 << 30) // page_bytes
    data = torch.empty(pages * page_bytes, dtype=torch.uint8, device="cuda")
    far = N.NystromKv4Cache(data, (pages - 1 - 7 * torch.arange(B * per, device="cuda")).to(torch.int32).view(B, per),
                            page, Hk, d)
    near = cache_of(B, Hk, d, page, per)
    apart = 2 ** 31 + 128  # elements between sequences
    room = torch.empty(2 * apart + (1 << 22), dtype=torch.bfloat16, device="cuda")
    at = 0

    def wide(H, rows):
        nonlocal at
        t = room.as_strided((B, H, rows, d), (apart, rows * d, d, 1), at)
        at += H * rows * d
        return t.normal_()

    k, v, q, out = wide(Hk, n), wide(Hk, n), wide(Hq, nq), wide(Hq, nq)
    ck, cv, cq, cout = (t.contiguous() for t in (k, v, q, out))
    inv = 10000.0 ** (-np.arange(64) / 64)
    starts, lens = i32([0] * B), i32([n, n - 7, n - 100])
    for cache, (a, b, x, y) in ((far, (k, v, q, out)), (near, (ck, cv, cq, cout))):
        N.nystrom_qk_norm_rope_fwd(a, b, a, b, None, inv)
        N.nystrom_kv4_write(cache, a, b, starts)
        N.nystrom_kv4_attn_fwd(cache, x, y, lens, n)
        N.nystrom_kv4_read(cache, a, b, i32([3, 0, 1]), i32([n - 3, n, n - 1]))
        N.nystrom_qk_norm_rope_bwd(x, None, y, None, y, None, None, inv)
    assert N.nystrom_get_status() == N.NYS_OK
    for x, y in ((k, ck), (v, cv), (q, cq), (out, cout)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 60])
def test_a_query_with_nan_or_infinity_spoils_its_own_row_alone(nq, dtype):
    import torch
    import nystr_self_attention_gb300 as N
    B, Hk, Hq, d, n = 2, 2, 4, 128, 3000
    c = cache_of(B, Hk, d, 64, 47)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(B, Hk, n, d, generator=g, device="cuda").to(t) for _ in range(2))
    N.nystrom_kv4_write(c, k, v)
    q = torch.randn(B, Hq, nq, d, generator=g, device="cuda").to(t)
    lens = i32([n, nq // 2])  # the second sequence's first queries see nothing
    want, out = torch.empty_like(q), torch.empty_like(q)
    N.nystrom_kv4_attn_fwd(c, q, want, lens, n)
    bad = torch.zeros(B, Hq, nq, dtype=torch.bool, device="cuda")
    for h, i, x in ((0, 0, float("nan")), (1, nq // 2, float("inf")), (3, nq - 1, -float("inf"))):
        q[:, h, i, 5 * h] = x
        bad[:, h, i] = True
    N.nystrom_kv4_attn_fwd(c, q, out, lens, n)
    assert N.nystrom_get_status() == N.NYS_OK
    sees = torch.arange(nq, device="cuda")[None] >= (nq - lens[:, None])  # [B, nq]
    sees = sees[:, None].expand(B, Hq, nq)
    assert torch.isnan(out[bad & sees]).all() and (out[~sees] == 0).all()
    assert torch.equal(out[~bad], want[~bad]) and torch.isfinite(want).all()


@pytest.mark.parametrize("nq", [1, 60])
def test_two_graphs_replayed_side_by_side(nq):
    """Captured one after the other, replayed at once on two streams: each has
    a workspace of its own."""
    import torch
    import nystr_self_attention_gb300 as N
    B, Hk, Hq, d, n = 3, 2, 8, 128, 3000
    runs = []
    for seed in range(2):
        c = cache_of(B, Hk, d, 64, 47)
        g = torch.Generator(device="cuda").manual_seed(seed)
        k, v = (torch.randn(B, Hk, n, d, generator=g, device="cuda") for _ in range(2))
        N.nystrom_kv4_write(c, k, v)
        q = torch.randn(B, Hq, nq, d, generator=g, device="cuda").to(torch.bfloat16)
        out, lens = torch.empty_like(q), i32([n, n - 700 * (seed + 1), 5])
        N.nystrom_kv4_attn_fwd(c, q, out, lens, n)
        want = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(4):
                N.nystrom_kv4_attn_fwd(c, q, out, lens, n)
        runs.append((graph, torch.cuda.Stream(), out, want, (c, q, lens)))
    torch.cuda.synchronize()
    for _ in range(25):
        for _, _, out, _, _ in runs:
            out.fill_(9.0)
        torch.cuda.synchronize()
        for graph, stream, _, _, _ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for _, _, out, want, _ in runs)
    assert N.nystrom_get_status() == N.NYS_OK
