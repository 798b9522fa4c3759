"""GPU parity of the 4-bit key/value cache (written and read back: bit for bit
the format's) and of attention over it, against the fp64 oracle.

Attention bounds, per element, with u = 2^-24, A = sum p |v| and S the largest
sum |q k| scale of the row's keys. A score is a sum of at most 128 products and
scales, held in fp32 along at most 32 dependent steps of at most 2u each: 64u S,
and the exponential adds 4u S for its argument and 4u of its own; numerator and
denominator both feel it: p is off by 2 (68 u S + 4u). The sum over V adds 64u.
So fp32: A (136 u S + 72u) + u |out|, taken as A u (160 S + 160). bf16 rounds each
probability to 2^-8 of itself and the result to 2^-8: A 2^-8 + |out| 2^-8 more.
bf16 calls with many queries unpack values to 16-bit floats: a product of a 4-bit
code and an 8-bit scale has 12 bits, rounded to fp16's 11 (2^-12 of itself, inside
what probabilities rounded to fp16 instead of bf16 leave) or, where the scales of
32 tokens span more than 2^8, to bf16's 8: |v| is then off by 2^-8 of itself and
the sum by A 2^-8 once more (`wide`)."""
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


def heads(x, dtype, order):
    """Device [B, H, n, d] view of a host array of that shape."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32))
    t = t.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    return t.transpose(1, 2).contiguous().transpose(1, 2) if order == "bnhd" else t


def host(t):
    return t.detach().double().cpu().numpy()


class Both:
    """The same pool on the device and in the oracle."""

    def __init__(self, B, Hk, d, page, per_seq, seed=1, spare=2):
        import torch
        import nystr_self_attention_gb300 as N
        rng = np.random.default_rng(seed)
        pool = B * per_seq + spare
        self.table = rng.permutation(pool)[:B * per_seq].reshape(B, per_seq).astype(np.int32)
        raw = rng.integers(0, 256, N.nystrom_kv4_cache_bytes(pool, page, Hk, d)).astype(np.uint8)
        self.data = torch.from_numpy(raw).cuda()
        self.dtable = torch.from_numpy(self.table).cuda()
        self.dev = N.NystromKv4Cache(self.data, self.dtable, page, Hk, d)
        self.ref = C.Cache(raw, self.table, page, Hk, d)
        self.rng, self.B, self.Hk, self.d = rng, B, Hk, d

    def bytes(self):
        return self.data.cpu().numpy().reshape(self.ref.raw.shape)

    def fill(self, lens, dtype="bf16"):
        """Tokens 0 .. lens[b]-1 of every sequence on both sides."""
        import nystr_self_attention_gb300 as N
        n = max(1, max(lens))
        k, v = (self.rng.standard_normal((self.B, self.Hk, n, self.d)) for _ in range(2))
        k, v = heads(k, dtype, "bnhd"), heads(v, dtype, "bnhd")
        N.nystrom_kv4_write(self.dev, k, v, None, i32(lens))
        self.ref.write(host(k), host(v), [0] * self.B, lens)


def i32(x):
    import torch
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


IO = {
    # B, Hk, d, page, pages per sequence, n, starts, counts, dtype, order
    "d128": (3, 2, 128, 64, 3, 70, [0, 50, 122], [70, 64, 70], "bf16", "bhnd"),
    "d128_f32": (2, 3, 128, 16, 9, 37, [3, 100], [37, 1], "f32", "bnhd"),
    "d64": (2, 5, 64, 32, 5, 130, [0, 15], [130, 129], "bf16", "bnhd"),
    "d64_f32": (4, 1, 64, 256, 1, 17, [0, 1, 239, 16], [17, 16, 17, 0], "f32", "bhnd"),
    "d32": (2, 2, 32, 48, 2, 33, [63, 16], [33, 31], "bf16", "bnhd"),
    "d32_f32": (1, 7, 32, 16, 6, 80, [11], [80], "f32", "bhnd"),
    "one": (5, 4, 128, 32, 2, 1, [0, 15, 16, 31, 63], [1, 1, 1, 0, 1], "bf16", "bnhd"),
}


@pytest.mark.parametrize("name", IO)
def test_write_and_read_bit_for_bit(name):
    import torch
    import nystr_self_attention_gb300 as N
    B, Hk, d, page, per, n, starts, counts, dtype, order = IO[name]
    c = Both(B, Hk, d, page, per)
    rng = np.random.default_rng(8)
    k = rng.standard_normal((B, Hk, n, d)) * np.exp2(rng.integers(-20, 20, (B, Hk, n, 1)))
    v = np.round(rng.standard_normal((B, Hk, n, d)) * 4) / 2  # many ties
    k[0, 0, 0] = 0
    k, v = heads(k, dtype, order), heads(v, dtype, order)
    N.nystrom_kv4_write(c.dev, k, v, i32(starts), i32(counts))
    c.ref.write(host(k), host(v), starts, counts)
    assert N.nystrom_get_status() == N.NYS_OK
    assert np.array_equal(c.bytes(), c.ref.raw)
    kb, vb = torch.full_like(k, 5.0), torch.full_like(v, 5.0)
    N.nystrom_kv4_read(c.dev, kb, vb, i32(starts), i32(counts))
    assert N.nystrom_get_status() == N.NYS_OK
    for b in range(B):
        for i in range(n):
            if i < counts[b]:
                K, V = c.ref.token(b, starts[b] + i)
                want = [torch.from_numpy(x).to(torch.float32).to(k.dtype) for x in (K, V)]
            else:
                want = [torch.full((Hk, d), 5.0, dtype=k.dtype)] * 2
            assert torch.equal(kb[b, :, i].cpu(), want[0]) and torch.equal(vb[b, :, i].cpu(), want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_values(dtype):
    """Zeros, the smallest and largest magnitudes, infinities and NaN, and
    ratios that fall on or next to a rounding border."""
    import nystr_self_attention_gb300 as N
    rng = np.random.default_rng(4)
    n = 64
    k = rng.standard_normal((1, 1, n, 64)).astype(np.float32)
    k *= np.exp2(np.linspace(-149, 126, n)).astype(np.float32)[:, None]
    v = rng.standard_normal((1, 1, n, 64)).astype(np.float32)
    v[0, 0, 0], v[0, 0, 1] = 0, -0.0
    v[0, 0, 2, 7], v[0, 0, 3, 40], v[0, 0, 4, 0] = np.inf, np.nan, -np.inf
    v[0, 0, 5] = 2.0 ** -149
    v[0, 0, 6] = np.float32(3.38e38)
    for i in range(8, n):  # (j + 1/2) scale, and fp32 neighbours of it
        top = np.float32(7 * (1 + i / 64))
        s = C.bf16_value(C.bf16_bits_toward_zero(np.float32(top) / np.float32(7)))
        v[0, 0, i, :32] = np.float32((np.arange(32) % 14 - 6.5) * s)
        if i % 3:
            v[0, 0, i, :32] = np.nextafter(v[0, 0, i, :32], np.float32(np.inf if i % 3 == 1 else -np.inf))
        v[0, 0, i, 31] = top
    c = Both(1, 1, 64, 64, 1)
    kd, vd = heads(k, dtype, "bhnd"), heads(v, dtype, "bhnd")
    N.nystrom_kv4_write(c.dev, kd, vd)
    c.ref.write(host(kd), host(vd), [0], [n])
    assert np.array_equal(c.bytes(), c.ref.raw)


def test_strided_and_packed_rows():
    """K and V as slices of one packed projection, read back into another."""
    import torch
    import nystr_self_attention_gb300 as N
    c = Both(2, 3, 64, 32, 2)
    qkv = torch.randn(2, 40, 9, 64, device="cuda").to(torch.bfloat16)
    k, v = qkv[:, :, 3:6].transpose(1, 2), qkv[:, :, 6:9].transpose(1, 2)
    N.nystrom_kv4_write(c.dev, k, v, i32([5, 24]))
    c.ref.write(host(k), host(v), [5, 24], [40, 40])
    assert np.array_equal(c.bytes(), c.ref.raw)
    out = torch.full((2, 3, 2, 48, 64), 9.0, device="cuda", dtype=torch.bfloat16)
    N.nystrom_kv4_read(c.dev, out[:, :, 0, :40], out[:, :, 1, :40], i32([5, 24]))
    assert (out[:, :, :, 40:] == 9.0).all() and not (out[:, :, :, :40] == 9.0).all()


def test_positions_and_pages_out_of_range():
    """Skipped, reported once, and nothing else disturbed."""
    import torch
    import nystr_self_attention_gb300 as N
    c = Both(3, 2, 64, 32, 3)
    c.table[1, 1] = c.ref.raw.shape[0]
    c.table[2, 0] = -1
    c.dtable.copy_(torch.from_numpy(c.table))
    c.ref.table = c.table
    k, v = (heads(np.random.default_rng(i).standard_normal((3, 2, 80, 64)), "f32", "bhnd") for i in (1, 2))
    starts, counts = [-30, 20, 10], [1000, 80, 80]
    N.nystrom_kv4_write(c.dev, k, v, i32(starts), i32(counts))
    assert N.nystrom_get_status() == N.NYS_ERR_INDEX
    assert N.nystrom_get_status() == N.NYS_OK
    c.ref.write(host(k), host(v), starts, [80, 80, 80])
    assert np.array_equal(c.bytes(), c.ref.raw)
    kb, vb = torch.full_like(k, 5.0), torch.full_like(v, 5.0)
    N.nystrom_kv4_read(c.dev, kb, vb, i32([90, 20, -7]), i32([80, -3, 2 ** 31 - 1]))
    assert N.nystrom_get_status() == N.NYS_ERR_INDEX
    assert (kb[0, :, 6:] == 0).all() and (vb[0, :, 6:] == 0).all()
    assert torch.equal(kb[0, :, 5].cpu().double(), torch.from_numpy(c.ref.token(0, 95)[0]))
    assert (kb[1] == 5.0).all() and (kb[2, :, :7] == 0).all() and (kb[2, :, 7:39] == 0).all()
    assert torch.equal(vb[2, :, 39].cpu().double(), torch.from_numpy(c.ref.token(2, 32)[1]))


def run_attn(c, q, lens, nq, counts=None, causal=True, scale=None, max_length=None, fill=3.0, **kw):
    import torch
    import nystr_self_attention_gb300 as N
    out = torch.full_like(q, fill)
    N.nystrom_kv4_attn_fwd(c.dev, q, out, i32(lens), max(lens) if max_length is None else max_length,
                           None if counts is None else i32(counts), causal, scale, **kw)
    torch.cuda.synchronize()
    return out


def check(out, q, c, lens, dtype, counts=None, causal=True, scale=None, fill=3.0, name="", wide=False):
    want, A, S = C.attention(host(q), c.ref, lens, counts, causal, scale)
    tol = A * U * (160 * S + 160)
    if dtype == "bf16":
        tol = tol * (1 + HB) + (A * (2 if wide else 1) + np.abs(want)) * HB * (1 + 2 * HB)
    got = host(out)
    for b in range(q.shape[0]):
        n = q.shape[2] if counts is None else counts[b]
        assert (got[b, :, n:] == fill).all(), "rows behind the queries changed"
        err = np.abs(got[b, :, :n] - want[b, :, :n])
        assert (err <= tol[b, :, :n]).all(), \
            f"{name}: {np.nanmax(err / np.maximum(tol[b, :, :n], 1e-300)):.2f} of the bound"


ATTN = {
    # B, Hq, Hk, d, page, nq, lens, dtype
    "one_token": (1, 4, 2, 128, 64, 1, [200], "bf16"),
    "one_token_f32": (1, 4, 2, 128, 64, 1, [200], "f32"),
    "one_key": (2, 8, 8, 64, 16, 1, [1, 2], "bf16"),
    "ragged": (5, 8, 2, 128, 32, 1, [17, 0, 333, 64, 16], "bf16"),
    "ragged_f32": (5, 8, 2, 64, 16, 1, [17, 0, 333, 64, 15], "f32"),
    "d32": (2, 6, 3, 32, 48, 1, [95, 48], "bf16"),
    "d32_f32": (2, 6, 3, 32, 48, 3, [95, 48], "f32"),
    "seven_heads": (2, 14, 2, 64, 32, 1, [129, 31], "bf16"),
    "sixteen_rows": (1, 16, 1, 128, 64, 1, [300], "bf16"),
    "seventeen_rows": (1, 17, 1, 128, 64, 1, [300], "bf16"),
    "draft": (3, 6, 2, 64, 16, 5, [5, 100, 2], "bf16"),
    "draft_f32": (3, 6, 2, 64, 16, 5, [5, 100, 2], "f32"),
    "draft_d128": (2, 8, 2, 128, 16, 4, [130, 77], "bf16"),
    "forty_rows": (2, 8, 1, 128, 32, 5, [161, 40], "bf16"),
    "forty_rows_f32": (2, 8, 1, 128, 32, 5, [161, 40], "f32"),
    "chunk": (2, 4, 2, 128, 64, 100, [300, 100], "bf16"),
    "chunk_f32": (2, 4, 2, 128, 64, 67, [200, 67], "f32"),
    "chunk_d64": (2, 3, 1, 64, 16, 131, [260, 40], "bf16"),
    "chunk_d32": (1, 2, 2, 32, 16, 150, [260], "bf16"),
    "chunk_one_head": (1, 1, 1, 128, 128, 129, [129], "bf16"),
    "long": (1, 8, 2, 128, 128, 1, [5000], "bf16"),
    "long_f32": (1, 8, 2, 64, 128, 2, [5000], "f32"),
    "many_short": (40, 4, 4, 64, 16, 1, list(range(40)), "bf16"),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", ATTN)
def test_attention(name, causal):
    import nystr_self_attention_gb300 as N
    B, Hq, Hk, d, page, nq, lens, dtype = ATTN[name]
    c = Both(B, Hk, d, page, -(-max(lens) // page))
    c.fill(lens, dtype)
    q = heads(c.rng.standard_normal((B, Hq, nq, d)), dtype, "bnhd" if len(name) % 2 else "bhnd")
    out = run_attn(c, q, lens, nq, causal=causal)
    assert N.nystrom_get_status() == N.NYS_OK
    check(out, q, c, lens, dtype, causal=causal, name=name)
    assert np.array_equal(host(out), host(run_attn(c, q, lens, nq, causal=causal))), "two runs differ"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 6, 90])
def test_padded_queries_and_larger_bounds(nq, dtype):
    """q_counts below nq (0 among them), max_length far above the lengths."""
    lens = [70, 33, 0, 120]
    counts = [nq, nq // 2, nq, 0]
    c = Both(4, 2, 64, 16, 60)
    c.fill(lens, dtype)
    q = heads(c.rng.standard_normal((4, 6, nq, 64)), dtype, "bnhd")
    out = run_attn(c, q, lens, nq, counts, max_length=959)
    check(out, q, c, lens, dtype, counts)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 90])
def test_scores_far_apart_and_scales(nq, dtype):
    """Large scores that grow along the keys (the running maximum moves at
    every tile), values of very different sizes, a scale of the caller's."""
    import nystr_self_attention_gb300 as N
    B, Hk, d, n = 2, 2, 128, 260
    c = Both(B, Hk, d, 64, 5)
    k = c.rng.standard_normal((B, Hk, n, d)) * 0.1 + np.linspace(0, 2, n)[:, None]
    k[1] = k[1, :, ::-1]
    v = c.rng.standard_normal((B, Hk, n, d)) * np.exp2(c.rng.integers(-30, 30, (B, Hk, n, 1)))
    k, v = heads(k, dtype, "bhnd"), heads(v, dtype, "bhnd")
    N.nystrom_kv4_write(c.dev, k, v)
    c.ref.write(host(k), host(v), [0, 0], [n, n])
    q = heads(0.3 + 0.1 * c.rng.standard_normal((B, 4, nq, d)), dtype, "bhnd")
    for scale in (None, 0.5, -0.25):
        out = run_attn(c, q, [n, n], nq, scale=scale)
        check(out, q, c, [n, n], dtype, scale=scale, wide=nq > 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [2.0 ** -90, 1e-6, 1e6, 2.0 ** 60])
def test_query_and_value_ranges(size, dtype):
    """Tiny and huge queries (the scale makes up for them) and values."""
    import nystr_self_attention_gb300 as N
    c = Both(1, 1, 64, 16, 4)
    k, v = (c.rng.standard_normal((1, 1, 50, 64)) for _ in range(2))
    k, v = heads(k, dtype, "bhnd"), heads(v * size, dtype, "bhnd")
    N.nystrom_kv4_write(c.dev, k, v)
    c.ref.write(host(k), host(v), [0], [50])
    for nq in (1, 70):
        q = heads(c.rng.standard_normal((1, 2, nq, 64)) / size, dtype, "bhnd")
        out = run_attn(c, q, [50], nq, scale=float(np.float32(0.1 * size)), causal=False)
        check(out, q, c, [50], dtype, scale=float(np.float32(0.1 * size)), causal=False)


@pytest.mark.parametrize("nq", [1, 70])
def test_what_lies_past_the_length_has_no_say(nq):
    """The rest of the last block and page full of NaN scales, then of large
    ones: the same bits."""
    import torch
    lens = [70, 37]
    c = Both(2, 2, 128, 64, 2)
    c.fill(lens)
    q = heads(c.rng.standard_normal((2, 4, nq, 128)), "bf16", "bhnd")
    outs = []
    for junk in (0x00, 0xFF, 0x7F):
        raw = c.bytes().copy()
        keep = C.Cache(raw, c.table, 64, 2, 128)
        for b in range(2):
            for t in range(lens[b], 128):
                blk, r = keep.block(b, t), t % 16
                for at, bytes_of in ((0, keep.kb), (9 * 128, keep.vb)):
                    blk[:, at + bytes_of[r]] = junk
                    for y in range(4):
                        blk[:, at + 8 * 128 + (y * 16 + r) * 2:][:, :2] = junk
        c.data.copy_(torch.from_numpy(keep.raw.reshape(-1)))
        outs.append(host(run_attn(c, q, lens, nq)))
    assert np.isfinite(outs[0]).all()
    assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])
    check(torch.from_numpy(outs[0]), q, c, lens, "bf16")


@pytest.mark.parametrize("nq", [1, 70])
def test_nan_tokens_reach_only_those_who_see_them(nq):
    import nystr_self_attention_gb300 as N
    c = Both(2, 1, 64, 16, 6)
    k, v = (c.rng.standard_normal((2, 1, 90, 64)) for _ in range(2))
    k[0, 0, 80, 3], v[1, 0, 85, 40] = np.inf, np.nan
    k, v = heads(k, "bf16", "bhnd"), heads(v, "bf16", "bhnd")
    N.nystrom_kv4_write(c.dev, k, v)
    q = heads(c.rng.standard_normal((2, 2, nq, 64)), "bf16", "bhnd")
    got = host(run_attn(c, q, [90, 90], nq))
    first = [max(0, 80 - 90 + nq), max(0, 85 - 90 + nq)]  # first query that sees the token
    assert np.isnan(got[0, :, first[0]:]).all() and np.isfinite(got[0, :, :first[0]]).all()
    assert np.isnan(got[1, :, first[1]:, 32:]).all() and np.isfinite(got[1, :, :, :32]).all()
    assert np.isfinite(got[1, :, :first[1]]).all()


@pytest.mark.parametrize("nq", [1, 70])
def test_lengths_and_pages_out_of_range(nq):
    import torch
    import nystr_self_attention_gb300 as N
    c = Both(4, 2, 64, 32, 4)
    c.fill([128] * 4)
    c.table[2, 1] = -5
    c.table[3, 3] = 10 ** 6
    c.dtable.copy_(torch.from_numpy(c.table))
    c.ref.table = c.table
    q = heads(c.rng.standard_normal((4, 4, nq, 64)), "bf16", "bhnd")
    out = run_attn(c, q, [200, -4, 100, 128], nq, max_length=500)
    assert N.nystrom_get_status() == N.NYS_ERR_INDEX
    assert N.nystrom_get_status() == N.NYS_OK
    check(out, q, c, [128, 0, 100, 128], "bf16")


def test_shared_pages():
    """Two sequences whose first pages are the same memory (a shared prompt)."""
    import torch
    c = Both(2, 2, 64, 16, 6)
    c.table[1, :3] = c.table[0, :3]
    c.dtable.copy_(torch.from_numpy(c.table))
    c.ref.table = c.table
    c.fill([90, 0])
    q = heads(c.rng.standard_normal((2, 4, 2, 64)), "f32", "bhnd")
    out = run_attn(c, q, [90, 48], 2)
    check(out, q, c, [90, 48], "f32")


@pytest.mark.parametrize("nq", [1, 70])
def test_replayed_from_a_graph_with_longer_lengths(nq):
    """One captured call, its lengths and table read anew at every replay; an
    eager call on another stream at the same time with its own workspace."""
    import torch
    import nystr_self_attention_gb300 as N
    c = Both(3, 2, 128, 32, 40)
    c.fill([1200, 900, 1000])
    q = heads(c.rng.standard_normal((3, 8, nq, 128)), "bf16", "bhnd")
    out, lens = torch.empty_like(q), i32([100, 90, 80])
    step = lambda o, **kw: N.nystrom_kv4_attn_fwd(c.dev, q, o, lens, 1280, **kw)  # noqa: E731
    step(out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(out)
    for now in ([101, 91, 81], [1200, 0, 1000], [7, 900, 33]):
        lens.copy_(i32(now))
        side, other = torch.cuda.Stream(), torch.empty_like(q)
        side.wait_stream(torch.cuda.current_stream())
        g.replay()
        step(other, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, other)
        check(out, q, c, now, "bf16")


def test_caller_and_cached_workspaces_agree():
    import ctypes
    import torch
    import nystr_self_attention_gb300 as N
    c = Both(1, 2, 128, 64, 64)
    c.fill([4000])
    q = heads(c.rng.standard_normal((1, 8, 1, 128)), "bf16", "bhnd")
    need = N.nystrom_kv4_attn_workspace_bytes(c.dev, 1, 1, 8, 4096, N.NYS_BF16)
    ws = torch.full((max(need, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    a = run_attn(c, q, [4000], 1, max_length=4096, workspace=ws)
    b, lens, s = torch.empty_like(q), i32([4000]), N.NysStrides(0, 128, 0)

    def raw(stream):
        return N.load_library().nystrom_kv4_attn_fwd(
            c.dev.desc, q.data_ptr(), b.data_ptr(), ctypes.byref(s), ctypes.byref(s), lens.data_ptr(), None,
            1, 1, 8, 4096, 1, 0.0, N.NYS_BF16, None, 0, stream)

    assert raw(torch.cuda.current_stream().cuda_stream) == N.NYS_OK
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    if need:
        codes, g = [], torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            codes.append(raw(torch.cuda.current_stream().cuda_stream))
            b.zero_()
        assert codes == [N.NYS_ERR_ARG]


def test_norm_write_attend_and_read_back_into_nystrom_attention():
    """A prompt and two decoding steps as a model runs them: queries and keys
    normalised and rotated, keys and values written, attention over the cache;
    then the cached context read back as inputs of the forward pass. Against
    the oracle run on what each step hands to the next."""
    import torch
    import nystr_self_attention_gb300 as N
    from oracle import nystrom_ref as R
    B, Hq, Hk, d, n = 2, 4, 2, 64, 96
    c = Both(B, Hk, d, 32, 4)
    inv = 10000.0 ** (-np.arange(d // 2) * 2.0 / d)
    w = torch.rand(d, device="cuda") + 0.5
    at = 0
    for step in (n, 1, 1):
        qkv = torch.randn(B, step, Hq + 2 * Hk, d, device="cuda").to(torch.bfloat16)
        q, k, v = (t.transpose(1, 2) for t in qkv.split([Hq, Hk, Hk], dim=2))
        pos = (torch.arange(step, device="cuda", dtype=torch.int32) + at).expand(1, B, step).contiguous()
        ang = C.rope_angles(pos.cpu().numpy(), inv, [d // 2])
        want = C.qk_norm_rope(host(k), host(w), ang, False)
        N.nystrom_qk_norm_rope_fwd(q, k, q, k, pos, inv, w, w)  # in place, inside the projection
        assert np.abs(host(k) - want).max() <= 2 * HB * np.abs(want).max()
        starts = i32([at] * B)
        N.nystrom_kv4_write(c.dev, k, v, starts)
        c.ref.write(host(k), host(v), [at] * B, [step] * B)
        at += step
        out = run_attn(c, q, [at] * B, step, max_length=128)
        check(out, q, c, [at] * B, "bf16")
    assert np.array_equal(c.bytes(), c.ref.raw)
    K, V = (torch.empty(B, Hk, at, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    N.nystrom_kv4_read(c.dev, K, V)
    q = torch.randn(B, Hk, at, d, device="cuda").to(torch.bfloat16)
    y = N.nystrom_attention(q, K, V, None, 16, 6)
    torch.cuda.synchronize()
    assert N.nystrom_get_status() == N.NYS_OK
    ref = R.nystrom_attention(host(q), host(K), host(V), np.zeros((Hk, 1)), 16, 6)
    assert np.abs(host(y) - ref).max() <= 2e-2 * np.abs(ref).max()


RAGGED_CHUNKS = {
    # B, Hq, Hk, d, page, nq, lens, counts: several items, cut and whole, of one and two groups of rows
    "two_groups": (3, 8, 2, 128, 64, 70, [700, 130, 71], [70, 40, 70]),
    "more_queries_than_tokens": (2, 4, 1, 128, 16, 90, [30, 257], [90, 90]),
    "odd_heads": (2, 7, 1, 64, 32, 45, [385, 128], [45, 8]),
    "some_without_queries": (5, 4, 4, 64, 16, 60, [1, 0, 128, 129, 300], [60, 60, 0, 1, 33]),
    "one_long_many_short": (9, 2, 1, 128, 16, 130, [2600] + [5] * 8, [130] + [3] * 8),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", RAGGED_CHUNKS)
def test_ragged_chunks(name, causal):
    import nystr_self_attention_gb300 as N
    B, Hq, Hk, d, page, nq, lens, counts = RAGGED_CHUNKS[name]
    c = Both(B, Hk, d, page, -(-max(lens) // page))
    c.fill(lens)
    q = heads(c.rng.standard_normal((B, Hq, nq, d)), "bf16", "bnhd")
    out = run_attn(c, q, lens, nq, counts, causal=causal)
    assert N.nystrom_get_status() == N.NYS_OK
    check(out, q, c, lens, "bf16", counts, causal=causal, name=name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rep", [1, 12])
def test_many_ragged_sequences_share_the_line(rep, dtype):
    """Lengths from none to thousands, far fewer tokens than max_length allows:
    ranges that end in, on and between items."""
    import nystr_self_attention_gb300 as N
    lens = [0, 3000, 31, 32, 33, 0, 0, 1, 640, 1999, 5, 64, 900, 0, 127, 2, 2304, 16, 17, 0]
    c = Both(20, 3, 64, 16, 188)
    c.fill(lens, dtype)
    q = heads(c.rng.standard_normal((20, 3 * rep, 1, 64)), dtype, "bnhd")
    out = run_attn(c, q, lens, 1, max_length=3008)
    assert N.nystrom_get_status() == N.NYS_OK
    check(out, q, c, lens, dtype)


@pytest.mark.parametrize("B,Hk,lens,limits", [
    (1, 2, [1024], [1024, 1025]), (2, 2, [1025, 1023], [1025, 4000]),
    (16, 4, [2048, 2047, 1, 0] * 4, [2048, 2049]), (1, 1, [0], [0, 5000]),
])
def test_both_ways_of_planning_agree_with_the_oracle(B, Hk, lens, limits):
    """Limits on both sides of where a CTA per item gives way to ranges."""
    c = Both(B, Hk, 64, 64, max(1, -(-max(lens) // 64)))
    c.fill(lens)
    q = heads(c.rng.standard_normal((B, 2 * Hk, 1, 64)), "bf16", "bnhd")
    for limit in limits:
        check(run_attn(c, q, lens, 1, max_length=limit), q, c, lens, "bf16", name=f"limit {limit}")


@pytest.mark.parametrize("nq", [1, 60])
def test_no_tokens_at_all(nq):
    c = Both(2, 2, 64, 16, 4)
    q = heads(c.rng.standard_normal((2, 4, nq, 64)), "bf16", "bnhd")
    assert (run_attn(c, q, [0, 0], nq, max_length=0) == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 100])
def test_result_over_the_queries(nq, dtype):
    """out may be q: whole items and items that several CTAs share."""
    import torch
    import nystr_self_attention_gb300 as N
    lens = [1800, 40]
    c = Both(2, 2, 64, 32, 57)
    c.fill(lens, dtype)
    q = heads(c.rng.standard_normal((2, 6, nq, 64)), dtype, "bnhd")
    apart = run_attn(c, q, lens, nq)
    N.nystrom_kv4_attn_fwd(c.dev, q, q, i32(lens), 1800)
    assert torch.equal(apart, q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_read_of_any_bytes(d, dtype):
    """Memory that nothing was written to, so every kind of scale: subnormal,
    infinite, NaN. A code times a scale has at most 12 bits: one rounding."""
    import torch
    import nystr_self_attention_gb300 as N
    n = 16 * 24
    c = Both(2, 2, d, 64, 6)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    k, v = (torch.empty(2, n, 2, d, dtype=t, device="cuda").transpose(1, 2) for _ in range(2))
    N.nystrom_kv4_read(c.dev, k, v)
    for b in range(2):
        with np.errstate(invalid="ignore"):
            toks = [c.ref.token(b, i) for i in range(n)]
        for got, kind in ((k, 0), (v, 1)):
            with np.errstate(over="ignore", invalid="ignore"):
                want = torch.from_numpy(np.stack([x[kind] for x in toks], 1)).to(torch.float32).to(t)
            assert torch.equal(torch.nan_to_num(got[b].cpu().float(), nan=1.5),
                               torch.nan_to_num(want.float(), nan=1.5))


def test_a_cache_keeps_its_memory():
    """Its tensors cannot be swapped under the addresses that it hands out."""
    c = Both(1, 1, 32, 16, 2)
    for name in ("data", "block_table"):
        with pytest.raises(AttributeError):
            setattr(c.dev, name, c.data)
    assert c.dev.data is c.data and c.dev.block_table is c.dtable


def test_workspaces_of_calls_one_after_another_and_side_by_side():
    """Calls of growing and shrinking needs on the default stream, whose
    workspace they share, with others on a second stream meanwhile."""
    import torch
    import nystr_self_attention_gb300 as N
    cases, side = [], torch.cuda.Stream()
    for i, (B, Hq, nq, n, dtype) in enumerate([(1, 8, 1, 1500, "f32"), (4, 8, 90, 1500, "bf16"),
                                               (2, 16, 2, 1200, "bf16"), (3, 8, 3, 1400, "f32")]):
        c = Both(B, 4, 64, 64, 24, seed=i)
        k, v = (heads(c.rng.standard_normal((B, 4, n, 64)), dtype, "bnhd") for _ in range(2))
        N.nystrom_kv4_write(c.dev, k, v)
        q = heads(c.rng.standard_normal((B, Hq, nq, 64)), dtype, "bnhd")
        lens = [n - 7 * b for b in range(B)]
        need = N.nystrom_kv4_attn_workspace_bytes(c.dev, B, nq, Hq, n, N.NYS_BF16 if dtype == "bf16" else N.NYS_FP32)
        assert need > 0
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        cases.append((c, q, i32(lens), n, run_attn(c, q, lens, nq, max_length=n, workspace=ws)))
    torch.cuda.synchronize()
    assert torch.cuda.current_stream().cuda_stream == 0
    for _ in range(5):
        outs = []
        for j, (c, q, lens, n, want) in enumerate(cases):
            o = torch.empty_like(q)
            N.nystrom_kv4_attn_fwd(c.dev, q, o, lens, n)
            c2, q2, lens2, n2, want2 = cases[-1 - j]
            p = torch.empty_like(q2)
            with torch.cuda.stream(side):
                N.nystrom_kv4_attn_fwd(c2.dev, q2, p, lens2, n2)
            outs += [(o, want), (p, want2)]
        torch.cuda.synchronize()
        for got, want in outs:
            assert torch.equal(got, want)
