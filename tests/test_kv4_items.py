"""Chunks of queries over the 4-bit cache whose CTAs walk several items: ranges
of many key tiles, cut and whole items, items of one group of 128 query rows
before and behind items of two. Every row against plain attention in 64 bits
over what the cache reads back (which its own tests hold bit for bit).

Bound per element, with u = 2^-24, A = sum p |v| and S the largest sum |q k| scale
of the row's keys: scores and sums in fp32 A u (160 S + 160); a code times a scale
has at most 7 x 255 < 2^11, 11 bits, which fp16 holds; probabilities are rounded
to 16-bit floats (at most bf16: 2^-8 of each, A 2^-8) and the result to bf16
(2^-8 of itself)."""
import numpy as np
import pytest

U, HB = 2.0 ** -24, 2.0 ** -8
TILE, ROWS, GROUP, COST = 128, 256, 128, 2  # keys of a tile, rows of an item, of a group, places of its start


def segments(lens, counts, nq, rep, Hk, causal, ctas):
    """(tiles that some row sees, groups of rows) of the segments that each CTA
    walks: the items' key tiles in one line, cut evenly."""
    items, at = [], 0
    row_tiles = -(-nq * rep // ROWS)
    for n, c in zip(lens, counts):
        tiles = -(-n // TILE)
        for i in range(Hk * row_tiles if tiles else 0):
            rows = min(ROWS, c * rep - i % row_tiles * ROWS)
            seen = n if not causal else max(0, n - c + 1 + (i % row_tiles * ROWS + rows - 1) // rep)
            items.append((at + COST, tiles, 0 if rows <= 0 else seen, 2 if rows > GROUP else 1))
            at += COST + tiles
    per = max(-(-at // ctas), 1)
    out = []
    for r0 in range(0, at, per):
        walk = []
        for first, tiles, seen, groups in items:
            lo, hi = max(first, r0), min(first + tiles, r0 + per)
            if lo < hi:
                walk.append((max(0, min(hi - first, -(-seen // TILE)) - (lo - first)), groups))
        out.append(walk)
    return out


def skips_then_works(walk, tiles=4):
    """A one-group segment of some length with a two-group one behind it."""
    return any(g == 1 and t >= tiles and any(g2 == 2 and t2 > 0 for t2, g2 in walk[i + 1:])
               for i, (t, g) in enumerate(walk))


CASES = {
    # B, Hq, Hk, d, page, nq, lens, counts
    "tails_of_88_rows": (8, 16, 8, 128, 64, 300, [4096] * 8, [300] * 8),
    "tails_of_44_rows": (8, 32, 8, 128, 128, 75, [4096] * 8, [75] * 8),
    "tails_of_32_rows_d64": (4, 32, 8, 64, 32, 200, [8192] * 4, [200] * 4),
    "mixed_counts": (6, 16, 4, 128, 64, 200, [9000, 7000, 8000, 9001, 5500, 64], [200, 30, 1, 120, 20, 60]),
    "short_chunks_first": (28, 8, 8, 128, 64, 400, [1500, 2900, 700, 2900] * 7, [100, 400, 7, 300] * 7),
    "odd_everything_d64": (9, 21, 3, 64, 16, 55, [5001, 4999, 6000, 128, 7333, 0, 3001, 6789, 901],
                           [55, 19, 41, 55, 18, 55, 0, 38, 55]),
}


@pytest.mark.parametrize("name", CASES)
def test_the_cases_have_the_arrangement(name):
    B, Hq, Hk, d, page, nq, lens, counts = CASES[name]
    walks = segments(lens, counts, nq, Hq // Hk, Hk, True, 152)
    assert len(walks) <= 152 and any(skips_then_works(w) for w in walks)


def attention(q, k, v, n, count, causal, scale):
    """q [Hq, count, d], k, v [Hk, n, d] in 64 bits: result, sum p |v| and the
    largest sum |q k| scale per row."""
    import torch
    if n == 0 or count == 0:
        return torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q[..., :1])
    rep = q.shape[0] // k.shape[0]
    k, v = k[:, :n].repeat_interleave(rep, 0), v[:, :n].repeat_interleave(rep, 0)
    s = q @ k.transpose(1, 2) * scale
    reach = q.abs() @ k.abs().transpose(1, 2) * abs(scale)
    if causal:
        i, j = torch.arange(count, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
        hidden = j > n - count + i
        s, reach = s.masked_fill(hidden, -np.inf), reach.masked_fill(hidden, 0)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -np.inf, 0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1, total)
    return p @ v, p @ v.abs(), reach.amax(-1, keepdim=True)


def filled(B, Hk, d, page, lens, seed, k_size=None, v_size=None):
    """A cache with pages in no order, and what it reads back in 64 bits."""
    import torch
    import nystr_self_attention_gb300 as N
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, per = max(lens), -(-max(lens) // page)
    data = torch.zeros(N.nystrom_kv4_cache_bytes(B * per, page, Hk, d), dtype=torch.uint8, device="cuda")
    table = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
    cache = N.NystromKv4Cache(data, table, page, Hk, d)
    k, v = (torch.randn(B, Hk, n, d, generator=g, device="cuda") for _ in range(2))
    if k_size is not None:
        k *= k_size
    if v_size is not None:
        v *= v_size
    N.nystrom_kv4_write(cache, k, v)
    N.nystrom_kv4_read(cache, k, v)
    return cache, k.double(), v.double(), g


def compare(out, q, k, v, lens, counts, causal, scale=None, name=""):
    import torch
    scale = q.shape[3] ** -0.5 if scale is None else scale
    for b, (n, c) in enumerate(zip(lens, counts)):
        want, A, S = attention(q[b, :, :c].double(), k[b], v[b], n, c, causal, scale)
        tol = A * U * (160 * S + 160) * (1 + HB) + (A + want.abs()) * HB * (1 + 2 * HB)
        err = (out[b, :, :c].double() - want).abs()
        assert torch.isfinite(err).all()
        assert (err <= tol).all(), f"{name} sequence {b}: {(err / tol.clamp(min=1e-300)).max():.2f} of the bound"
        assert (out[b, :, c:] == 3.0).all(), "rows behind the queries changed"


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", CASES)
def test_items_of_one_and_two_groups_in_one_range(name, causal):
    import torch
    import nystr_self_attention_gb300 as N
    B, Hq, Hk, d, page, nq, lens, counts = CASES[name]
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    assert any(skips_then_works(w) for w in segments(lens, counts, nq, Hq // Hk, Hk, causal, ctas))
    cache, k, v, g = filled(B, Hk, d, page, lens, seed=3)
    q = torch.randn(B, nq, Hq, d, generator=g, device="cuda").to(torch.bfloat16).transpose(1, 2)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    outs = []
    for _ in range(2):
        out = torch.full_like(q, 3.0)
        N.nystrom_kv4_attn_fwd(cache, q, out, i32(lens), max(lens), i32(counts), causal)
        assert N.nystrom_get_status() == N.NYS_OK
        outs.append(out)
    compare(outs[0], q, k, v, lens, counts, causal, name=name)
    assert torch.equal(outs[0], outs[1]), "two runs differ"


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["tails_of_88_rows", "mixed_counts"])
@pytest.mark.parametrize("few", [False, True])
def test_result_over_the_queries_of_many_items(name, few):
    """out may be q where CTAs go from item to item; `few`: the kernel for calls
    of few query rows as well."""
    import torch
    import nystr_self_attention_gb300 as N
    B, Hq, Hk, d, page, nq, lens, counts = CASES[name]
    if few:
        nq, counts = 5, [min(c, 5) for c in counts]
    cache, _, _, g = filled(B, Hk, d, page, lens, seed=4)
    q = torch.randn(B, nq, Hq, d, generator=g, device="cuda").to(torch.bfloat16).transpose(1, 2)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    apart = q.clone()
    N.nystrom_kv4_attn_fwd(cache, q, apart, i32(lens), max(lens), i32(counts))
    N.nystrom_kv4_attn_fwd(cache, q, q, i32(lens), max(lens), i32(counts))
    assert N.nystrom_get_status() == N.NYS_OK
    assert torch.equal(apart, q)
