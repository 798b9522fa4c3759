"""Attention over the 4-bit cache where keys, values or weights of very different
sizes meet in one tile, for calls of few query rows and of many, against plain
attention in 64 bits over what the cache reads back.

The bound is that of tests/test_kv4_items.py with one refinement: S, the largest
sum |q k| scale, is taken over the keys whose weight is at least e^-40 of the
row's largest even if their score is off by 160 u of that sum. A key's score
feels only its own sum's rounding, and 65537 keys below e^-40 add up to less than
2^-41, a fraction 2^-33 of A's least rounding, if values lie within 2^30.

Calls of many query rows hold keys as fp16 times a power of two that brings the
largest scale of 32 tokens to 2^12 .. 2^13: scales down to 2^-17 (2^-29 of the
largest) lose nothing, a key of a smaller one is rounded to multiples of 2^-24,
so it is off by at most 2^-25, which is 2^-37 of the largest scale. A score is
then off by that times sum |q| scale, a weight by twice it (`lost`)."""
import numpy as np
import pytest

from tests.test_kv4_items import HB, U, filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    import torch
    from nystr_self_attention_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)


def lost(k, q, scale):
    """Bound of what a row's scores lose where key scales span more than 2^29."""
    scales = k.unflatten(3, (-1, 32)).abs().amax(-1).flatten(2) / 7  # the largest code is 7 or -7
    top, least = scales.amax(-1), scales.amin(-1)
    far = (q.shape[2] > 48) * (top > least * 2.0 ** 29)
    return (far * top * 2.0 ** -37)[:, :, None, None] * q.abs().sum(-1, keepdim=True) * scale


def attend(q, cache, k, v, n, causal=True, scale=None, name=""):
    """All sequences n tokens long; q, k, v [B, H, ., d] with one query head per
    cache head."""
    import torch
    import nystr_self_attention_gb300 as N
    B, H, nq, d = q.shape
    out, lens = torch.empty_like(q), torch.full((B,), n, dtype=torch.int32, device="cuda")
    N.nystrom_kv4_attn_fwd(cache, q, out, lens, n, None, causal, scale)
    assert N.nystrom_get_status() == N.NYS_OK
    scale = d ** -0.5 if scale is None else scale
    x = q.double()
    s, reach = x @ k.transpose(2, 3) * scale, x.abs() @ k.abs().transpose(2, 3) * scale
    if causal:
        i, j = torch.arange(nq, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
        s = s.masked_fill(j > n - nq + i, -np.inf)
    top = s.amax(-1, keepdim=True)
    S = reach.masked_fill(s + 160 * U * reach < top - 40, 0).amax(-1, keepdim=True)
    p = torch.softmax(s, -1)
    want, A = p @ v, p @ v.abs()
    tol = A * (U * (160 * S + 160) + 2 * lost(k, x, scale)) * (1 + HB) + (A + want.abs()) * HB * (1 + 2 * HB)
    err = (out.double() - want).abs()
    assert torch.isfinite(err).all()
    assert (err <= tol).all(), f"{name}: {(err / tol.clamp(min=1e-300)).max():.2f} of the bound"


ROWS = [10, 100]  # on either side of where a call's kernel changes


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("span", [8, 12, 16, 20, 24])
@pytest.mark.parametrize("nq", ROWS)
def test_key_sizes_between_groups_of_channels(nq, span, d):
    """The first 32 channels of every key 2^span larger, of every query 2^span
    smaller: both parts of a score count alike."""
    import torch
    size = torch.ones(d, device="cuda")
    size[:32] = 2.0 ** span
    cache, k, v, g = filled(2, 2, d, 64, [700, 700], seed=span, k_size=size)
    q = (torch.randn(2, 2, nq, d, generator=g, device="cuda") * 2 / size).to(torch.bfloat16)
    attend(q, cache, k, v, 700, name=f"span {span}")


@pytest.mark.parametrize("span", [8, 12, 16, 20, 24, 28])
@pytest.mark.parametrize("nq", ROWS)
def test_queries_of_small_keys_beside_large_ones(nq, span):
    """Keys large in channels where the queries are zero, and tokens large
    where every query scores them far down: neither has a say."""
    import torch
    d, n = 128, 500
    size = torch.ones(1, 2, n, d, device="cuda")
    size[:, 0, :, :32] = 2.0 ** span
    size[:, 1, ::7] = 2.0 ** span
    cache, k, v, g = filled(1, 2, d, 64, [n], seed=span)
    q = torch.randn(1, 2, nq, d, generator=g, device="cuda") * 2
    x = torch.randn(1, 2, n, d, generator=g, device="cuda")
    q[:, 0, :, :32] = 0
    q[:, 1, :, 0] = 3
    x[:, 1, ::7] *= 0.01  # along -channel 0, so that these score about -3 x 2^span
    x[:, 1, ::7, 0] = -7
    import nystr_self_attention_gb300 as N
    back = torch.empty_like(x)
    N.nystrom_kv4_write(cache, x * size, v.float())
    N.nystrom_kv4_read(cache, back, torch.empty_like(x))
    attend(q.to(torch.bfloat16), cache, back.double(), v, n, name=f"span {span}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("span", [4, 6, 8, 9, 12, 20, 28, 40])
@pytest.mark.parametrize("nq", ROWS)
def test_value_sizes_between_groups_of_channels(nq, span, d):
    import torch
    size = torch.ones(d, device="cuda")
    size[32:] = 2.0 ** -span
    cache, k, v, g = filled(2, 2, d, 64, [700, 700], seed=span, v_size=size)
    q = torch.randn(2, 2, nq, d, generator=g, device="cuda").to(torch.bfloat16)
    attend(q, cache, k, v, 700, name=f"span {span}")


@pytest.mark.parametrize("span", [6, 12, 18, 24])
@pytest.mark.parametrize("nq", ROWS)
def test_values_of_blocks_far_apart(nq, span):
    """32 tokens whose first channels' values are 2^span larger and whose others
    are zero: there the rest of the context has the word alone."""
    import torch
    d, n = 128, 900
    size = torch.ones(n, d, device="cuda")
    size[96:128, :32] = 2.0 ** span
    size[96:128, 32:] = 0
    cache, k, v, g = filled(2, 2, d, 64, [n, n], seed=span, v_size=size)
    q = torch.randn(2, 2, nq, d, generator=g, device="cuda").to(torch.bfloat16)
    attend(q, cache, k, v, n, name=f"span {span}")


@pytest.mark.parametrize("tail", [65536, 3000])
@pytest.mark.parametrize("bits", [8.0, 16.3, 20.0, 22.9, 25.1])
@pytest.mark.parametrize("own", [0.0, 2.0 ** -20, 2.0 ** -7])
@pytest.mark.parametrize("nq", ROWS)
def test_a_dominant_key_and_a_long_even_tail(nq, own, bits, tail):
    """One key 2^bits above all others, which weigh alike; its values are near
    zero, so that the tail's mean is most of the result."""
    import torch
    import nystr_self_attention_gb300 as N
    d, n = 128, tail + 1
    cache, k, v, g = filled(1, 1, d, 128, [n], seed=int(bits))
    at = n // 3
    x = torch.zeros(1, 1, n, d, device="cuda")
    x[:, :, at, :32] = 1
    y = v.float() * 0.25 + 1
    y[:, :, at] *= own
    N.nystrom_kv4_write(cache, x, y)
    N.nystrom_kv4_read(cache, x, y)
    q = torch.randn(1, 1, nq, d, generator=g, device="cuda")
    q[..., :32] = bits * np.log(2.0) * d ** 0.5 / 32
    attend(q.to(torch.bfloat16), cache, x.double(), y.double(), n, causal=False, name=f"2^-{bits}")


@pytest.mark.parametrize("n", [2, 3, 12, 30, 500])
@pytest.mark.parametrize("nq", [20, 100])
def test_weights_far_below_the_largest(nq, n):
    """Scores tens apart: where the heaviest key's code is zero, a channel is the
    sum of keys of far smaller weight. With more than 48 rows a weight times the
    largest scale s of its 32 tokens is off by at most 2^-36 of the row's largest
    such product x <= s, and an element is at most 8 s: n 2^-36 8 s beside the
    bound, s at most twice (a power of two is kept) the largest |v| / 7."""
    import torch
    import nystr_self_attention_gb300 as N
    B, H, d = 4, 4, 128
    cache, k, v, g = filled(B, H, d, 64, [n] * B, seed=n)
    q = torch.randn(B, H, nq, d, generator=g, device="cuda").to(torch.bfloat16)
    out, lens = torch.empty_like(q), torch.full((B,), n, dtype=torch.int32, device="cuda")
    N.nystrom_kv4_attn_fwd(cache, q, out, lens, n, None, False, 0.3)
    assert N.nystrom_get_status() == N.NYS_OK
    scale, x = float(np.float32(0.3)), q.double()
    s, reach = x @ k.transpose(2, 3) * scale, x.abs() @ k.abs().transpose(2, 3) * scale
    p = torch.softmax(s, -1)
    want, A = p @ v, p @ v.abs()
    tol = A * U * (160 * reach.amax(-1, keepdim=True) + 160) * (1 + HB) + (A + want.abs()) * HB * (1 + 2 * HB)
    if nq > 48:
        tol += n * 2.0 ** -36 * 8 * 2 * v.abs().max() / 7
    err = (out.double() - want).abs()
    assert (err <= tol).all(), f"{(err / tol.clamp(min=1e-300)).max():.2f} of the bound"
