"""Sums over a million elements and more, all of one sign, with bf16 results. The
matrix units cut sums off towards zero, so what a sum that stays there loses grows
with its length and does not average out over the results, as rounding does.

Operands repeat themselves along the sum with a period of 4096, so that a product of
that length in 64 bits, times the repetitions, is the exact result. At most 1024
instructions are summed by the unit, each cut off by at most 2^-23 of the sum, and
the up to 64 sums of those are rounded at 2^-24: 2^-13 + 2^-18 in all. Results lie
within that and a rounding of the exact ones, and so does their mean error, less the
mean error of the exact results rounded: that is not 0, since results lie about a
power of two, below which steps are half as long (-1.2e-4 for the forward products
here, in 64 bits). A result next to a border may round the other way, which leaves of
the mean at most a step, 2^-8, over the root of the number of columns (the rows may be
alike)."""
import pytest

from layer_helpers import HB, done, own_status

pytestmark = pytest.mark.gpu
PERIOD = 4096


@pytest.fixture(scope="module", autouse=True)
def library():
    import torch
    from nystr_self_attention_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    import nystr_self_attention_gb300 as N
    own_status(N)
    yield
    torch.cuda.empty_cache()


def positive(*shape):
    """bf16 values of 0.5 to 1.5."""
    import torch
    return (torch.rand(*shape, device="cuda") + 0.5).to(torch.bfloat16)


def check(got, want):
    import torch
    off = (got.double() - want) / want
    rounding = (want.to(torch.bfloat16).double() - want) / want
    cut = 2.0 ** -13 + 2.0 ** -18
    assert float(off.abs().max()) <= HB + cut * (1 + HB)
    assert abs(float((off - rounding).mean())) <= cut + HB / got.shape[1] ** 0.5


def test_weight_gradients():
    """2^20 tokens; sizes whose tiles fill the GPU, so that time asks for no split of
    the tokens. g, u and gh are one row for all tokens: dg = u, du = g."""
    import torch
    import nystr_self_attention_gb300 as N
    torch.manual_seed(1)
    T, d, f = 1 << 20, 4864, 512
    some, g, u = positive(PERIOD, d), positive(1, f), positive(1, f)
    x = some.repeat(T // PERIOD, 1)
    rows = [t.expand(T, f) for t in (g, u, torch.ones_like(g))]
    w = torch.zeros(d, f, dtype=torch.bfloat16, device="cuda")
    dwg, dwu = torch.empty_like(w), torch.empty_like(w)
    N.nystrom_gated_ff_bwd(x, w, w, *rows, None, dwg, dwu, activation=N.NYS_ACT_RELU)
    done(N)
    total = some.double().sum(0)[:, None] * (T // PERIOD)
    check(dwg, total * u.double())
    check(dwu, total * g.double())


@pytest.mark.parametrize("T,f", [(1024, 2432), (16, 9728)])
def test_forward(T, f):
    import torch
    import nystr_self_attention_gb300 as N
    torch.manual_seed(2)
    d = 1 << 19
    some, wg, wu = positive(T, PERIOD), positive(PERIOD, f), positive(PERIOD, f)
    times = d // PERIOD
    h, g, u = (torch.empty(T, f, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    N.nystrom_gated_ff_fwd(some.repeat(1, times), wg.repeat(times, 1), wu.repeat(times, 1), h, g, u,
                           activation=N.NYS_ACT_RELU)
    done(N)
    check(g, some.double() @ wg.double() * times)
    check(u, some.double() @ wu.double() * times)


@pytest.mark.parametrize("T", [1024, 16])
def test_input_gradient(T):
    """K is twice the features: dg = u, du = g of one row for all tokens."""
    import torch
    import nystr_self_attention_gb300 as N
    torch.manual_seed(3)
    d, f = 4864 if T > 128 else 9728, 1 << 18
    times = f // PERIOD
    g, u, wg, wu = positive(1, PERIOD), positive(1, PERIOD), positive(d, PERIOD), positive(d, PERIOD)
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    rows = [t.repeat(1, times).expand(T, f) for t in (g, u, torch.ones_like(g))]
    dx = torch.empty_like(x)
    N.nystrom_gated_ff_bwd(x, wg.repeat(1, times), wu.repeat(1, times), *rows, dx, activation=N.NYS_ACT_RELU)
    done(N)
    want = (u.double() @ wg.double().T + g.double() @ wu.double().T) * times
    check(dx, want.expand(T, d))


@pytest.mark.parametrize("T,n", [(1024, 4256), (16, 9728)])
def test_eight_bits(T, n):
    """Codes of 1 to 15 eighths, one scale."""
    import torch
    import nystr_self_attention_gb300 as N
    torch.manual_seed(4)
    K = 1 << 20

    def some(rows):
        codes = torch.randint(0x38, 0x40, (rows, PERIOD), dtype=torch.uint8, device="cuda")
        scales = torch.full((K // 512, rows), 0x7f7f7f7f, dtype=torch.int32, device="cuda")
        return codes.view(torch.float8_e4m3fn).double(), N.NystromQ8(codes.repeat(1, K // PERIOD), scales)
    (av, a), (wv, w) = some(T), some(n)
    out = torch.empty(T, n, dtype=torch.bfloat16, device="cuda")
    N.nystrom_q8_matmul(a, w, out)
    done(N)
    check(out, av @ wv.T * (K // PERIOD))
