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
