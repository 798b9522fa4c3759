"""Outputs of the operators around a cached attention layer that share memory
with one another, or with an input whose rows lie elsewhere in it: refused, and
nothing is written."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

INV = 10000.0 ** (-np.arange(32) / 32)


@pytest.fixture(scope="module", autouse=True)
def library():
    import torch
    from nystr_self_attention_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)


def heads(n=2):
    """Views [2, 4, 6, 64]: as they lie, and the same memory taken token by token."""
    import torch
    x = [torch.randn(2, 4, 6, 64, device="cuda") for _ in range(n)]
    return x, [t.view(2, 6, 4, 64).transpose(1, 2) for t in x]


def refused(call, *unchanged):
    import torch
    import nystr_self_attention_gb300 as N
    before = [t.clone() for t in unchanged]
    with pytest.raises(N.NystromError) as e:
        call()
    assert e.value.code == N.NYS_ERR_ARG
    torch.cuda.synchronize()
    assert all(torch.equal(t, t0) for t, t0 in zip(unchanged, before))


def test_norm_and_rotation():
    import torch
    import nystr_self_attention_gb300 as N
    (q, k), (qt, kt) = heads()
    o = torch.empty_like(q)
    for q_out, k_out in ((o, o), (k, o), (o, q), (qt, o), (o, kt), (k, q)):
        refused(lambda: N.nystrom_qk_norm_rope_fwd(q, k, q_out, k_out, None, INV), q, k)
    N.nystrom_qk_norm_rope_fwd(q, k, q, k, None, INV)


def test_gradients():
    import torch
    import nystr_self_attention_gb300 as N
    (q, k, gq, gk), (_, _, gqt, gkt) = heads(4)
    o, dw = torch.empty_like(q), torch.zeros(64, device="cuda")

    def call(dq, dk, dqw=None, dkw=None):
        N.nystrom_qk_norm_rope_bwd(q, k, gq, gk, dq, dk, None, INV, None, None, dqw, dkw)
    for dq, dk in ((o, o), (gk, o), (o, gq), (gqt, o), (o, gkt)):
        refused(lambda: call(dq, dk), gq, gk)
    refused(lambda: call(gq, gk, dw, dw), gq, gk, dw)
    call(gq, gk, dw, torch.empty_like(dw))


@pytest.mark.parametrize("nq", [6, 60])
def test_cache(nq):
    import torch
    import nystr_self_attention_gb300 as N
    B, Hk, d, n = 2, 2, 64, 96
    data = torch.zeros(N.nystrom_kv4_cache_bytes(B * 3, 32, Hk, d), dtype=torch.uint8, device="cuda")
    cache = N.NystromKv4Cache(data, torch.arange(B * 3, dtype=torch.int32, device="cuda").view(B, 3), 32, Hk, d)
    k = torch.randn(B, Hk, n, d, device="cuda").to(torch.bfloat16)
    N.nystrom_kv4_write(cache, k, k)
    refused(lambda: N.nystrom_kv4_read(cache, k, k), k)
    q = torch.randn(B, 4, nq, d, device="cuda").to(torch.bfloat16)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    refused(lambda: N.nystrom_kv4_attn_fwd(cache, q, q.view(B, nq, 4, d).transpose(1, 2), lens, n), q)
    N.nystrom_kv4_attn_fwd(cache, q, q, lens, n)
    assert N.nystrom_get_status() == N.NYS_OK


def test_one_entry_has_no_stride():
    """One sequence, one head or one token: any stride there is the same."""
    import torch
    import nystr_self_attention_gb300 as N
    q = torch.randn(1, 1, 6, 64, device="cuda")
    want = torch.empty_like(q)
    N.nystrom_qk_norm_rope_fwd(q, None, want, None, None, INV)
    N.nystrom_qk_norm_rope_fwd(q, None, q.view(1, 6, 1, 64).transpose(1, 2), None, None, INV)
    assert torch.equal(q, want)
