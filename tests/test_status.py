"""nystrom_get_status and workspaces that the caller gave and took back."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    import torch
    from nystr_self_attention_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)


@pytest.mark.parametrize("clustered", [False, True])
def test_a_workspace_is_the_caller_s_again_behind_the_call(clustered):
    """Its memory may hold anything by the time the status is read, and is left alone."""
    import torch
    import nystr_self_attention_gb300 as N
    q = torch.randn(1, 2, 256, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    if clustered:
        need = N.nystrom_clustered_workspace_bytes(1, 2, 256, 64, 32, N.NYS_BF16)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        N.nystrom_clustered_attn_fwd(q, q, q, out, 1, 2, 256, 64, 32, 2, N.NYS_BF16, ws, need)
    else:
        need = N.nystrom_attn_workspace_bytes(1, 2, 256, 64, 32, N.NYS_BF16)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        N.nystrom_attn_fwd_ws(q, q, q, None, out, 1, 2, 256, 64, 32, 6, 0, N.NYS_BF16, ws, need)
    torch.cuda.synchronize()
    ws.fill_(0xF9)
    torch.cuda.synchronize()
    assert N.nystrom_get_status() == N.NYS_OK
    assert bool((ws == 0xF9).all())


FIRST = """
import torch
import nystr_self_attention_gb300 as N
torch.cuda.set_device(0)
q = torch.randn(1, 2, 256, 64, dtype=torch.bfloat16, device="cuda")
out = torch.empty_like(q)
need = N.nystrom_attn_workspace_bytes(1, 2, 256, 64, 32, N.NYS_BF16)
ws = torch.empty(need, dtype=torch.uint8, device="cuda")
def call():
    N.nystrom_attn_fwd_ws(q, q, q, None, out, 1, 2, 256, 64, 32, 6, 0, N.NYS_BF16, ws, need)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    call()
g.replay()
torch.cuda.synchronize()
got = out.clone()
call()
torch.cuda.synchronize()
assert torch.equal(got, out) and N.nystrom_get_status() == 0
"""


def test_a_process_s_first_forward_call_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
