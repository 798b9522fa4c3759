"""Shared by the GPU tests of the operators around the attention module."""
import numpy as np

U, HB = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and of bf16, relative
HALF = {"bf16": HB, "f32": U}
ACTS = ["silu", "gelu", "gelu_tanh", "relu"]


def tdtype(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def upload(x, dtype, pad=0):
    """Device [rows, width] matrix of a host array; pad: elements between its rows."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(tdtype(dtype)).cuda()
    if not pad:
        return t
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def empty(rows, width, dtype, pad=0):
    import torch
    return torch.full((rows, width + pad), 7.0, dtype=tdtype(dtype), device="cuda")[:, :width]


def host(t):
    return t.detach().double().cpu().numpy()


def eight(N, rows, K, pad=0):
    """An empty 8-bit matrix whose memory holds something."""
    import torch
    codes = torch.full((rows, K + pad), 0x35, dtype=torch.uint8, device="cuda")[:, :K]
    return N.NystromQ8(codes, torch.full((-(-K // 512), rows), -1, dtype=torch.int32, device="cuda"))


def upload_eight(N, codes, words, pad=0):
    import torch
    q = eight(N, *codes.shape, pad)
    q.codes.copy_(torch.from_numpy(np.ascontiguousarray(codes)))
    q.scales.copy_(torch.from_numpy(np.ascontiguousarray(words)))
    return q


def untouched(t, width):
    """Whether what lies between a padded matrix's rows is as `empty` left it."""
    import torch
    base = torch.as_strided(t, (t.shape[0], t.stride(0)), (t.stride(0), 1))
    return bool((base[:-1, width:] == 7).all())


def act_code(N, name):
    return {"silu": N.NYS_ACT_SILU, "gelu": N.NYS_ACT_GELU, "gelu_tanh": N.NYS_ACT_GELU_TANH,
            "relu": N.NYS_ACT_RELU}[name]


def own_status(N):
    """A forward pass in the library's own workspace: nystrom_get_status reads the
    last one's status word, and a workspace that an earlier test gave may be gone."""
    import torch
    q = torch.zeros(1, 1, 64, 32, dtype=torch.bfloat16, device="cuda")
    N.nystrom_attention(q, q, q, None, 8, 2)
    torch.cuda.synchronize()
    N.nystrom_get_status()


def done(N):
    import torch
    torch.cuda.synchronize()
    assert N.nystrom_get_status() == N.NYS_OK
