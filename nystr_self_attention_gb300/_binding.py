"""ctypes binding of libnystrom.so: same names as the C ABI
(include/nystrom.h), argument marshalling only. Every step of the forward
pass runs in the library's CUDA kernels; there is no Python or CPU path, and
calling without the built library raises."""
from __future__ import annotations

import ctypes
import os
import struct
import threading

NYS_FP32, NYS_BF16 = 0, 1
NYS_OK, NYS_ERR_ARG, NYS_ERR_SHAPE, NYS_ERR_ALIGN = 0, -1, -2, -3
NYS_ERR_UNSUPPORTED, NYS_ERR_NOMEM, NYS_ERR_CUDA, NYS_ERR_TIMEOUT = -4, -5, -6, -7
NYS_ERR_INDEX = -8
NYS_ROPE_HALVES, NYS_ROPE_PAIRS = 0, 1
NYS_STAGE_Q_TILDE, NYS_STAGE_K_TILDE, NYS_STAGE_G, NYS_STAGE_A_S, NYS_STAGE_W, NYS_STAGE_Z = range(6)
NYS_CONV_PER_HEAD, NYS_CONV_PER_CHANNEL = 0, 1
NYS_CSTAGE_ASSIGN, NYS_CSTAGE_CENTROIDS_PREV, NYS_CSTAGE_CENTROIDS, NYS_CSTAGE_G = range(4)

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnystrom.so")
_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int


class NysStrides(ctypes.Structure):
    """nys_strides_t: distances between rows, in elements."""
    _fields_ = [("batch", ctypes.c_longlong), ("head", ctypes.c_longlong), ("token", ctypes.c_longlong)]


class NysQkRope(ctypes.Structure):
    """nys_qk_rope_t."""
    _fields_ = [("B", _I), ("n", _I), ("Hq", _I), ("Hk", _I), ("d", _I), ("rot", _I), ("axes", _I),
                ("section", _I * 4), ("pairing", _I), ("norm", _I), ("dtype", _I),
                ("eps", ctypes.c_float), ("q", NysStrides), ("k", NysStrides),
                ("q_out", NysStrides), ("k_out", NysStrides), ("dq", NysStrides), ("dk", NysStrides)]


class NysKv4Cache(ctypes.Structure):
    """nys_kv4_cache_t."""
    _fields_ = [("data", _P), ("block_table", _P), ("num_pages", _I), ("max_pages", _I),
                ("page_size", _I), ("Hk", _I), ("d", _I)]


_SIG = {
    "nystrom_attn_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P]),
    "nystrom_attn_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I, _I]),
    "nystrom_attn_fwd_ws": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P,
                                 ctypes.c_size_t, _P]),
    "nystrom_attn_fwd_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P]),
    "nystrom_attn_fwd_host": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P]),
    "nystrom_attn_fwd_ex": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P,
                                 ctypes.c_size_t, _P]),
    "nystrom_attn_stage_offset": (ctypes.c_longlong, [_I, _I, _I, _I, _I, _I, _I]),
    "nystrom_plan_describe": (_I, [_I, _I, _I, _I, _I, _I, _I, _I, ctypes.c_char_p, _I]),
    "nystrom_get_status": (_I, [_P]),
    "nystrom_strerror": (ctypes.c_char_p, [_I]),
    "nystrom_last_error_string": (ctypes.c_char_p, []),
    "nystrom_launch_count": (ctypes.c_ulonglong, []),
    "nystrom_profile_enable": (_I, [_I]),
    "nystrom_debug_stall_pinv": (_I, [_I]),
    "nystrom_mha_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I, _I]),
    "nystrom_clustered_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I, _I]),
    "nystrom_clustered_stage_offset": (ctypes.c_longlong, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "nystrom_clustered_attn_fwd": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P,
                                        ctypes.c_size_t, _P]),
    "nystrom_mha_fwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P,
                             ctypes.c_size_t, _P]),
    "nystrom_qk_norm_rope_fwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "nystrom_qk_norm_rope_workspace_bytes": (ctypes.c_size_t, [_P]),
    "nystrom_qk_norm_rope_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                      ctypes.c_size_t, _P]),
    "nystrom_kv4_cache_bytes": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "nystrom_kv4_write": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
    "nystrom_kv4_read": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
    "nystrom_kv4_attn_workspace_bytes": (ctypes.c_size_t, [_P, _I, _I, _I, _I, _I]),
    "nystrom_kv4_attn_fwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.c_float, _I,
                                  _P, ctypes.c_size_t, _P]),
    "nystrom_profile_read": (_I, [_I, ctypes.c_char_p, _I, ctypes.POINTER(ctypes.c_double),
                                  ctypes.POINTER(ctypes.c_longlong)]),
}


class NystromError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        detail = ""
        if code == NYS_ERR_CUDA:
            detail = ": " + load_library().nystrom_last_error_string().decode()
        super().__init__(f"{where} returned {code} ({nystrom_strerror(code)}){detail}")


def load_library(path: str | None = None):
    """Load libnystrom.so (built by __graft_entry__.build()). Raises if it
    is missing: there is no fallback."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIG.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if hasattr(x, "ctypes"):  # numpy array (host buffers)
        return x.ctypes.data
    raise TypeError(f"cannot take a pointer of {type(x)}")


def _stream(s) -> int | None:
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(rc: int, where: str) -> int:
    if rc < 0:
        raise NystromError(rc, where)
    return rc


def nystrom_attn_fwd(q, k, v, conv_w, out, B, H, n, d, m, iters, conv_ks, dtype, stream=None):
    lib = load_library()
    return _check(lib.nystrom_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(conv_w), _ptr(out),
                                       B, H, n, d, m, iters, conv_ks, dtype, _stream(stream)),
                  "nystrom_attn_fwd")


def nystrom_attn_workspace_bytes(B, H, n, d, m, dtype) -> int:
    return load_library().nystrom_attn_workspace_bytes(B, H, n, d, m, dtype)


def nystrom_attn_fwd_ws(q, k, v, conv_w, out, B, H, n, d, m, iters, conv_ks, dtype,
                        workspace, ws_bytes, stream=None):
    lib = load_library()
    return _check(lib.nystrom_attn_fwd_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(conv_w), _ptr(out),
                                          B, H, n, d, m, iters, conv_ks, dtype, _ptr(workspace),
                                          ws_bytes, _stream(stream)),
                  "nystrom_attn_fwd_ws")


def nystrom_attn_fwd_noalloc(q, k, v, conv_w, out, B, H, n, d, m, iters, conv_ks, dtype,
                             stream=None):
    """The forward pass with no device allocation: scratch is a fixed 32 MiB
    array inside the library (see include/nystrom.h)."""
    lib = load_library()
    return _check(lib.nystrom_attn_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(conv_w), _ptr(out),
                                               B, H, n, d, m, iters, conv_ks, dtype,
                                               _stream(stream)),
                  "nystrom_attn_fwd_noalloc")


def nystrom_attn_fwd_ex(q, k, v, conv_w, out, B, H, n, d, m, iters, conv_ks, dtype,
                        conv_layout=NYS_CONV_PER_HEAD, lengths=None, workspace=None, ws_bytes=0,
                        stream=None):
    """The forward pass with per-channel conv filters and/or padded sequences
    (see include/nystrom.h). `lengths`: a host sequence of B ints, or None."""
    lib = load_library()
    lens = None
    if lengths is not None:
        lens = (ctypes.c_int * B)(*[int(x) for x in lengths])
    return _check(lib.nystrom_attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(conv_w), _ptr(out),
                                          B, H, n, d, m, iters, conv_ks, dtype, conv_layout,
                                          ctypes.cast(lens, ctypes.c_void_p) if lens is not None
                                          else None, _ptr(workspace), ws_bytes, _stream(stream)),
                  "nystrom_attn_fwd_ex")


def nystrom_attn_fwd_host(q, k, v, conv_w, out, B, H, n, d, m, iters, conv_ks, dtype, stream=None):
    lib = load_library()
    return _check(lib.nystrom_attn_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(conv_w), _ptr(out),
                                            B, H, n, d, m, iters, conv_ks, dtype, _stream(stream)),
                  "nystrom_attn_fwd_host")


def nystrom_attn_stage_offset(B, H, n, d, m, dtype, stage) -> int:
    return load_library().nystrom_attn_stage_offset(B, H, n, d, m, dtype, stage)


def nystrom_plan_describe(B, H, n, d, m, iters, conv_ks, dtype) -> str:
    """The kernels a forward call of this shape launches (host only)."""
    lib = load_library()
    need = _check(lib.nystrom_plan_describe(B, H, n, d, m, iters, conv_ks, dtype, None, 0),
                  "nystrom_plan_describe")
    buf = ctypes.create_string_buffer(need + 1)
    lib.nystrom_plan_describe(B, H, n, d, m, iters, conv_ks, dtype, buf, need + 1)
    return buf.value.decode()


def nystrom_get_status(stream=None) -> int:
    return load_library().nystrom_get_status(_stream(stream))


def nystrom_strerror(code: int) -> str:
    return load_library().nystrom_strerror(code).decode()


def nystrom_last_error_string() -> str:
    return load_library().nystrom_last_error_string().decode()


def nystrom_attention(q, k, v, conv_w, m: int, iters: int, out=None, stream=None):
    """Convenience call on CUDA torch tensors q, k, v [B, H, n, d] (float32
    or bfloat16, contiguous) and conv_w [H, ks] float32 (or None): allocates
    `out` if not given and calls nystrom_attn_fwd on the current stream."""
    import torch
    for t in (q, k, v):
        if not (t.is_cuda and t.is_contiguous() and t.dim() == 4 and t.dtype == q.dtype):
            raise ValueError("q, k, v must be contiguous CUDA tensors [B, H, n, d] of one dtype")
    if q.dtype == torch.float32:
        dtype = NYS_FP32
    elif q.dtype == torch.bfloat16:
        dtype = NYS_BF16
    else:
        raise ValueError("dtype must be float32 or bfloat16")
    B, H, n, d = q.shape
    ks = 0
    if conv_w is not None:
        if not (conv_w.is_cuda and conv_w.dtype == torch.float32 and conv_w.is_contiguous()
                and conv_w.dim() == 2 and conv_w.shape[0] == H):
            raise ValueError("conv_w must be a contiguous float32 CUDA tensor [H, ks]")
        ks = conv_w.shape[1]
    if out is None:
        out = torch.empty_like(q)
    nystrom_attn_fwd(q, k, v, conv_w if ks > 0 else None, out, B, H, n, d, m, iters, ks, dtype,
                     stream)
    return out


def nystrom_mha_workspace_bytes(B, n, H, d, m, dtype) -> int:
    return load_library().nystrom_mha_workspace_bytes(B, n, H, d, m, dtype)


def nystrom_mha_fwd(x, w_qkv, b_qkv, w_o, b_o, conv_w, y, B, n, H, d, m, iters, conv_ks, dtype,
                    workspace=None, ws_bytes=0, stream=None):
    """The attention module around the op (see include/nystrom.h)."""
    lib = load_library()
    return _check(lib.nystrom_mha_fwd(_ptr(x), _ptr(w_qkv), _ptr(b_qkv), _ptr(w_o), _ptr(b_o),
                                      _ptr(conv_w), _ptr(y), B, n, H, d, m, iters, conv_ks, dtype,
                                      _ptr(workspace), ws_bytes, _stream(stream)),
                  "nystrom_mha_fwd")


def nystrom_clustered_workspace_bytes(B, H, n, d, C, dtype) -> int:
    return load_library().nystrom_clustered_workspace_bytes(B, H, n, d, C, dtype)


def nystrom_clustered_stage_offset(B, H, n, d, C, iters, dtype, stage) -> int:
    return load_library().nystrom_clustered_stage_offset(B, H, n, d, C, iters, dtype, stage)


def nystrom_clustered_attn_fwd(q, k, v, out, B, H, n, d, C, iters, dtype, workspace=None,
                               ws_bytes=0, stream=None):
    """Clustered attention, centroid path (see include/nystrom.h)."""
    lib = load_library()
    return _check(lib.nystrom_clustered_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, H, n, d,
                                                 C, iters, dtype, _ptr(workspace), ws_bytes,
                                                 _stream(stream)),
                  "nystrom_clustered_attn_fwd")


def nystrom_debug_stall_pinv(on: bool) -> int:
    """Timeout-path test switch (see include/nystrom.h)."""
    return _check(load_library().nystrom_debug_stall_pinv(1 if on else 0),
                  "nystrom_debug_stall_pinv")


def nystrom_launch_count() -> int:
    return load_library().nystrom_launch_count()


def nystrom_profile_enable(on: bool) -> int:
    return load_library().nystrom_profile_enable(1 if on else 0)


def nystrom_profile_read(max_kernels: int = 16) -> dict:
    """{kernel name: (total ms, launches)} recorded since the last read."""
    lib = load_library()
    name_len = 64
    names = ctypes.create_string_buffer(max_kernels * name_len)
    ms = (ctypes.c_double * max_kernels)()
    cnt = (ctypes.c_longlong * max_kernels)()
    n = _check(lib.nystrom_profile_read(max_kernels, names, name_len, ms, cnt), "nystrom_profile_read")
    out = {}
    for i in range(min(n, max_kernels)):
        nm = names.raw[i * name_len:(i + 1) * name_len].split(b"\0", 1)[0].decode()
        out[nm] = (ms[i], cnt[i])
    return out


# ------------------------------------------- around a cached attention layer
#
# These take torch tensors whose strides they pass on: heads are [B, H, n, d]
# views with contiguous channels (a token-major [B, n, H, d] tensor or a slice
# of a packed projection: its transpose). The descriptors go over as packed
# bytes (a fraction of the time that filling ctypes structures takes).

_ROPE_DESC = struct.Struct("=14if4x18q")  # nys_qk_rope_t
_KV4_DESC = struct.Struct("=QQ5i4x")      # nys_kv4_cache_t
_STRIDES = struct.Struct("=3q")           # nys_strides_t
_NO_STRIDES = (0, 0, 0)
_INT_MAX = 2 ** 31 - 1  # ctypes cuts what is larger to an int's 32 bits
_torch = None
_np = None


def _lazy_torch():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _check_first(name, t):
    """(strides, dtype code, device index) of a call's first heads."""
    torch = _torch or _lazy_torch()
    dtype = t.dtype
    if dtype is torch.bfloat16:
        code = NYS_BF16
    elif dtype is torch.float32:
        code = NYS_FP32
    else:
        raise ValueError(f"{name} must be float32 or bfloat16")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor [B, H, n, d]")
    device = torch._C._cuda_getDevice()
    return _heads(name, t, dtype, None, device), code, device


def _heads(name, t, dtype, shape, device):
    """(batch, head, token) strides of a [B, H, n, d] view of the given type and
    shape on the current device. An axis with one entry has no stride."""
    s, n = t.stride(), t.shape
    if len(s) != 4 or s[3] != 1:
        raise ValueError(f"{name} must be [B, H, n, d] with contiguous channels")
    if shape is not None and n != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(n)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype} like the other heads")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on the current CUDA device")
    if 1 in n:
        return (s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0, s[2] if n[2] > 1 else 0)
    return s[:3]


def _flat(name, t, dtype, shape, device):
    """Address of a contiguous array of the given type, shape and device
    index, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on device {device}")
    return t.data_ptr()


def _raw_stream(stream, device):
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


class _Scratch(threading.local):
    """by_device: device index: workspace of this thread's calls on its default stream."""

    def __init__(self):
        self.by_device = {}


_default_scratch = _Scratch()


def _scratch(nbytes, workspace, device, stream):
    """(address, bytes, tensor to keep until the launch) of a call's workspace:
    the caller's; on the default stream one that this thread's calls share (the
    kernels of one run behind those of another, and it cannot be captured; two
    threads' calls could enqueue theirs in between each other); else memory of
    torch's allocator that belongs to the call's stream, so that it is reused only
    behind the call."""
    torch = _torch
    if workspace is not None:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on device {device}")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if nbytes == 0:
        return None, 0, None
    raw, current = _raw_stream(stream, device), torch._C._cuda_getCurrentRawStream(device)
    if raw == 0 == current:
        kept = _default_scratch.by_device
        t = kept.get(device)
        if t is None or t.numel() < nbytes:
            t = kept[device] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    elif raw == current:
        t = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    else:
        with torch.cuda.stream(torch.cuda.ExternalStream(raw)):
            t = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return t.data_ptr(), nbytes, t


def _rope_args(names, tensors, inv_freq, positions, sections, norm, eps, pairing):
    """Packed descriptor, frequencies as bytes, address of the positions and
    device of a call on (q, k, q_out or gq, k_out or gk[, dq, dk])."""
    global _np
    q, k = tensors[0], tensors[1]
    qs, code, device = _check_first(names[0], q)
    dtype, shape = q.dtype, q.shape
    B, Hq, n, d = shape
    if k is None:
        Hk, kshape = 0, None
    else:
        kshape = k.shape
        if len(kshape) != 4 or kshape[0] != B or kshape[2] != n or kshape[3] != d:
            raise ValueError(f"k must have shape [{B}, Hk, {n}, {d}], not {tuple(kshape)}")
        Hk = kshape[1]
    strides = list(qs)
    for i in range(1, len(tensors)):
        if i & 1 == 0:
            strides += _heads(names[i], tensors[i], dtype, shape, device)
        elif k is None:
            strides += _NO_STRIDES
        else:
            strides += _heads(names[i], tensors[i], dtype, kshape, device)
    if len(tensors) == 4:
        strides += _NO_STRIDES * 2
    if _np is None:
        import numpy as _np
    freq = _np.asarray(inv_freq, dtype=_np.float64)
    if freq.ndim != 1 or len(freq) > 64:
        raise ValueError("inv_freq must be one-dimensional, at most 64 long")
    half = len(freq)
    axes = 1 if sections is None else len(sections)
    if not 1 <= axes <= 4:
        raise ValueError("one to four axes")
    sec = (half, 0, 0, 0) if sections is None else (*sections, *(0,) * (4 - axes))
    desc = _ROPE_DESC.pack(B, n, Hq, Hk, d, 2 * half, axes, *sec, pairing, 1 if norm else 0, code, eps, *strides)
    pos = None if positions is None else _flat("positions", positions, _torch.int32, (axes, B, n), device)
    return desc, freq.tobytes(), pos, device


def nystrom_qk_norm_rope_fwd(q, k, q_out, k_out, positions, inv_freq, q_weight=None, k_weight=None, *,
                             sections=None, pairing=NYS_ROPE_HALVES, norm=True, eps=1e-6, stream=None):
    """Per-head RMS norm and position rotation of queries q [B, Hq, n, d] and
    keys k [B, Hk, n, d] (or None) into q_out, k_out (see include/nystrom.h).
    positions: int32 [axes, B, n] on the device, or None for 0 .. n-1.
    inv_freq: host sequence of rot/2 radians per position. sections: pairs per
    axis (None: one axis). q_weight, k_weight: float32 [d], or None."""
    lib = _lib or load_library()
    desc, freq, pos, dev = _rope_args(("q", "k", "q_out", "k_out"), (q, k, q_out, k_out), inv_freq,
                                      positions, sections, norm, eps, pairing)
    d, f32 = (q.shape[3],), _torch.float32
    rc = lib.nystrom_qk_norm_rope_fwd(
        desc, q.data_ptr(), None if k is None else k.data_ptr(),
        _flat("q_weight", q_weight, f32, d, dev), _flat("k_weight", k_weight, f32, d, dev), pos, freq,
        q_out.data_ptr(), None if k is None else k_out.data_ptr(), _raw_stream(stream, dev))
    return rc if rc >= 0 else _check(rc, "nystrom_qk_norm_rope_fwd")


def nystrom_qk_norm_rope_workspace_bytes(desc) -> int:
    """desc: NysQkRope."""
    return load_library().nystrom_qk_norm_rope_workspace_bytes(
        ctypes.byref(desc) if isinstance(desc, NysQkRope) else desc)


def nystrom_qk_norm_rope_bwd(q, k, gq, gk, dq, dk, positions, inv_freq, q_weight=None, k_weight=None,
                             dq_weight=None, dk_weight=None, *, sections=None, pairing=NYS_ROPE_HALVES,
                             norm=True, eps=1e-6, workspace=None, stream=None):
    """Gradients of nystrom_qk_norm_rope_fwd: from its inputs q, k and the
    outputs' gradients gq, gk into dq, dk (which may be gq, gk) and, where
    given, dq_weight, dk_weight (float32 [d])."""
    lib = _lib or load_library()
    desc, freq, pos, dev = _rope_args(("q", "k", "gq", "gk", "dq", "dk"), (q, k, gq, gk, dq, dk), inv_freq,
                                      positions, sections, norm, eps, pairing)
    d, f32 = (q.shape[3],), _torch.float32
    need = 0
    if dq_weight is not None or dk_weight is not None:
        need = lib.nystrom_qk_norm_rope_workspace_bytes(desc)
    ws, nbytes, keep = _scratch(need, workspace, dev, stream)
    rc = lib.nystrom_qk_norm_rope_bwd(
        desc, q.data_ptr(), None if k is None else k.data_ptr(), gq.data_ptr(),
        None if k is None else gk.data_ptr(), _flat("q_weight", q_weight, f32, d, dev),
        _flat("k_weight", k_weight, f32, d, dev), pos, freq, dq.data_ptr(),
        None if k is None else dk.data_ptr(), _flat("dq_weight", dq_weight, f32, d, dev),
        _flat("dk_weight", dk_weight, f32, d, dev), ws, nbytes, _raw_stream(stream, dev))
    del keep
    return rc if rc >= 0 else _check(rc, "nystrom_qk_norm_rope_bwd")


def nystrom_kv4_cache_bytes(num_pages, page_size, Hk, d) -> int:
    if max(num_pages, page_size, Hk, d) > _INT_MAX:
        return 0  # like other sizes that a call refuses
    return load_library().nystrom_kv4_cache_bytes(num_pages, page_size, Hk, d)


class NystromKv4Cache:
    """A 4-bit key/value cache over the caller's memory (format: see
    include/nystrom.h). data: uint8 CUDA tensor, a whole number of pages;
    block_table: int32 [B, max_pages], sequence b's pages in order. Both are
    kept; new pages are entered into the same tensor."""

    __slots__ = ("_data", "_block_table", "B", "Hk", "d", "device", "desc")

    def __init__(self, data, block_table, page_size, Hk, d):
        torch = _torch or _lazy_torch()
        if page_size % 16 or not 16 <= page_size <= 4096 or Hk < 1 or d not in (32, 64, 128):
            raise NystromError(NYS_ERR_SHAPE, "NystromKv4Cache")
        if not data.is_cuda or data.dtype != torch.uint8 or not data.is_contiguous():
            raise ValueError("data must be a contiguous uint8 CUDA tensor")
        page = Hk * (page_size // 16) * 18 * d
        pages, rest = divmod(data.numel(), page)
        if pages < 1 or rest:
            raise ValueError(f"data must be a whole number of {page}-byte pages")
        if (block_table.dtype != torch.int32 or block_table.dim() != 2
                or block_table.get_device() != data.get_device() or not block_table.is_contiguous()):
            raise ValueError("block_table must be a contiguous int32 tensor [B, max_pages] beside the data")
        self._data, self._block_table = data, block_table
        self.B, max_pages = block_table.shape
        self.Hk, self.d, self.device = Hk, d, data.get_device()
        self.desc = _KV4_DESC.pack(data.data_ptr(), block_table.data_ptr(), pages, max_pages, page_size, Hk, d)

    @property
    def data(self):
        return self._data

    @property
    def block_table(self):
        return self._block_table


def _kv4_io(cache, k, v, starts, counts):
    ks, code, dev = _check_first("k", k)
    shape, dtype, B = k.shape, k.dtype, cache.B
    if dev != cache.device or shape[0] != B or shape[1] != cache.Hk or shape[3] != cache.d:
        raise ValueError(f"k must be [{B}, {cache.Hk}, n, {cache.d}] on the cache's device, not {tuple(shape)}")
    vs = _heads("v", v, dtype, shape, dev)
    if shape[2] > _INT_MAX:
        raise ValueError(f"{shape[2]} tokens are more than a call takes")
    i32 = _torch.int32
    return (k.data_ptr(), v.data_ptr(), _STRIDES.pack(*ks), _STRIDES.pack(*vs),
            _flat("starts", starts, i32, (B,), dev), _flat("counts", counts, i32, (B,), dev), B, shape[2], code)


def nystrom_kv4_write(cache, k, v, starts=None, counts=None, stream=None):
    """Quantises rows i < counts[b] of k, v [B, Hk, n, d] into the cache at
    positions starts[b] + i (int32 device tensors; None: n rows, from 0)."""
    rc = (_lib or load_library()).nystrom_kv4_write(cache.desc, *_kv4_io(cache, k, v, starts, counts),
                                                    _raw_stream(stream, cache.device))
    return rc if rc >= 0 else _check(rc, "nystrom_kv4_write")


def nystrom_kv4_read(cache, k, v, starts=None, counts=None, stream=None):
    """What the cache holds at positions starts[b] + i to rows i < counts[b]
    of k, v [B, Hk, n, d]; rows behind are left as they were."""
    rc = (_lib or load_library()).nystrom_kv4_read(cache.desc, *_kv4_io(cache, k, v, starts, counts),
                                                   _raw_stream(stream, cache.device))
    return rc if rc >= 0 else _check(rc, "nystrom_kv4_read")


def nystrom_kv4_attn_workspace_bytes(cache, B, nq, Hq, max_length, dtype) -> int:
    if max(B, nq, Hq, max_length) > _INT_MAX:
        return 0  # like other sizes that a call refuses
    return load_library().nystrom_kv4_attn_workspace_bytes(cache.desc, B, nq, Hq, max_length, dtype)


def nystrom_kv4_attn_fwd(cache, q, out, lengths, max_length, q_counts=None, causal=True, scale=None,
                         workspace=None, stream=None):
    """Attention of queries q [B, Hq, nq, d] over the cached tokens of each
    sequence into out (same shape). lengths: int32 [B], tokens in the cache;
    max_length: an upper bound of them; q_counts: int32 [B], real queries
    (None: nq); scale: None for 1/sqrt(d)."""
    lib = _lib or load_library()
    if scale is None:
        scale = 0.0
    elif ctypes.c_float(scale).value == 0.0:
        raise ValueError("scale must not be zero in fp32 (None: 1/sqrt(d))")
    qs, dt, dev = _check_first("q", q)
    shape = q.shape
    B, Hq, nq, d = shape
    if B != cache.B or d != cache.d or dev != cache.device:
        raise ValueError("q must be [B, Hq, nq, d] with the cache's B and d, on its device")
    if max(nq, Hq, max_length) > _INT_MAX or max_length < 0:
        raise ValueError(f"sizes past 32 bits or below zero: {nq} queries, {Hq} heads, max_length {max_length}")
    os_ = _heads("out", out, q.dtype, shape, dev)
    i32 = _torch.int32
    need = lib.nystrom_kv4_attn_workspace_bytes(cache.desc, B, nq, Hq, max_length, dt)
    ws, nbytes, keep = _scratch(need, workspace, dev, stream)
    rc = lib.nystrom_kv4_attn_fwd(
        cache.desc, q.data_ptr(), out.data_ptr(), _STRIDES.pack(*qs), _STRIDES.pack(*os_),
        _flat("lengths", lengths, i32, (B,), dev), _flat("q_counts", q_counts, i32, (B,), dev), B, nq, Hq,
        max_length, 1 if causal else 0, scale, dt, ws, nbytes,
        _raw_stream(stream, dev))
    del keep
    return rc if rc >= 0 else _check(rc, "nystrom_kv4_attn_fwd")
