"""fp64 numpy reference of the operators around the attention module: the
residual's addition with its norm and their gradients, matrices in 8 bits, the
gated feed-forward product with its gradients. Written from the formulas in
include/nystrom.h; shares no code with the library."""
import math

import numpy as np

BLOCK = 128


def to_bf16(x):
    """x rounded to bfloat16 (ties to even), as fp64. x fits fp32's range."""
    x = np.asarray(x, np.float64)
    m, e = np.frexp(x)  # |m| in [1/2, 1): 8 significant bits are multiples of 2^-8
    return np.ldexp(np.rint(np.ldexp(m, 8)), e - 8)


def rounded(x, dtype):
    return to_bf16(x) if dtype == "bf16" else np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


# ------------------------------------------------------------------- norm

def add_rms_norm(x, residual, weight, eps, dtype):
    """(s, y): s rounded to dtype, y not rounded."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = rounded(s + np.asarray(residual, np.float64), dtype)
    r = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    return s, s * r * (1.0 if weight is None else np.asarray(weight, np.float64))


def add_rms_norm_grad(s, gy, gs, weight, eps):
    """(dx, dweight)."""
    s, gy = np.asarray(s, np.float64), np.asarray(gy, np.float64)
    w = np.ones(s.shape[1]) if weight is None else np.asarray(weight, np.float64)
    r = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    h = r * s
    wg = w * gy
    dx = r * (wg - h * (wg * h).mean(-1, keepdims=True))
    return dx + (0.0 if gs is None else np.asarray(gs, np.float64)), (gy * h).sum(0)


# ------------------------------------------------------------- 8-bit values

def e4m3_value(code):
    """The value of one code (0 .. 255)."""
    sign, e, m = code >> 7, code >> 3 & 15, code & 7
    if e == 15 and m == 7:
        return math.nan
    v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -v if sign else v


VALUES = np.array([e4m3_value(c) for c in range(256)])


def e4m3_code(v):
    """Codes of the nearest values (ties to the even code); v finite, |v| <= 464."""
    v = np.asarray(v, np.float64)
    mags = VALUES[:127]  # 0 .. 448, increasing
    a = np.abs(v)
    hi = np.minimum(np.searchsorted(mags, a), 126)
    lo = np.maximum(hi - 1, 0)
    up, down = mags[hi] - a, a - mags[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def scale_byte(top):
    """Byte of the smallest power of two with top <= 448 * 2^(byte - 127)."""
    if not math.isfinite(top):
        return 255
    e = -127
    if top > 0:
        e = math.frexp(top / 448)[1]  # 2^(e-1) <= top / 448 < 2^e
        if top <= 448 * 2.0 ** (e - 1):
            e -= 1
    return max(e, -127) + 127


def q8_write(x, block_rows=1):
    """(codes [rows, K], bytes [rows, blocks]). Blocks that are not finite: codes undefined (0)."""
    x = np.asarray(x, np.float64)
    rows, K = x.shape
    blocks = -(-K // BLOCK)
    codes, bytes_ = np.zeros((rows, K), np.uint8), np.zeros((rows, blocks), np.uint8)
    for r in range(0, rows, block_rows):
        for b in range(blocks):
            at = np.s_[r:r + block_rows, b * BLOCK:(b + 1) * BLOCK]
            part = x[at]
            top = np.abs(part).max() if np.isfinite(part).all() else math.inf
            byte = scale_byte(top)
            bytes_[r:r + block_rows, b] = byte
            if byte != 255:
                codes[at] = e4m3_code(part / 2.0 ** (byte - 127))
    return codes, bytes_


def q8_words(bytes_):
    """Scale words [ceil(blocks / 4), rows] (int32) of scale bytes [rows, blocks]."""
    rows, blocks = bytes_.shape
    pad = np.zeros((rows, -(-blocks // 4) * 4), np.uint8)
    pad[:, :blocks] = bytes_
    return np.ascontiguousarray(pad.reshape(rows, -1, 4).transpose(1, 0, 2)).view(np.int32)[..., 0]


def q8_bytes(words, K):
    """Scale bytes [rows, blocks] of scale words."""
    w = np.ascontiguousarray(words, dtype=np.int32)
    b = w[..., None].view(np.uint8).transpose(1, 0, 2).reshape(w.shape[1], -1)
    return b[:, :-(-K // BLOCK)]


def q8_read(codes, bytes_):
    scale = np.where(bytes_ == 255, np.nan, 2.0 ** (bytes_.astype(np.float64) - 127))
    return VALUES[codes] * np.repeat(scale, BLOCK, 1)[:, :codes.shape[1]]


# ------------------------------------------------------------- feed-forward

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act(g, name):
    """act(g) and act'(g)."""
    g = np.asarray(g, np.float64)
    if name == "relu":
        return np.maximum(g, 0.0), (g > 0).astype(np.float64)
    if name == "gelu":
        p = 0.5 * _erfc(-g / math.sqrt(2))
        return g * p, p + g * np.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        z, dz = 1.5957691216057308 * (g + 0.044715 * g ** 3), 1.5957691216057308 * (1 + 3 * 0.044715 * g * g)
    else:
        z, dz = g, np.ones_like(g)
    s = 1.0 / (1.0 + np.exp(-z))
    return g * s, s + g * s * (1 - s) * dz


def gated_ff(x, w_gate, w_up, name):
    """(h, g, u)."""
    x = np.asarray(x, np.float64)
    g, u = x @ np.asarray(w_gate, np.float64), x @ np.asarray(w_up, np.float64)
    return act(g, name)[0] * u, g, u


def gated_ff_grad(x, w_gate, w_up, g, u, gh, name, dtype=None):
    """(dx, dw_gate, dw_up); dtype: dg and du are rounded to it."""
    a, slope = act(g, name)
    gh = np.asarray(gh, np.float64)
    dg, du = gh * np.asarray(u, np.float64) * slope, gh * a
    if dtype is not None:
        dg, du = rounded(dg, dtype), rounded(du, dtype)
    x = np.asarray(x, np.float64)
    return dg @ np.asarray(w_gate, np.float64).T + du @ np.asarray(w_up, np.float64).T, x.T @ dg, x.T @ du
