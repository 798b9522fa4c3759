"""Timed cases of the operators around an attention module in a Transformer
layer: the residual's addition with its root-mean-square norm (output in the
input's type or in 8 bits, and its gradients), the product in 8-bit floating
point with a scale for each block of 128, and the gated feed-forward product
with its gradients.

`run` computes a case either in plain torch operations (`own` false) or with
this package's kernels (`own` true), from the same prepared state."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6


# ------------------------------------------------------------------- cases

def listed():
    norm = dict(op="norm", back=False, eight=False, res=True, dtype="bf16")
    q8 = dict(op="q8", wide=False, given=True)
    ff = dict(op="ff", back=False, keep=False, act="silu", order="in_out", dtype="bf16")
    return [
        # one decoding step of 32 sequences: latency
        dict(norm, name="norm_step", rows=32, d=2048),
        # the long-context workload's tokens at its module width, into the next
        # projection's 8 bits (and back to the values they stand for)
        dict(norm, name="norm_long_8bit", rows=65536, d=2048, eight=True),
        # odd width, fp32, no residual: a model's last norm
        dict(norm, name="norm_last_f32", rows=16381, d=1544, res=False, dtype="f32"),
        # training step over two sequences of 8192
        dict(norm, name="norm_back", back=True, rows=16384, d=4096),
        # four sequences' single tokens through a packed QKV projection: latency, weights' bytes
        dict(q8, name="q8_step", T=4, N=6144, K=2048),
        # a prompt's chunk, tokens still in 16 bits: quantised on the way
        dict(q8, name="q8_chunk", T=1000, N=6144, K=2048, given=False),
        # every token of the long-context workload through a wide projection
        dict(q8, name="q8_long", T=65536, N=4096, K=2048),
        # odd sizes, result in 32 bits
        dict(q8, name="q8_odd_f32", T=509, N=1000, K=1456, wide=True),
        # one token through a feed-forward block: the weights' bytes
        dict(ff, name="ff_step", T=1, d=4096, f=11264),
        # training, forward, with what the gradients need kept
        dict(ff, name="ff_train", T=16384, d=2048, f=5632, keep=True),
        # training, gradients of the input and both weights
        dict(ff, name="ff_back", back=True, T=16384, d=2048, f=5632),
        # a short odd batch in fp32, weights as a linear layer keeps them
        dict(ff, name="ff_back_small_f32", back=True, T=509, d=512, f=1368, act="gelu_tanh",
             order="out_in", dtype="f32"),
    ]


def _cost(c):
    """Rough time of the plain form: bytes of its intermediates, and products."""
    if c["op"] == "norm":
        return (60.0 if c["back"] or c["eight"] else 30.0) * c["rows"] * c["d"]
    if c["op"] == "q8":
        return 0.25 * c["T"] * c["N"] * c["K"] + 60.0 * (c["T"] + c["N"]) * c["K"]
    return (1.0 if c["back"] else 0.5) * c["T"] * c["d"] * c["f"] + 16.0 * c["d"] * c["f"]


def _log(rng, lo, hi, step=1):
    x = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + step)))))
    return max(lo, min(hi, x // step * step))


def draw(rng):
    most = {c["op"]: 0.0 for c in listed()}
    for c in listed():
        most[c["op"]] = max(most[c["op"]], _cost(c))
    while True:
        op = rng.choice(["norm", "q8", "ff"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if op == "norm":
            eight = rng.random() < 0.4
            c = dict(op=op, rows=_log(rng, 1, 65536), d=_log(rng, 64, 16384, 16 if eight else 8),
                     eight=eight, back=not eight and rng.random() < 0.5, res=rng.random() < 0.75,
                     dtype=dtype)
        elif op == "q8":
            c = dict(op=op, T=rng.choice([_log(rng, 1, 64), _log(rng, 1, 65536)]),
                     N=_log(rng, 64, 16384, 8), K=_log(rng, 128, 16384, 16),
                     wide=dtype == "f32", given=rng.random() < 0.6)
        else:
            back = rng.random() < 0.5
            c = dict(op=op, T=rng.choice([_log(rng, 1, 64), _log(rng, 1, 32768)]),
                     d=_log(rng, 64, 8192, 8), f=_log(rng, 64, 16384, 8), back=back,
                     keep=not back and rng.random() < 0.4,
                     act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"]),
                     order=rng.choice(["in_out", "out_in"]), dtype=dtype)
        if _cost(c) <= most[op]:
            return c


# ------------------------------------------------------------------ inputs

def _normal(g, shape, dtype, spread=1.0):
    return torch.empty(shape, dtype=DTYPES[dtype], device="cuda").normal_(0.0, spread, generator=g)


def _eight_bits(x, block_rows):
    """Codes [rows, K] and scale words [ceil(K/512), rows] of a matrix: the
    exponent (offset 127) of block 4 g + j is byte j of word g."""
    rows, K = x.shape
    up, right = -rows % block_rows, -K % 128
    pad = torch.nn.functional.pad(x.double(), (0, right, 0, up))
    tiles = pad.view((rows + up) // block_rows, block_rows, (K + right) // 128, 128)
    top = tiles.abs().amax((1, 3), keepdim=True)
    e = _exponent(top)
    codes = (tiles / torch.exp2(e)).float().to(torch.float8_e4m3fn).view(torch.uint8).view(pad.shape)
    bytes_ = (e + 127).to(torch.uint8)[:, 0, :, 0].repeat_interleave(block_rows, 0)[:rows]
    words = torch.nn.functional.pad(bytes_, (0, -bytes_.shape[1] % 4)).view(rows, -1, 4)
    words = words.transpose(0, 1).contiguous().view(torch.int32)[..., 0]
    return codes[:rows, :K].contiguous(), words.contiguous()


def _exponent(top):
    """Smallest e with top <= 448 * 2^e, -127 where all is zero."""
    m, e = torch.frexp(top / 448)
    return torch.where(top > 0, torch.where(m == 0.5, e - 1, e), -127).clamp(min=-127).double()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    if c["op"] == "norm":
        rows, d = c["rows"], c["d"]
        # a residual stream: some channels much larger than the rest
        big = 1 + 12 * (torch.rand(d, device="cuda", generator=g) > 0.98)
        st = dict(case=c, weight=1 + 0.2 * torch.randn(d, device="cuda", generator=g))
        st["x"] = _normal(g, (rows, d), c["dtype"])
        st["r"] = (_normal(g, (rows, d), c["dtype"]) * big).to(DTYPES[c["dtype"]]) if c["res"] else None
        if c["back"]:
            st["gy"] = _normal(g, (rows, d), c["dtype"])
        return st
    if c["op"] == "q8":
        T, N, K = c["T"], c["N"], c["K"]
        x = _normal(g, (T, K), "bf16") * (1 + 12 * (torch.rand(K, device="cuda", generator=g) > 0.98))
        w = _normal(g, (N, K), "bf16", 1 / math.sqrt(K))
        st = dict(case=c, x=x.to(torch.bfloat16), w=_eight_bits(w, 128))
        if c["given"]:
            st["x"] = _eight_bits(st["x"], 1)
        return st
    T, d, f = c["T"], c["d"], c["f"]
    st = dict(case=c, x=_normal(g, (T, d), c["dtype"]))
    for name in ("wg", "wu"):
        w = _normal(g, (d, f) if c["order"] == "in_out" else (f, d), c["dtype"], 1 / math.sqrt(d))
        st[name] = w if c["order"] == "in_out" else w.T
    if c["back"]:  # what the forward pass kept, and the gradient that arrives
        st["g"] = (st["x"].float() @ st["wg"].float()).to(DTYPES[c["dtype"]])
        st["u"] = (st["x"].float() @ st["wu"].float()).to(DTYPES[c["dtype"]])
        st["gh"] = _normal(g, (T, f), c["dtype"])
    return st


# -------------------------------------------------------------- plain forms

def _plain_norm(state):
    c, w = state["case"], state["weight"]
    x = state["x"].float()
    if c["back"]:
        # the forward pass kept the sum; the gradients of the norm and of the sum arrive
        s, gs, gy = x, state["r"].float() if c["res"] else None, state["gy"].float()
        r = torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS)
        hat = s * r
        gh = gy * w
        dx = r * (gh - hat * (gh * hat).mean(-1, keepdim=True))
        dw = (gy * hat).sum(0, dtype=torch.float64).float()
        return [(dx if gs is None else dx + gs).to(state["x"].dtype), dw]
    s = (x + state["r"].float()).to(state["x"].dtype) if c["res"] else state["x"]
    outs = [s] if c["res"] else []
    if not c["eight"]:
        sf = s.float()
        return outs + [(sf * torch.rsqrt(sf.square().mean(-1, keepdim=True) + EPS) * w).to(s.dtype)]
    sd = s.double()  # 64 bits: values next to the border between two codes
    y = sd * torch.rsqrt(sd.square().mean(-1, keepdim=True) + EPS) * w
    return outs + [_plain_rounded(y)]


def _plain_rounded(y):
    """The values that 8 bits and a power of two for each 128 channels stand for."""
    rows, K = y.shape
    tiles = torch.nn.functional.pad(y, (0, -K % 128)).view(rows, -1, 128)
    step = torch.exp2(_exponent(tiles.abs().amax(-1, keepdim=True)))
    near = (tiles / step).float().to(torch.float8_e4m3fn).double() * step
    return near.view(rows, -1)[:, :K].to(torch.bfloat16)


def _plain_values(eight):
    """[rows, K] in 32 bits of codes and scale words."""
    codes, words = eight
    rows, K = codes.shape
    e = words[..., None].view(torch.uint8).transpose(0, 1).reshape(rows, -1)[:, :-(-K // 128)]
    step = torch.exp2(e.float() - 127).repeat_interleave(128, 1)[:, :K]
    return codes.view(torch.float8_e4m3fn).float() * step


def _plain_q8(state):
    c = state["case"]
    x = _plain_values(state["x"]) if c["given"] else _plain_rounded(state["x"].double()).float()
    y = x @ _plain_values(state["w"]).T
    return y if c["wide"] else y.to(torch.bfloat16)


def _act(g, name):
    """An activation and its derivative."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if name == "relu":
        on = (g > 0).to(g.dtype)
        return g * on, on
    if name == "gelu":
        p = 0.5 * (1 + torch.erf(g / math.sqrt(2)))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def _plain_ff(state):
    c, dt = state["case"], state["x"].dtype
    x, wg, wu = state["x"].float(), state["wg"].float(), state["wu"].float()
    if not c["back"]:
        g, u = x @ wg, x @ wu
        h = (_act(g, c["act"])[0] * u).to(dt)
        return [h, g.to(dt), u.to(dt)] if c["keep"] else h
    g, u, gh = state["g"].float(), state["u"].float(), state["gh"].float()
    a, slope = _act(g, c["act"])
    dg, du = gh * u * slope, gh * a
    return [(dg @ wg.T + du @ wu.T).to(dt), (x.T @ dg).to(dt), (x.T @ du).to(dt)]


def run(state):
    c = state["case"]
    if own:
        return {"norm": _own_norm, "q8": _own_q8, "ff": _own_ff}[c["op"]](state)
    return {"norm": _plain_norm, "q8": _plain_q8, "ff": _plain_ff}[c["op"]](state)


# ------------------------------------------------------ the package's calls

def _own_eight(N, rows, K):
    return N.NystromQ8(torch.empty(rows, K, dtype=torch.uint8, device="cuda"),
                       torch.empty(-(-K // 512), rows, dtype=torch.int32, device="cuda"))


def _own_norm(state):
    import nystr_self_attention_gb300 as N
    c, x, r, w = state["case"], state["x"], state["r"], state["weight"]
    if c["back"]:
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        N.nystrom_add_rms_norm_bwd(x, state["gy"], r, w, dx, dw, eps=EPS)
        return [dx, dw]
    s = torch.empty_like(x) if c["res"] else None
    if not c["eight"]:
        y = torch.empty_like(x)
        N.nystrom_add_rms_norm_fwd(x, r, w, s, y, eps=EPS)
    else:
        y = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
        eight = _own_eight(N, *x.shape)
        N.nystrom_add_rms_norm_fwd(x, r, w, s, eight, eps=EPS)
        N.nystrom_q8_read(eight, y)
    return [s, y] if c["res"] else [y]


def _own_q8(state):
    import nystr_self_attention_gb300 as N
    c = state["case"]
    if c["given"]:
        x = N.NystromQ8(*state["x"])
    else:
        x = _own_eight(N, c["T"], c["K"])
        N.nystrom_q8_write(x, state["x"])
    y = torch.empty(c["T"], c["N"], dtype=torch.float32 if c["wide"] else torch.bfloat16, device="cuda")
    N.nystrom_q8_matmul(x, N.NystromQ8(*state["w"]), y)
    return y


def _own_ff(state):
    import nystr_self_attention_gb300 as N
    c, x, wg, wu = state["case"], state["x"], state["wg"], state["wu"]
    act = {"silu": N.NYS_ACT_SILU, "gelu": N.NYS_ACT_GELU, "gelu_tanh": N.NYS_ACT_GELU_TANH,
           "relu": N.NYS_ACT_RELU}[c["act"]]
    if c["back"]:
        dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
        N.nystrom_gated_ff_bwd(x, wg, wu, state["g"], state["u"], state["gh"], dx, dwg, dwu, activation=act)
        return [dx, dwg, dwu]
    h = torch.empty(c["T"], c["f"], dtype=x.dtype, device="cuda")
    if not c["keep"]:
        N.nystrom_gated_ff_fwd(x, wg, wu, h, activation=act)
        return h
    g, u = torch.empty_like(h), torch.empty_like(h)
    N.nystrom_gated_ff_fwd(x, wg, wu, h, g, u, activation=act)
    return [h, g, u]


# ------------------------------------------------------------ work and truth

def work(case):
    c = case
    if c["op"] == "norm":
        e, n = ESIZE[c["dtype"]], float(c["rows"]) * c["d"]
        if c["back"]:
            return {"bytes": n * e * (4 if c["res"] else 3) + 8 * c["d"], "flops": 12 * n}
        stored = 2 * (1 + 1 / 128) + 2 if c["eight"] else e  # written, read back, its values written
        return {"bytes": n * (e * (3 if c["res"] else 1) + stored) + 4 * c["d"], "flops": 6 * n}
    if c["op"] == "q8":
        T, N, K = float(c["T"]), float(c["N"]), float(c["K"])
        eight = 1 + 1 / 128
        return {"bytes": T * K * (eight if c["given"] else 2) + N * K * eight + T * N * (4 if c["wide"] else 2),
                "flops": 2 * T * N * K}
    T, d, f, e = float(c["T"]), float(c["d"]), float(c["f"]), ESIZE[c["dtype"]]
    if c["back"]:
        return {"bytes": e * (2 * T * d + 4 * d * f + 3 * T * f), "flops": 8 * T * d * f}
    return {"bytes": e * (T * d + 2 * d * f + (3 if c["keep"] else 1) * T * f), "flops": 4 * T * d * f}


def _exact_block_values(y):
    """8-bit rounding from the format: sign, 4 exponent bits down to 2^-6, 3 of mantissa."""
    out = torch.empty_like(y)
    for j in range(0, y.shape[1], 128):
        part = y[:, j:j + 128]
        top = part.abs().max(1, keepdim=True).values
        e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 448))
        e = torch.where(top > 448 * torch.exp2(e), e + 1, torch.where(top <= 224 * torch.exp2(e), e - 1, e))
        v = part / torch.exp2(e)
        ulp = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        out[:, j:j + 128] = torch.where(top > 0, torch.round(v / ulp) * ulp * torch.exp2(e), 0.0)
    return out


def _exact_norm(state):
    c = state["case"]
    w = state["weight"].double()
    if c["back"]:
        s, w = state["x"].double().requires_grad_(), w.requires_grad_()
        y = w * s / (torch.linalg.vector_norm(s, dim=1, keepdim=True) ** 2 / c["d"] + EPS) ** 0.5
        dx, dw = torch.autograd.grad(y, (s, w), state["gy"].double())
        return [dx + state["r"].double() if c["res"] else dx, dw]
    s = state["x"].double()
    if c["res"]:  # the sum is kept, and normed, in its own type
        s = (s + state["r"].double()).to(state["x"].dtype).double()
    y = w * s / (torch.linalg.vector_norm(s, dim=1, keepdim=True) ** 2 / c["d"] + EPS) ** 0.5
    if c["eight"]:
        y = _exact_block_values(y)
    return [s, y] if c["res"] else [y]


def _exact_matrix(codes, words):
    bits = codes.long()
    e, m = bits >> 3 & 15, (bits & 7).double()
    v = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)
    v = torch.where(bits > 127, -v, v)
    for b in range(-(-codes.shape[1] // 128)):
        power = (words[b // 4].long() >> (8 * (b % 4)) & 255) - 127
        v[:, 128 * b:128 * b + 128] *= torch.exp2(power.double())[:, None]
    return v


def _exact_ff(state):
    c = state["case"]
    x, wg, wu = (state[k].double() for k in ("x", "wg", "wu"))
    f = torch.nn.functional
    act = {"silu": f.silu, "gelu": f.gelu, "gelu_tanh": lambda z: f.gelu(z, approximate="tanh"),
           "relu": f.relu}[c["act"]]
    if not c["back"]:
        g, u = x @ wg, x @ wu
        h = act(g) * u
        return [h, g, u] if c["keep"] else h
    g, u = state["g"].double().requires_grad_(), state["u"].double().requires_grad_()
    dg, du = torch.autograd.grad(act(g) * u, (g, u), state["gh"].double())
    return [torch.cat([dg, du], 1) @ torch.cat([wg, wu], 1).T, (dg.T @ x).T, (du.T @ x).T]


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(state)
    if case["op"] == "ff":
        return _exact_ff(state)
    x = _exact_matrix(*state["x"]) if case["given"] else _exact_block_values(state["x"].double())
    return (_exact_matrix(*state["w"]) @ x.T).T
