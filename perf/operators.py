"""Timed cases of the operators around a cached attention layer: norm and
rotation of queries and keys (forward and backward), the 4-bit key/value cache
as it is written and read back, and attention over that cache.

`run` computes a case either in plain torch operations (`own` false) or with
this package's kernels (`own` true), from the same prepared state."""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------- cases

def listed():
    rope = dict(op="rope", back=False, sections="", pairs=False, norm=True, base=10000.0, far=0)
    kv = dict(op="kv4")
    att = dict(op="attn", causal=True, empty=False)
    return [
        # one decoding step of 32 sequences far into their contexts: latency
        dict(rope, name="rope_step", B=32, n=1, Hq=16, Hk=4, d=128, rot=128, dtype="bf16",
             order="bnhd", far=1000000),
        # the long-context workload's queries and keys, all tokens at once
        dict(rope, name="rope_long", B=2, n=32768, Hq=16, Hk=16, d=128, rot=128, dtype="bf16",
             order="bhnd"),
        # video tokens with time, height and width axes, odd count, fp32
        dict(rope, name="rope_axes", B=8, n=8190, Hq=8, Hk=8, d=64, rot=64, sections="8,12,12",
             pairs=True, dtype="f32", order="bnhd"),
        # training step at the clustered long-input workload's size
        dict(rope, name="rope_back", back=True, B=8, n=8192, Hq=8, Hk=8, d=64, rot=64,
             dtype="bf16", order="bhnd"),
        # training in fp32 on one short odd sequence, half of each head rotated
        dict(rope, name="rope_back_small", back=True, B=1, n=509, Hq=12, Hk=4, d=64, rot=32,
             dtype="f32", order="bnhd"),
        # a step's one token of each sequence into the cache, and back
        dict(kv, name="kv4_step", B=64, n=1, Hk=8, d=128, page=64, L=4096, dtype="bf16",
             order="bnhd"),
        # whole prompts into the cache, and back as attention inputs
        dict(kv, name="kv4_prompt", B=2, n=32765, Hk=16, d=128, page=64, L=0, dtype="bf16",
             order="bhnd"),
        # fp32 chunks that start and end inside pages
        dict(kv, name="kv4_chunk", B=8, n=1021, Hk=8, d=64, page=16, L=509, dtype="f32",
             order="bnhd"),
        # one token over a short context: latency
        dict(att, name="attn_short", B=1, n=1, Hq=16, Hk=4, d=128, page=64, L=512, ragged=False,
             dtype="bf16"),
        # one token of each sequence over long ragged contexts: bandwidth
        dict(att, name="attn_long", B=8, n=1, Hq=32, Hk=8, d=128, page=64, L=32768, ragged=True,
             dtype="bf16"),
        # a few drafted tokens over middling contexts in fp32
        dict(att, name="attn_draft", B=16, n=5, Hq=12, Hk=4, d=64, page=16, L=4095, ragged=True,
             dtype="f32"),
        # a prompt's chunk over what came before it: tensor cores
        dict(att, name="attn_chunk", B=2, n=1000, Hq=16, Hk=4, d=128, page=128, L=8192,
             ragged=False, dtype="bf16"),
    ]


def _cost(c):
    """Rough cost of the plain form: bytes moved by its intermediate tensors."""
    if c["op"] == "rope":
        return 60.0 * c["B"] * c["n"] * (c["Hq"] + c["Hk"]) * c["d"] * (2 if c["back"] else 1)
    if c["op"] == "kv4":
        return 60.0 * c["B"] * c["n"] * c["Hk"] * c["d"] * 2
    return (40.0 * c["B"] * c["L"] * c["Hk"] * c["d"] * 2 + 30.0 * c["B"] * c["Hq"] * c["n"] * c["L"]
            + c["B"] * c["Hq"] * c["n"] * c["L"] * c["d"] / 8)


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    most = {c["op"]: 0.0 for c in listed()}
    for c in listed():
        most[c["op"]] = max(most[c["op"]], _cost(c))
    while True:
        op = rng.choice(["rope", "rope", "kv4", "attn", "attn"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        if op == "rope":
            d = rng.choice([32, 64, 72, 96, 128, 128])
            rot = rng.choice([d, d, d // 2])
            axes = rng.choice([1, 1, 2, 3])
            sections = ""
            if axes > 1:
                half = rot // 2
                cut = sorted(rng.sample(range(1, half), axes - 1))
                sections = ",".join(str(b - a) for a, b in zip([0] + cut, cut + [half]))
            c = dict(op=op, back=rng.random() < 0.45, B=_log(rng, 1, 64), n=_log(rng, 1, 32768),
                     Hq=Hk * rng.choice([1, 1, 2, 4]), Hk=Hk, d=d, rot=rot, sections=sections,
                     pairs=rng.random() < 0.4, norm=rng.random() < 0.8,
                     base=rng.choice([10000.0, 500000.0]), far=rng.choice([0, 0, 100000, 20000000]),
                     dtype=dtype, order=rng.choice(["bnhd", "bhnd"]))
        elif op == "kv4":
            c = dict(op=op, B=_log(rng, 1, 64), n=_log(rng, 1, 32768), Hk=Hk,
                     d=rng.choice([32, 64, 128]), page=rng.choice([16, 32, 64, 128, 256]),
                     L=rng.choice([0, _log(rng, 1, 8192)]), dtype=dtype,
                     order=rng.choice(["bnhd", "bhnd"]))
        else:
            n = rng.choice([1, 1, 1, _log(rng, 2, 16), _log(rng, 17, 1024)])
            c = dict(op=op, B=_log(rng, 1, 64), n=n, Hq=Hk * rng.choice([1, 2, 3, 4, 7, 8]), Hk=Hk,
                     d=rng.choice([32, 64, 128, 128]), page=rng.choice([16, 32, 64, 128, 256]),
                     L=max(n, _log(rng, 16, 65536)), ragged=rng.random() < 0.6,
                     empty=rng.random() < 0.2, causal=rng.random() < 0.85, dtype=dtype)
        if _cost(c) <= most[op]:
            return c


# ------------------------------------------------------------------ inputs

def _seeds(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    return g, np.random.default_rng(seed * 7 + 3)


def _heads(g, B, H, n, d, dtype, order, spread=1.0):
    """[B, H, n, d] normal values, laid out token-major ("bnhd") or head-major."""
    shape = (B, n, H, d) if order == "bnhd" else (B, H, n, d)
    x = torch.empty(shape, dtype=DTYPES[dtype], device="cuda").normal_(0.0, spread, generator=g)
    return x.transpose(1, 2) if order == "bnhd" else x


def _like(x, B, H, n, d, order, value=0.0):
    shape = (B, n, H, d) if order == "bnhd" else (B, H, n, d)
    y = torch.full(shape, value, dtype=x.dtype, device="cuda")
    return y.transpose(1, 2) if order == "bnhd" else y


def _sections(c):
    return [int(s) for s in c["sections"].split(",")] if c["sections"] else [c["rot"] // 2]


def _lengths(c):
    """Cached tokens of each sequence, in an order the seed gives."""
    B, L = c["B"], c["L"]
    if not c["ragged"]:
        lens = [L] * B
    else:
        lens = [max(min(c["n"], L), L - (3 * L * b) // (4 * B)) for b in range(B)]
    if c["empty"]:
        lens[-1] = 0
    return lens


def _table(rs, B, per_seq):
    """Pages of a pool a little larger than needed, handed out in no order."""
    pool = B * per_seq + 3
    ids = rs.permutation(pool)[:B * per_seq].reshape(B, per_seq).astype(np.int32)
    return torch.from_numpy(ids).cuda(), pool


def _block_bytes(d):
    return 18 * d  # 16 tokens: K codes 8 d, K scales d, V codes 8 d, V scales d


def prepare(case, seed):
    c = case
    g, rs = _seeds(c, seed)
    B, n, d = c["B"], c["n"], c["d"]
    if c["op"] == "rope":
        sec = _sections(c)
        q = _heads(g, B, c["Hq"], n, d, c["dtype"], c["order"])
        k = _heads(g, B, c["Hk"], n, d, c["dtype"], c["order"])
        start = torch.from_numpy(rs.integers(c["far"] // 2, c["far"] + 1, size=(B, 1))).cuda()
        t = torch.arange(n, device="cuda")
        if len(sec) == 1:
            pos = (start + t)[None]
        else:  # a grid 24 wide and, with three axes, 16 high
            frame = 24 if len(sec) == 2 else 24 * 16
            pos = torch.stack([start + t // frame] + ([(t % frame // 24).expand(B, n)] if len(sec) == 3 else [])
                              + [(t % 24).expand(B, n)])
        st = dict(case=c, q=q, k=k, positions=pos.to(torch.int32).contiguous(),
                  inv_freq=c["base"] ** (-np.arange(c["rot"] // 2, dtype=np.float64) * 2 / c["rot"]),
                  sections=sec, q_weight=None, k_weight=None)
        if c["norm"]:
            st["q_weight"] = 1 + 0.2 * torch.randn(d, device="cuda", generator=g)
            st["k_weight"] = 1 + 0.2 * torch.randn(d, device="cuda", generator=g)
        if c["back"]:
            st["gq"] = _heads(g, B, c["Hq"], n, d, c["dtype"], c["order"])
            st["gk"] = _heads(g, B, c["Hk"], n, d, c["dtype"], c["order"])
        return st
    Hk, P = c["Hk"], c["page"]
    if c["op"] == "kv4":
        per_seq = -(-(c["L"] + n) // P)
        table, pool = _table(rs, B, per_seq)
        starts = rs.integers(0, c["L"] + 1, size=B).astype(np.int32)
        counts = rs.integers((n + 1) // 2, n + 1, size=B).astype(np.int32)
        counts[0] = n
        k = _heads(g, B, Hk, n, d, c["dtype"], c["order"])
        v = _heads(g, B, Hk, n, d, c["dtype"], c["order"])
        # keys have a few large channels, values now and then a large token
        k *= 1 + 6 * (torch.rand(Hk, 1, d, device="cuda", generator=g) > 0.95).to(k.dtype)
        v *= 1 + 4 * (torch.rand(B, 1, n, 1, device="cuda", generator=g) > 0.98).to(v.dtype)
        cache = torch.randint(0, 256, (pool * Hk * (P // 16) * _block_bytes(d),), dtype=torch.uint8,
                              device="cuda", generator=g)
        return dict(case=c, k=k, v=v, cache=cache, table=table, starts=torch.from_numpy(starts).cuda(),
                    counts=torch.from_numpy(counts).cuda(), k_back=_like(k, B, Hk, n, d, c["order"]),
                    v_back=_like(v, B, Hk, n, d, c["order"]))
    lens = np.array(_lengths(c), dtype=np.int32)
    rs.shuffle(lens)
    per_seq = -(-c["L"] // P)
    table, pool = _table(rs, B, per_seq)
    # Codes of normal values in blocks of 32 hardly favour any level, so the
    # pages hold random codes 1..15; the scales are those of normal values.
    shape = (pool, Hk, P // 16)
    lo = torch.randint(1, 16, shape + (2, 8 * d), dtype=torch.uint8, device="cuda", generator=g)
    hi = torch.randint(1, 16, shape + (2, 8 * d), dtype=torch.uint8, device="cuda", generator=g)
    scale = 0.22 + 0.25 * torch.rand(shape + (2, d // 2), device="cuda", generator=g)
    scale = scale.to(torch.bfloat16).view(torch.uint8)
    cache = torch.cat([lo | (hi << 4), scale], dim=-1)  # (..., K or V, codes and scales)
    # what no token has been written to yet is whatever the memory held
    tail = torch.from_numpy(lens).cuda().long() // P
    last = table[torch.arange(B, device="cuda"), tail.clamp(max=per_seq - 1)].long()
    keep = (torch.from_numpy(lens).cuda() % P // 16 + 1)[:, None] > torch.arange(P // 16, device="cuda")
    junk = torch.where(keep[:, None, :, None, None] | (tail >= per_seq)[:, None, None, None, None],
                       cache[last], torch.full_like(cache[last], 0xFF))
    cache[last] = junk
    q = _heads(g, B, c["Hq"], n, d, c["dtype"], "bnhd", 0.5)
    return dict(case=c, cache=cache.reshape(-1), table=table, lengths=torch.from_numpy(lens).cuda(), q=q,
                out=_like(q, B, c["Hq"], n, d, "bnhd"))


# -------------------------------------------------------------- plain forms

def _angles(state):
    """cos, sin [B, 1, n, rot/2] of position times frequency, in 64 bits."""
    c = state["case"]
    axis = torch.repeat_interleave(torch.arange(len(state["sections"]), device="cuda"),
                                   torch.tensor(state["sections"], device="cuda"))
    pos = state["positions"].double()[axis].permute(1, 2, 0)  # [B, n, rot/2]
    a = pos * torch.from_numpy(state["inv_freq"]).cuda()
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _split(x, c):
    """First and second members of the rotated pairs, and the rest."""
    r = x[..., :c["rot"]]
    if c["pairs"]:
        return r[..., 0::2], r[..., 1::2], x[..., c["rot"]:]
    return r[..., :c["rot"] // 2], r[..., c["rot"] // 2:], x[..., c["rot"]:]


def _join(a, b, rest, c):
    r = torch.stack([a, b], dim=-1).flatten(-2) if c["pairs"] else torch.cat([a, b], dim=-1)
    return torch.cat([r, rest], dim=-1)


def _plain_rope_one(x, w, cos, sin, c):
    y = x.float()
    if c["norm"]:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w
    a, b, rest = _split(y, c)
    return _join(a * cos - b * sin, b * cos + a * sin, rest, c).to(x.dtype)


def _plain_rope_back(x, w, gy, cos, sin, c):
    a, b, rest = _split(gy.float(), c)
    gz = _join(a * cos + b * sin, b * cos - a * sin, rest, c)
    if not c["norm"]:
        return gz.to(x.dtype), None
    xf = x.float()
    r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + 1e-6)
    hat = xf * r
    gw = (gz * hat).sum(dim=(0, 1, 2), dtype=torch.float64).float()
    gh = gz * w
    return (r * (gh - hat * (gh * hat).mean(-1, keepdim=True))).to(x.dtype), gw


def _plain_quantised(x):
    """The values 4 bits and a scale for every 32 channels stand for."""
    s32 = x.float().unflatten(-1, (-1, 32))
    scale = s32.abs().amax(-1, keepdim=True) / 7
    scale = (scale.view(torch.int32) & -65536).view(torch.float32)  # bf16, towards zero
    code = torch.where(scale > 0, torch.round(s32.double() / scale.double()), 0.0).clamp(-7, 7)
    return (code.float() * scale).flatten(-2).to(x.dtype)


def _plain_unpacked(state):
    """Keys and values [B, Hk, tokens, d] in 32 bits of the pages of each sequence."""
    c = state["case"]
    B, Hk, d, P = c["B"], c["Hk"], c["d"], c["page"]
    G = d // 32
    blocks = state["cache"].view(-1, Hk, P // 16, 18 * d)[state["table"].long()]
    blocks = blocks.permute(0, 2, 1, 3, 4).reshape(B, Hk, -1, 18 * d)  # 16-token blocks in order

    def scaled(codes, scales):  # codes [B, Hk, blk, 16, G, 16 bytes], scales [.., G, 16]
        both = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)  # [.., 16, G, 32]
        s = scales.contiguous().view(torch.bfloat16).float().unflatten(-1, (G, 16)).transpose(-1, -2)
        return ((both.float() - 8) * s[..., None]).flatten(-2).flatten(2, 3)

    kc = blocks[..., :8 * d].unflatten(-1, (16, 4, G, 4)).transpose(-3, -2).flatten(-2)
    vc = blocks[..., 9 * d:17 * d].unflatten(-1, (2, 8, 4, 2, G, 2))
    vc = vc.permute(0, 1, 2, 3, 5, 6, 7, 4, 8).flatten(-2).flatten(3, 5)
    return scaled(kc, blocks[..., 8 * d:9 * d]), scaled(vc, blocks[..., 17 * d:])


def _plain_attention(state):
    c = state["case"]
    k, v = _plain_unpacked(state)
    B, Hk, T, d = k.shape
    n, rep = c["n"], c["Hq"] // Hk
    lens = state["lengths"].long()
    key = torch.arange(T, device="cuda")
    held = key < lens[:, None]  # [B, T]
    k = torch.where(held[:, None, :, None], k, 0.0)
    v = torch.where(held[:, None, :, None], v, 0.0)
    last = lens[:, None] - n + torch.arange(n, device="cuda") if c["causal"] else (lens - 1)[:, None].expand(B, n)
    seen = held[:, None, :] & (key <= last[..., None])  # [B, n, T]
    q = state["q"].float().reshape(B, Hk, rep, n, d)
    s = (q.flatten(2, 3) @ k.transpose(-1, -2)).unflatten(2, (rep, n)) * (1 / math.sqrt(d))
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (rep, n)) / torch.where(total == 0, 1.0, total)
    return o.reshape(B, c["Hq"], n, d).to(state["q"].dtype)


def run(state):
    c = state["case"]
    if c["op"] == "rope":
        return _run_rope(state)
    if c["op"] == "kv4":
        if own:
            import nystr_self_attention_gb300 as N
            cache = N.NystromKv4Cache(state["cache"], state["table"], c["page"], c["Hk"], c["d"])
            N.nystrom_kv4_write(cache, state["k"], state["v"], state["starts"], state["counts"])
            N.nystrom_kv4_read(cache, state["k_back"], state["v_back"], state["starts"], state["counts"])
            return [state["k_back"], state["v_back"]]
        live = (torch.arange(c["n"], device="cuda") < state["counts"][:, None])[:, None, :, None]
        return [torch.where(live, _plain_quantised(state["k"]), state["k_back"]),
                torch.where(live, _plain_quantised(state["v"]), state["v_back"])]
    if own:
        import nystr_self_attention_gb300 as N
        cache = N.NystromKv4Cache(state["cache"], state["table"], c["page"], c["Hk"], c["d"])
        N.nystrom_kv4_attn_fwd(cache, state["q"], state["out"], state["lengths"], c["L"], causal=c["causal"])
        return state["out"]
    return _plain_attention(state)


def _run_rope(state):
    c = state["case"]
    q, k, qw, kw = state["q"], state["k"], state["q_weight"], state["k_weight"]
    if own:
        import nystr_self_attention_gb300 as N
        args = dict(sections=state["sections"], norm=c["norm"], eps=1e-6,
                    pairing=N.NYS_ROPE_PAIRS if c["pairs"] else N.NYS_ROPE_HALVES)
        a, b = torch.empty_like(q), torch.empty_like(k)
        if not c["back"]:
            N.nystrom_qk_norm_rope_fwd(q, k, a, b, state["positions"], state["inv_freq"], qw, kw, **args)
            return [a, b]
        gqw, gkw = (torch.empty_like(qw), torch.empty_like(kw)) if c["norm"] else (None, None)
        N.nystrom_qk_norm_rope_bwd(q, k, state["gq"], state["gk"], a, b, state["positions"],
                                   state["inv_freq"], qw, kw, gqw, gkw, **args)
        return [a, b, gqw, gkw] if c["norm"] else [a, b]
    cos, sin = _angles(state)
    if not c["back"]:
        return [_plain_rope_one(q, qw, cos, sin, c), _plain_rope_one(k, kw, cos, sin, c)]
    gq, gqw = _plain_rope_back(q, qw, state["gq"], cos, sin, c)
    gk, gkw = _plain_rope_back(k, kw, state["gk"], cos, sin, c)
    return [gq, gk, gqw, gkw] if c["norm"] else [gq, gk]


# ------------------------------------------------------------ work and truth

def work(case):
    c, e = case, ESIZE[case["dtype"]]
    B, n, d = c["B"], c["n"], c["d"]
    if c["op"] == "rope":
        rows = B * n * (c["Hq"] + c["Hk"])
        return {"bytes": rows * d * e * (3 if c["back"] else 2) + 4 * B * n * len(_sections(c))
                + (16.0 * d if c["norm"] else 0),
                "flops": rows * d * (16.0 if c["back"] else 8.0)}
    if c["op"] == "kv4":
        # on average three quarters of the padded rows are tokens
        rows = c["Hk"] * 2 * (n + (B - 1) * 0.75 * n)
        return {"bytes": rows * d * (2 * e + 2 * 9 / 16), "flops": rows * d * 6.0}
    lens = _lengths(c)
    pairs = sum(sum(max(0, min(x, x - n + 1 + i)) for i in range(n)) if c["causal"] else x * n for x in lens)
    return {"bytes": 2.0 * B * c["Hq"] * n * d * e + sum(lens) * c["Hk"] * d * 18 / 16,
            "flops": 4.0 * c["Hq"] * d * pairs}


def _exact_rope(state, back):
    """Complex rotation in 64 bits; the gradients come from its differentiation."""
    c = state["case"]
    half = c["rot"] // 2
    parts, at = [], 0
    for a, width in enumerate(state["sections"]):
        f = torch.tensor([c["base"] ** (-2.0 * i / c["rot"]) for i in range(at, at + width)],
                         dtype=torch.float64, device="cuda")
        parts.append(state["positions"][a].double()[..., None] * f)
        at += width
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.cat(parts, -1))
    outs, grads = [], []
    for x, w, gy in ((state["q"], state["q_weight"], state.get("gq")),
                     (state["k"], state["k_weight"], state.get("gk"))):
        x = x.double().requires_grad_(back)
        z, leaves = x, [x]
        if c["norm"]:
            w = w.double().requires_grad_(back)
            leaves.append(w)
            z = w * x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["d"] + 1e-6)
        idx = torch.arange(c["rot"], device="cuda").view(half, 2) if c["pairs"] else \
            torch.arange(c["rot"], device="cuda").view(2, half).T
        first, second = idx[:, 0].contiguous(), idx[:, 1].contiguous()
        spun = torch.complex(z[..., first], z[..., second]) * turn[:, None]
        y = z.index_copy(-1, first, spun.real).index_copy(-1, second, spun.imag)
        if back:
            grads.append(torch.autograd.grad(y, leaves, gy.double()))
        else:
            outs.append(y)
    if not back:
        return outs
    return [g[0] for g in grads] + ([g[1] for g in grads] if c["norm"] else [])


def _exact_kv4(state):
    c, outs = state["case"], []
    for x, was in ((state["k"], state["k_back"]), (state["v"], state["v_back"])):
        y = was.double().clone()
        for b in range(c["B"]):
            m = int(state["counts"][b])
            for j in range(0, c["d"], 32):
                part = x[b, :, :m, j:j + 32].double()
                top = part.abs().max(-1, keepdim=True).values.float()
                exponent = torch.floor(torch.log2((top / 7).double()))
                step = torch.exp2(exponent - 7)  # bf16 has 8 significant bits
                scale = torch.floor((top / 7).double() / step) * step
                level = torch.clamp(torch.round(part / scale), -7, 7)
                y[b, :, :m, j:j + 32] = torch.where(top > 0, level * scale, 0.0)
        outs.append(y)
    return outs


def _exact_attention(state):
    c = state["case"]
    d, Hk, P, n, rep = c["d"], c["Hk"], c["page"], c["n"], c["Hq"] // c["Hk"]
    raw = state["cache"]
    ch = torch.arange(d, device="cuda")
    grp, within = ch // 32, ch % 32
    out = torch.zeros(c["B"], c["Hq"], n, d, dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        m = int(state["lengths"][b])
        if m == 0:
            continue
        tok = torch.arange(m, device="cuda")
        page = state["table"][b].long()[tok // P]
        r = (tok % 16)[:, None]
        for h in range(Hk):
            base = (((page * Hk + h) * (P // 16) + tok % P // 16) * (18 * d))[:, None]

            def value(codes_at, byte, scales_at):
                code = (raw[base + codes_at + byte].long() >> (4 * (ch % 2))) & 15
                at = base + scales_at + (grp * 16 + r) * 2
                bits = raw[at].int() | (raw[at + 1].int() << 8)
                return (code - 8).double() * (bits << 16).view(torch.float32).double()

            k = value(0, r * (d // 2) + (within // 8) * (d // 8) + grp * 4 + within % 8 // 2, 8 * d)
            v = value(9 * d, r // 8 * 4 * d + ((within // 4) * 4 + r % 8 // 2) * (d // 8) + r % 2 * (d // 16)
                      + grp * 2 + within % 4 // 2, 17 * d)
            q = state["q"][b, h * rep:(h + 1) * rep].double()
            s = q @ k.T / math.sqrt(d)
            if c["causal"]:
                late = tok[None] > (m - n + torch.arange(n, device="cuda"))[:, None]
                s = torch.where(late, -math.inf, s)
            p = torch.nan_to_num(torch.softmax(s, -1), nan=0.0)  # a row that sees no key
            out[b, h * rep:(h + 1) * rep] = p @ v
    return out


def exact(case, seed):
    if case["op"] == "attn" and case["B"] * case["Hk"] > 600:
        return None
    state = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(state, case["back"])
    return _exact_kv4(state) if case["op"] == "kv4" else _exact_attention(state)
