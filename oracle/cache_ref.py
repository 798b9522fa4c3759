"""fp64 numpy reference of the operators around a cached attention layer: norm
and rotation of queries and keys with their gradients, the 4-bit key/value
cache byte by byte, attention over it. Written from the formulas in
include/nystrom.h; shares no code with the library."""
import math

import numpy as np

BLOCK = 16


# ------------------------------------------------------- norm and rotation

def rope_pairs(rot, pairs):
    """[(a, b)] channels of the rotated pairs."""
    half = rot // 2
    return [(2 * i, 2 * i + 1) if pairs else (i, i + half) for i in range(half)]


def rope_angles(positions, inv_freq, sections):
    """Angles [B, n, rot/2] in fp64: positions [axes, B, n]."""
    axis = [a for a, s in enumerate(sections) for _ in range(s)]
    pos = np.asarray(positions, dtype=np.float64)
    return np.stack([pos[a] * float(f) for a, f in zip(axis, inv_freq)], axis=-1) if axis else \
        np.zeros(pos.shape[1:] + (0,))


def norm_rows(x, w, eps):
    x = np.asarray(x, dtype=np.float64)
    return w * (x / np.sqrt((x * x).mean(-1, keepdims=True) + eps))


def rotate(z, angles, pairs):
    """z [B, H, n, d]; the inverse rotation is that of -angles."""
    y = np.array(z, dtype=np.float64)
    for i, (a, b) in enumerate(rope_pairs(2 * angles.shape[-1], pairs)):
        c, s = np.cos(angles[:, None, :, i]), np.sin(angles[:, None, :, i])
        y[..., a] = z[..., a] * c - z[..., b] * s
        y[..., b] = z[..., b] * c + z[..., a] * s
    return y


def qk_norm_rope(x, w, angles, pairs, norm=True, eps=1e-6):
    return rotate(norm_rows(x, w, eps) if norm else np.asarray(x, np.float64), angles, pairs)


def qk_norm_rope_grad(x, w, gy, angles, pairs, norm=True, eps=1e-6):
    """(dx, dw): dw None without the norm."""
    g = rotate(np.asarray(gy, np.float64), -angles, pairs)
    if not norm:
        return g, None
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h = x * r
    dw = (g * h).sum(axis=(0, 1, 2))
    wg = w * g
    return r * (wg - h * (wg * h).mean(-1, keepdims=True)), dw


# ------------------------------------------------------------- 4-bit cache

def bf16_bits_toward_zero(x):
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def bf16_value(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def quantise(x):
    """x [..., d] (float32 values) -> codes int [..., d], scale bits uint16
    [..., d/32]."""
    x = np.asarray(x, np.float32)
    g = x.reshape(x.shape[:-1] + (-1, 32))
    top = np.abs(g).max(-1)
    bad = ~np.isfinite(g).all(-1)
    with np.errstate(invalid="ignore", over="ignore"):
        bits = bf16_bits_toward_zero((top * np.float32(1 / 7)).astype(np.float32))
    bits = np.where(bad, np.uint16(0x7FC0), bits)
    s = bf16_value(bits)
    zero = bad | (bits == 0)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.rint(g.astype(np.float64) / np.where(zero, 1.0, s)[..., None])
    q = np.where(zero[..., None], 0, np.clip(np.nan_to_num(q), -7, 7)).astype(np.int64)
    return q.reshape(x.shape), bits


def dequantise(codes, bits):
    s = np.repeat(bf16_value(bits), 32, axis=-1)
    return codes * s


def key_byte(r, c, d):
    w = c % 32
    return r * (d // 2) + (w // 8) * (d // 8) + 4 * (c // 32) + (w % 8) // 2


def value_byte(r, c, d):
    w = c % 32
    return ((r // 8) * 4 * d + ((w // 4) * 4 + (r % 8) // 2) * (d // 8) + (r % 2) * (d // 16)
            + 2 * (c // 32) + (w % 4) // 2)


class Cache:
    """The pool as bytes [num_pages, Hk, page/16, 18 d], written and read one
    token at a time."""

    def __init__(self, raw, table, page, Hk, d):
        self.raw = np.array(raw, dtype=np.uint8).reshape(-1, Hk, page // BLOCK, 18 * d)
        self.table, self.page, self.Hk, self.d = np.asarray(table), page, Hk, d
        c = np.arange(d)
        self.kb = np.stack([key_byte(r, c, d) for r in range(BLOCK)])
        self.vb = np.stack([value_byte(r, c, d) for r in range(BLOCK)])

    def block(self, b, pos):
        """[Hk, 18 d] view, or None."""
        if pos < 0 or pos // self.page >= self.table.shape[1]:
            return None
        pg = int(self.table[b, pos // self.page])
        if not 0 <= pg < self.raw.shape[0]:
            return None
        return self.raw[pg, :, pos % self.page // BLOCK]

    def _put(self, blk, at, r, codes, bits, bytes_of):
        d = self.d
        for c in range(d):
            i = at + bytes_of[r, c]
            field = (codes[:, c] + 8).astype(np.uint8)
            blk[:, i] = (blk[:, i] & 0xF0 | field) if c % 2 == 0 else (blk[:, i] & 0x0F | field << 4)
        for y in range(d // 32):
            i = at + 8 * d + (y * BLOCK + r) * 2
            blk[:, i] = bits[:, y] & 255
            blk[:, i + 1] = bits[:, y] >> 8

    def _get(self, blk, at, r, bytes_of):
        d = self.d
        byte = blk[:, at + bytes_of[r]].astype(np.int64)
        codes = (byte >> (4 * (np.arange(d) % 2)) & 15) - 8
        i = at + 8 * d + (np.arange(d // 32) * BLOCK + r) * 2
        return dequantise(codes, blk[:, i].astype(np.uint16) | blk[:, i + 1].astype(np.uint16) << 8)

    def write(self, k, v, starts, counts):
        """k, v [B, Hk, n, d]."""
        kc, kbits = quantise(k)
        vc, vbits = quantise(v)
        for b in range(k.shape[0]):
            for i in range(max(0, min(int(counts[b]), k.shape[2]))):
                pos = int(starts[b]) + i
                blk = self.block(b, pos)
                if blk is None:
                    continue
                self._put(blk, 0, pos % BLOCK, kc[b, :, i], kbits[b, :, i], self.kb)
                self._put(blk, 9 * self.d, pos % BLOCK, vc[b, :, i], vbits[b, :, i], self.vb)

    def token(self, b, pos):
        """(K, V) [Hk, d] of one token; None where there is no page."""
        blk = self.block(b, pos)
        if blk is None:
            return None
        r = pos % BLOCK
        return self._get(blk, 0, r, self.kb), self._get(blk, 9 * self.d, r, self.vb)


def attention(q, cache, lengths, counts=None, causal=True, scale=None):
    """out [B, Hq, nq, d] (rows past a count: 0), with `spread` = sum p |v| and
    `reach` = the largest sum |q k| scale of a row's keys, the quantities that
    rounding errors scale with."""
    q = np.asarray(q, np.float64)
    B, Hq, nq, d = q.shape
    rep = Hq // cache.Hk
    scale = 1 / math.sqrt(d) if scale is None else scale
    out, spread = np.zeros_like(q), np.zeros_like(q)
    reach = np.zeros((B, Hq, nq, 1))
    for b in range(B):
        n = int(lengths[b])
        toks = [cache.token(b, t) for t in range(n)]
        there = [t for t in range(n) if toks[t] is not None]
        cnt = nq if counts is None else int(counts[b])
        for i in range(cnt):
            seen = [t for t in there if not causal or t <= n - cnt + i]
            if not seen:
                continue
            K = np.stack([toks[t][0] for t in seen], 1)  # [Hk, keys, d]
            V = np.stack([toks[t][1] for t in seen], 1)
            for h in range(Hq):
                s = K[h // rep] @ q[b, h, i] * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                out[b, h, i] = p @ V[h // rep]
                spread[b, h, i] = p @ np.abs(V[h // rep])
                reach[b, h, i] = (np.abs(K[h // rep]) @ np.abs(q[b, h, i])).max() * abs(scale)
    return out, spread, reach
