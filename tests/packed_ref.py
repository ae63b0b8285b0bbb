"""Plain 64-bit references of the projection step (norm, rotation, layout) and of the 4-bit
packed history, written from their formulas in numpy; the attention over unpacked values is
checked by the fp64 oracle."""
from __future__ import annotations

import numpy as np

CHUNK = 64
U32 = 2.0 ** -24  # half a step of fp32, relative
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}  # half a step of an output


# ------------------------------------------------------------------ norm and rotation
def rope_table(theta, rot, n_pos):
    i = np.arange(rot // 2, dtype=np.float64)
    ang = np.arange(n_pos, dtype=np.float64)[:, None] * theta ** (-2.0 * i / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)


def norm_rope(x, w, cs, rot, eps):
    """x [..., S, D] head rows, cs [..., S, R]: the rows and, per output, the sum of the
    magnitudes of its two products (what its fp32 roundings are relative to)."""
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    n = x * r * w
    h = rot // 2
    c, s = cs[..., :h], cs[..., h:]
    a, b = n[..., :h], n[..., h:rot]
    y = np.concatenate([a * c - b * s, b * c + a * s, n[..., rot:]], axis=-1)
    mag = np.concatenate([abs(a * c) + abs(b * s), abs(b * c) + abs(a * s), abs(n[..., rot:])], axis=-1)
    return y, mag


def norm_rope_bwd(x, w, cs, rot, eps, dy):
    """dx, the magnitude its roundings are relative to, and per row dn * xh with the magnitude
    of its products."""
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    h = rot // 2
    c, s = cs[..., :h], cs[..., h:]
    a, b = dy[..., :h], dy[..., h:rot]
    dn = np.concatenate([a * c + b * s, b * c - a * s, dy[..., rot:]], axis=-1)
    dmag = np.concatenate([abs(a * c) + abs(b * s), abs(b * c) + abs(a * s), abs(dy[..., rot:])], axis=-1)
    xh = x * r
    g, gmag = dn * w, dmag * abs(w)
    dx = r * (g - xh * np.mean(g * xh, axis=-1, keepdims=True))
    mag = r * (gmag + abs(xh) * np.mean(gmag * abs(xh), axis=-1, keepdims=True))
    return dx, mag, dn * xh, dmag * abs(xh)


# ------------------------------------------------------------------ 4-bit records
def to_bf16(x):
    """float64 -> nearest bf16 value, ties to even, one rounding (NaN and infinities kept)."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(np.where(np.isfinite(x), x, 0.0))
    y = np.ldexp(np.rint(np.ldexp(m, 8)), e - 8)
    return np.where(np.isfinite(x), y, x)


def bf16_bits(x):
    """Bits of bf16 values; a NaN is 0x7FFF, as CUDA's conversion writes it."""
    x = np.asarray(x, dtype=np.float32)
    return np.where(np.isnan(x), 0x7FFF, x.view(np.uint32) >> 16).astype(np.uint16)


def quant(x, axis):
    """Grid (s, z) and codes of x (bf16 or fp32 values as float64) in groups along axis."""
    with np.errstate(all="ignore"):
        mn, mx = x.min(axis, keepdims=True), x.max(axis, keepdims=True)
        spread = (mx - mn).astype(np.float32)  # rounded to fp32, as are 1/15 and the product
        s = to_bf16((spread * np.float32(1 / 15)).astype(np.float64))
        s = np.where(s < 2.0 ** -100, 0.0, s)
        z = to_bf16((mn - 16 * s).astype(np.float32).astype(np.float64))
        bad = ~np.isfinite(x).all(axis, keepdims=True) | ~np.isfinite(s) | ~np.isfinite(z)
        s, z = np.where(bad, np.nan, s), np.where(bad, np.nan, z)
        c = np.clip(np.rint((x - z) / np.where(s == 0, 1.0, s)), 16, 31) - 16
        c = np.where((s == 0) | bad, 0, c).astype(np.int64)
    return s, z, c


def values(s, z, c):
    return to_bf16(s * (16.0 + c) + z)


_SHIFT = np.array([0, 16, 4, 20, 8, 24, 12, 28], dtype=np.uint32)


def _words(c):
    return np.bitwise_or.reduce(c.astype(np.uint32) << _SHIFT, axis=-1)


def _bytes(a, lead):
    return np.ascontiguousarray(a).reshape(*lead, -1).view(np.uint8)


def pack(k, v):
    """k, v float64 [B][H][n * 64][D] -> records uint8 [B][H][n][72 D] and their values."""
    B, H, T, D = k.shape
    n = T // CHUNK
    lead = (B, H, n)
    s, z, c = quant(k.reshape(B, H, n, CHUNK, D), 3)
    kv = values(s, z, c).reshape(k.shape)
    parts = [_bytes(_words(c.reshape(B, H, n, CHUNK, D // 8, 8)), lead), _bytes(bf16_bits(s), lead),
             _bytes(bf16_bits(z), lead)]
    s, z, c = quant(v.reshape(B, H, n, CHUNK, D // 64, 64), 5)
    vv = values(s, z, c).reshape(v.shape)
    ct = c.reshape(B, H, n, CHUNK, D).swapaxes(3, 4).reshape(B, H, n, D, 8, 8)
    parts += [_bytes(_words(ct), lead), _bytes(bf16_bits(s[..., 0].swapaxes(3, 4)), lead),
              _bytes(bf16_bits(z[..., 0].swapaxes(3, 4)), lead)]
    return np.concatenate(parts, axis=-1), kv, vv


# ------------------------------------------------------------------ attention
def attend(q, keys, vals, mask):
    """q [R][D], keys / vals [T][D], mask [R or 1][T] (float64): out, lse, the magnitude
    sum_t p_t |v_t| of every output, and the largest sum_i |q_i k_i| / sqrt(D) of a row."""
    scale = q.shape[-1] ** -0.5
    x = np.where(mask, (q @ keys.T) * scale, -np.inf)
    top = x.max(-1, keepdims=True)
    p = np.exp(x - top)
    l = p.sum(-1, keepdims=True)
    p /= l
    size = np.where(mask, (abs(q) @ abs(keys).T) * scale, 0.0).max(-1, keepdims=True)
    return p @ vals, (top + np.log(l))[..., 0], p @ abs(vals), size


def attend_tol(out, mag, size, d, n):
    """Bounds of bf16 attention over n tokens with fp32 sums.  A score is d products and sums
    whose additions may truncate (2 u each) and a scaling, its exponential has the same
    absolute error and 4 u of its own; the row sum and the products over P add n truncating
    sums; P and the output are rounded to bf16."""
    score = (2 * d + 8) * U32 * size
    rel = 2 * score + (4 * n + 64) * U32
    return HALF["bf16"] * abs(out) + (HALF["bf16"] + rel) * mag, rel[..., 0]
