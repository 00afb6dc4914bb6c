"""Plain numpy restatement, in 64 bits, of the norm and rotation of query and
key heads and of attention over the values a 4-bit cache stands for; the stored
bits of that cache are defined by fp32 operations, restated here one by one.
Test infrastructure only; it shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np

GROUP = 32


def norm_rope(x, weight, pos, inv_freq, rot_dim, interleaved, eps):
    """x [T, H, D] -> (y, per-element |a| + |b| of the rotated pair, or |y|), float64."""
    y = np.asarray(x, np.float64)
    if weight is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    out, mag = y.copy(), np.abs(y)
    for i in range(rot_dim // 2):
        u = np.asarray(pos, np.float64) * float(inv_freq[i])
        c, s = np.cos(u)[:, None], np.sin(u)[:, None]
        p, r = (2 * i, 2 * i + 1) if interleaved else (i, i + rot_dim // 2)
        a, b = y[..., p], y[..., r]
        out[..., p], out[..., r] = a * c - b * s, b * c + a * s
        mag[..., p] = mag[..., r] = np.abs(a) + np.abs(b)
    return out, mag


def _cut16(x32, bf16):
    """fp32 cut toward zero to a 16-bit type, as fp32."""
    if bf16:
        return (x32.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
    with np.errstate(over="ignore"):
        h = x32.astype(np.float16)
    up = h.astype(np.float32) > x32
    return np.where(up, (h.view(np.uint16) - up.astype(np.uint16)).view(np.float16), h).astype(np.float32)


def store(x, bf16):
    """Rows [..., D] (values of the layer's type) -> codes [..., D], scale and smallest value [..., D / 32], fp32."""
    g = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)
        span = hi - lo
        ok = np.isfinite(g).all(-1) & np.isfinite(span)
        s = _cut16(span / np.float32(15), bf16)
        safe = np.where(ok & (s > 0), s, np.float32(1))
        c = np.minimum(np.rint((g - lo[..., None]) / safe[..., None]), 15)
    c = np.where((ok & (s > 0))[..., None], c, 0)
    return c.reshape(x.shape).astype(np.int64), np.where(ok, s, np.float32(np.nan)), lo


def values(codes, scale, lo):
    """What codes [..., D] stand for, before the last rounding, float64."""
    g = codes.reshape(*codes.shape[:-1], -1, GROUP).astype(np.float64)
    v = np.asarray(lo, np.float64)[..., None] + g * np.asarray(scale, np.float64)[..., None]
    return v.reshape(codes.shape)


def unpack(code_bytes):
    """uint8 [..., D / 2] -> codes [..., D]: channel 8w + 2i at bit 4i of word w, channel 8w + 2i + 1 at 16 + 4i."""
    w = np.ascontiguousarray(code_bytes).view("<u4")
    out = np.empty((*w.shape, 8), np.int64)
    for i in range(4):
        out[..., 2 * i] = (w >> np.uint32(4 * i)) & 15
        out[..., 2 * i + 1] = (w >> np.uint32(16 + 4 * i)) & 15
    return out.reshape(*code_bytes.shape[:-1], -1)


def attention(q, k, v, past, scale):
    """q [R, Hq, D] at positions past + i over k, v [n, Hkv, D] -> (out, sum_j p_j |v_j|), float64."""
    r, hq, d = q.shape
    group = hq // k.shape[1]
    out, mag = np.empty((r, hq, d)), np.empty((r, hq, d))
    hide = np.arange(k.shape[0])[None] > past + np.arange(r)[:, None]
    for h in range(hq):
        s = (q[:, h] @ k[:, h // group].T) * scale
        s[hide] = -np.inf
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        out[:, h], mag[:, h] = p @ v[:, h // group], p @ np.abs(v[:, h // group])
    return out, mag
