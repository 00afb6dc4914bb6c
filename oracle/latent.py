"""Plain numpy restatement, in 64 bits, of latent caches and drafted trees:
norm and rotation of the appended rows, what a row sees, and attention.  Test
infrastructure only; it shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np


def norm(x, weight, eps):
    """Root-mean-square norm of rows [T, C], float64."""
    y = np.asarray(x, np.float64)
    if weight is None:
        return y
    return y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def rotate(x, pos, inv_freq, rot, interleaved):
    """x [T, H, R] -> (rotated, per-element |a| + |b| of its pair), float64."""
    y = np.asarray(x, np.float64)
    out, mag = y.copy(), np.zeros_like(y)
    for i in range(rot // 2):
        u = np.asarray(pos, np.float64) * float(inv_freq[i])
        c, s = np.cos(u)[:, None], np.sin(u)[:, None]
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = y[..., p], y[..., q]
        out[..., p], out[..., q] = a * c - b * s, b * c + a * s
        mag[..., p] = mag[..., q] = np.abs(a) + np.abs(b)
    return out, mag


def sees(rows, past, parents=None):
    """[rows, past + rows]: the positions that each row sees; parents [rows], or None for rows that follow one another."""
    see = np.zeros((rows, past + rows), bool)
    see[:, :past] = True
    for i in range(rows):
        p = i - 1 if parents is None else int(parents[i])
        if p >= 0:
            see[i] = see[p]
        see[i, past + i] = True
    return see


def attention(q, k, v, see, scale):
    """q [R, H, K], k [n, G, K], v [n, G, V], see [R, n] -> (out [R, H, V], sum_j p_j |v_j|, the largest
    sum |q k| * scale of a row's scores [R, H, 1]), float64.  H / G query heads share a key's."""
    r, h, _ = q.shape
    per = h // k.shape[1]
    out, mag = np.zeros((r, h, v.shape[2])), np.zeros((r, h, v.shape[2]))
    big = np.zeros((r, h, 1))
    some = see.any(-1)
    if not some.any():
        return out, mag, big
    for j in range(h):
        g = j // per
        s = np.where(see, np.nan_to_num(q[:, j] @ k[:, g].T) * scale, -np.inf)
        s = s[some]
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        out[some, j], mag[some, j] = p @ v[:, g], p @ np.abs(v[:, g])
        big[:, j, 0] = (np.abs(q[:, j]) @ np.abs(k[:, g]).T).max(-1, initial=0.0) * scale
    return out, mag, big


def tolerance(u, ref, mag, big, channels, keys, fp16, vmax):
    """Bound on |kernel - ref| element by element.  A weight is rounded to the layer's type (u, half a step, of each:
    u * mag) and so is the result (u * |ref|); sums over keys and the exponentials add at most 2^-12 of mag at these
    lengths.  A score is a sum of channels / 16 steps in fp32, each off by at most 2^-23 of sum |q k|; a score off by e
    changes its weight and the weights' sum by a factor of 1 + e each.  A weight below fp16's normal range is off by up
    to 2^-25 of the largest, whose share is 1."""
    e = (channels / 16 + 1) * 2.0 ** -23 * big
    tol = u * np.abs(ref) + (u + 2.0 ** -12 + 2 * e) * mag + 1e-30
    return tol + keys * 2.0 ** -25 * vmax if fp16 else tol
