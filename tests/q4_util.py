"""Buffers of a 4-bit cache for the GPU tests, and the derived error bounds."""
from __future__ import annotations

import numpy as np
import torch

import chunked_prefill_causal_cp_gb300 as cp
from oracle import q4


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


class Cache4:
    """A contiguous or paged 4-bit cache, every unwritten byte poisoned: codes
    all ones, params NaN.  Paged: pages dealt at random, one spare page."""

    def __init__(self, dtype, hq, hkv, d, n_seqs, ctx, page=0, scale=0.0, seed=0):
        self.dtype, self.hq, self.hkv, self.d, self.page, self.n = dtype, hq, hkv, d, page, n_seqs
        self.scale = scale or d ** -0.5
        if page:
            blocks = -(-ctx // page) + 1
            self.pages = n_seqs * blocks + 1
            perm = torch.randperm(self.pages, generator=torch.Generator().manual_seed(seed))[:-1]
            self.table = perm.reshape(n_seqs, blocks).to(torch.int32).cuda()
            self.desc = cp.layer_desc(dtype, 0, hq, hkv, d, cp.CP_CACHE_PAGED, page_size=page, num_pages=self.pages,
                                      max_blocks=blocks, scale=scale)
            lead = (self.pages, hkv, page)
        else:
            self.cap, self.table = ctx, None
            self.desc = cp.layer_desc(dtype, n_seqs, hq, hkv, d, cp.CP_CACHE_CONTIG, capacity=ctx, scale=scale)
            lead = (n_seqs, hkv, ctx)
        nan = float("nan")
        self.kc = torch.full((*lead, d // 2), 255, dtype=torch.uint8, device="cuda")
        self.vc = torch.full_like(self.kc, 255)
        self.kp = torch.full((*lead, d // 32, 2), nan, dtype=dtype, device="cuda")
        self.vp = torch.full_like(self.kp, nan)
        self.arg = cp.q4_cache(self.kc, self.vc, self.kp, self.vp)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def slot(self, s, pos):
        if not self.page:
            return s, pos
        return int(self.table[s, pos // self.page]), pos % self.page

    def rows(self, s, n):
        """Codes and params of positions [0, n) of sequence s: K and V as ([n, Hkv, D], scale, lo) in numpy."""
        if self.page:
            b = self.table[s, :-(-n // self.page)].long()
            pick = lambda x: x[b].transpose(1, 2).flatten(0, 1)[:n]  # noqa: E731
        else:
            pick = lambda x: x[s, :, :n].transpose(0, 1)  # noqa: E731
        out = []
        for c, p in ((self.kc, self.kp), (self.vc, self.vp)):
            c, p = pick(c).cpu().contiguous().numpy(), pick(p).float().cpu().numpy()
            out.append((q4.unpack(c), p[..., 0], p[..., 1]))
        return out

    def values(self, s, n):
        """K and V of positions [0, n), [n, Hkv, D] float64, rounded once to the layer's type."""
        return [f64(torch.from_numpy(q4.values(*x)).to(self.dtype)) for x in self.rows(s, n)]

    def workspace(self, total_rows, max_ctx, n=None):
        b = cp.cp_workspace_size_q4(self.desc, total_rows, max_ctx, n or self.n)
        return torch.full((max(b, 16),), 255, dtype=torch.uint8, device="cuda")  # contents do not matter

    def fill(self, rows, seed=1, k_scale=1.0):
        """Appends rows[s] random rows to each sequence through the library; returns (k, v) rows."""
        g = torch.Generator().manual_seed(seed)
        t = sum(rows)
        k = (torch.randn(t, self.hkv, self.d, generator=g) * k_scale).to(self.dtype).cuda()
        v = torch.randn(t, self.hkv, self.d, generator=g).to(self.dtype).cuda()
        keep = [i for i, r in enumerate(rows) if r > 0]  # every listed sequence has rows
        for i in keep:
            r0 = sum(rows[:i])
            sub = slice(i, i + 1)
            cache, desc, table = self.view(i)
            cp.cp_kv_append_q4(desc, k[r0:r0 + rows[i]], v[r0:r0 + rows[i]], cache,
                               torch.zeros(1, dtype=torch.int32, device="cuda"), 1, rows[i], max(rows),
                               block_table=table if table is None else table[sub], dev_status=self.status)
        return k, v

    def view(self, i):
        """The cache as seen by a call on sequence i alone (contiguous: its own slice)."""
        if self.page:
            return self.arg, self.desc, self.table
        cut = [x[i:i + 1] for x in (self.kc, self.vc, self.kp, self.vp)]
        desc = cp.layer_desc(self.dtype, 1, self.hq, self.hkv, self.d, cp.CP_CACHE_CONTIG, capacity=self.cap,
                             scale=self.desc.scale)
        return cp.q4_cache(*cut), desc, None


def check_attention(cache, q, out, past, rows, seqs=None):
    """Every row of out against 64 bits.  Bound: P is rounded to the layer's type before the product with V
    (half a step of each weight, so half_step * sum p |v|) and the result once (half_step * |o|); fp32 sums over
    the keys and the weights' exponentials add at most 2^-12 * sum p |v| at these lengths.  A weight below fp16's
    normal range is off by up to 2^-25 of the largest (whose share is 1): n * 2^-25 * max |v|."""
    u = half_step(cache.dtype)
    r0 = 0
    worst = 0.0
    for i, (p, r) in enumerate(zip(past, rows)):
        k, v = cache.values(i if seqs is None else seqs[i], p + r)
        ref, mag = q4.attention(f64(q[r0:r0 + r]), k, v, p, cache.scale)
        err = np.abs(f64(out[r0:r0 + r]) - ref)
        tol = u * np.abs(ref) + (u + 2.0 ** -12) * mag + 1e-30
        if cache.dtype == torch.float16:
            tol = tol + (p + r) * 2.0 ** -25 * np.abs(v).max()
        assert np.isfinite(err).all(), (i, p, r)
        worst = max(worst, float((err / tol).max()))
        r0 += r
    assert worst <= 1.0, worst
