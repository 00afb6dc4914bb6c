"""Caches for the GPU tests of latent attention and drafted trees, and the checks against 64 bits."""
from __future__ import annotations

import numpy as np
import torch

import chunked_prefill_causal_cp_gb300 as cp
from oracle import latent as oracle


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def ints(xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


def cu(rows):
    return ints([0, *np.cumsum(rows).tolist()])


def tree(rows, kind, seed=0):
    """Parents of a tree of `rows` nodes: "chain", "star", "heap" (three children a node), "forest" (several roots)
    or "random"."""
    g = np.random.default_rng(seed)
    of = {"chain": lambda i: i - 1, "star": lambda i: 0 if i else -1, "heap": lambda i: (i - 1) // 3 if i else -1,
          "forest": lambda i: i - 4 if i >= 4 else -1, "random": lambda i: int(g.integers(-1, i)) if i else -1}[kind]
    return [of(i) for i in range(rows)]


class Cache:
    """A contiguous or paged cache, every slot NaN: of latents (latent, rope), or of K and V (kv heads, d)."""

    def __init__(self, dtype, heads, n_seqs, ctx, page=0, latent=0, rope=0, kv=0, d=0, scale=0.0, seed=0, **kw):
        self.dtype, self.heads, self.n, self.page, self.latent, self.rope, self.kv, self.d = (
            dtype, heads, n_seqs, page, latent, rope, kv, d)
        if page:
            blocks = -(-ctx // page) + 1
            self.pages = n_seqs * blocks + 1
            perm = torch.randperm(self.pages, generator=torch.Generator().manual_seed(seed))[:-1]
            self.table = perm.reshape(n_seqs, blocks).to(torch.int32).cuda()
            kind = dict(kind=cp.CP_CACHE_PAGED, page_size=page, num_pages=self.pages, max_blocks=blocks)
            lead, slots = (self.pages,), page
        else:
            self.table, kind, lead, slots = None, dict(kind=cp.CP_CACHE_CONTIG, capacity=ctx), (n_seqs,), ctx
        nan = dict(fill_value=float("nan"), dtype=dtype, device="cuda")
        if latent:
            self.desc = cp.latent_desc(dtype, n_seqs, heads, latent, rope, scale=scale, **kind, **kw)
            self.scale = scale or (self.desc.nope_dim + rope) ** -0.5
            self.x = torch.full((*lead, slots, latent + rope), **nan)
            self.arrays = [self.x]
        else:
            self.desc = cp.layer_desc(dtype, n_seqs, heads, kv, d, scale=scale, **kind)
            self.scale = scale or d ** -0.5
            self.k, self.v = torch.full((*lead, kv, slots, d), **nan), torch.full((*lead, kv, slots, d), **nan)
            self.arrays = [self.k, self.v]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def at(self, x, s, first, count):
        """View-free rows [count, kv, d] (latent: [count, 1, C + R]) of positions first .. of array x."""
        pos = torch.arange(first, first + count, device="cuda")
        i, j = (torch.full_like(pos, s), pos) if not self.page else (self.table[s].long()[pos // self.page], pos % self.page)
        return x[i, j][:, None] if self.latent else x[i, :, j]

    def put(self, x, s, first, rows):
        pos = torch.arange(first, first + rows.shape[0], device="cuda")
        i, j = (torch.full_like(pos, s), pos) if not self.page else (self.table[s].long()[pos // self.page], pos % self.page)
        if self.latent:
            x[i, j] = rows[:, 0].to(x.dtype)
        else:
            x[i, :, j] = rows.to(x.dtype)

    def fill(self, lens, seed=1, k_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        for s, n in enumerate(lens):
            for x in self.arrays:
                w = torch.randn(n, 1 if self.latent else self.kv, x.shape[-1], generator=g)
                self.put(x, s, 0, (w * (k_scale if x is self.arrays[0] and not self.latent else 1.0)).cuda())

    def values(self, s, n):
        """K [n, G, K] and V [n, G, V] of positions [0, n), float64."""
        k = f64(self.at(self.arrays[0], s, 0, n))
        return (k, k[..., :self.latent]) if self.latent else (k, f64(self.at(self.v, s, 0, n)))

    def queries(self, t, seed=3):
        w = self.latent + self.rope if self.latent else self.d
        return torch.randn(t, self.heads, w, generator=torch.Generator().manual_seed(seed)).to(self.dtype).cuda()

    def empty_out(self, t):
        return torch.full((t, self.heads, self.latent or self.d), float("nan"), dtype=self.dtype, device="cuda")

    def attend(self, q, past, rows, parents=None, out=None, uniform=False, commit=False, max_ctx=None, ws=None, **kw):
        """One call; parents: a list for each sequence.  Returns out."""
        t, n = q.shape[0], len(rows)
        out = self.empty_out(t) if out is None else out
        mc = max_ctx or max(p + r for p, r in zip(past, rows))
        call = dict(cu_rows=None if uniform else cu(rows), block_table=self.table, dev_status=self.status)
        call.update(kw)
        par = None if parents is None else ints([p for x in parents for p in x] + [0] * (t - sum(rows)))
        lens = past if torch.is_tensor(past) else ints(past)
        size = (cp.cp_workspace_size_latent if self.latent else cp.cp_workspace_size_tree)(self.desc, t, mc, n)
        ws = torch.full((max(size, 16),), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
        if self.latent:
            cp.cp_latent_attn(self.desc, q, self.x, lens, n, t, mc, out, ws, parents=par, commit=commit, **call)
        else:
            cp.cp_tree_attn(self.desc, q, self.k, self.v, lens, par, n, t, mc, out, ws, **call)
        return out

    def check(self, q, out, past, rows, parents=None):
        """Every row of out against 64 bits."""
        r0, worst = 0, 0.0
        for s, (p, r) in enumerate(zip(past, rows)):
            k, v = self.values(s, p + r)
            worst = max(worst, off(self.dtype, f64(q[r0:r0 + r]), k, v,
                                   oracle.sees(r, p, None if parents is None else parents[s]), self.scale,
                                   f64(out[r0:r0 + r])))
            r0 += r
        assert worst <= 1.0, worst


def off(dtype, q, k, v, see, scale, got):
    """The largest error of `got` in units of its tolerance."""
    ref, mag, big = oracle.attention(q, k, v, see, scale)
    tol = oracle.tolerance(half_step(dtype), ref, mag, big, q.shape[2], k.shape[0], dtype == torch.float16,
                           np.abs(v).max(initial=0.0))
    err = np.abs(got - ref)
    assert np.isfinite(err).all()
    return float((err / tol).max(initial=0.0))
