"""GPU tests of latent caches and drafted trees at the edges of what a call may be: caches shorter than a tile of keys,
offsets that begin behind rows of no sequence, lists of sequences most of which are skipped, values that are not finite
under a causal mask, and calls that need no workspace.  Against 64 bits."""
import numpy as np
import pytest
import torch

import chunked_prefill_causal_cp_gb300 as cp
from latent_util import Cache, f64, ints, off, tree
from oracle import latent as oracle

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
BOTH = [dict(heads=16, latent=512, rope=64), dict(heads=8, kv=2, d=128)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from chunked_prefill_causal_cp_gb300 import _build
    _build.build()


def _split(kw):
    return kw["heads"], {k: v for k, v in kw.items() if k != "heads"}


@pytest.mark.parametrize("kw", BOTH + [dict(heads=3, latent=384, rope=16), dict(heads=7, kv=7, d=64)])
@pytest.mark.parametrize("ctx", [1, 5, 40, 63])
def test_caches_shorter_than_a_tile(kw, ctx):
    """No workspace, either: one tile of keys."""
    heads, kw = _split(kw)
    rows = [1, min(ctx, 4), min(ctx, 3)]
    past = [ctx - r for r in rows]
    x = Cache(F16, heads, 3, ctx, **kw)
    x.fill([ctx] * 3)
    q = x.queries(sum(rows))
    parents = [tree(r, "heap") for r in rows]
    size = (cp.cp_workspace_size_latent if x.latent else cp.cp_workspace_size_tree)(x.desc, sum(rows), ctx, 3)
    assert size == 0
    out = x.attend(q, past, rows, parents)
    assert int(x.status) == 0
    x.check(q, out, past, rows, parents)


@pytest.mark.parametrize("kw", BOTH)
def test_most_sequences_skipped(kw):
    """130 sequences: without rows, of negative or too long contexts, and every fifth one computed, its keys over SMs."""
    heads, kw = _split(kw)
    n, r = 130, 3
    rows = [0 if s % 5 == 1 else r for s in range(n)]
    past = [(7919 * (s + 3)) % 1500 for s in range(n)]
    lens = [-1 - s if s % 5 == 2 else 1998 + s if s % 5 == 3 else 2 ** 31 - 1 - s if s % 5 == 4 else past[s] for s in range(n)]
    x = Cache(BF16, heads, n, 2000, 64, **kw)
    taken = range(0, n, 5)
    for s in taken:
        for a in x.arrays:
            g = torch.Generator().manual_seed(s)
            x.put(a, s, 0, torch.randn(past[s] + r, 1 if x.latent else x.kv, a.shape[-1], generator=g).cuda())
    starts = np.concatenate([[0], np.cumsum(rows)])
    t = int(starts[-1])
    q = x.queries(t)
    parents = [tree(m, "star") for m in rows]
    out = x.attend(q, ints(lens), rows, parents, max_ctx=2000)
    assert int(x.status) == cp.CP_DEV_BOUNDS
    for s in range(n):
        at = slice(int(starts[s]), int(starts[s + 1]))
        if s % 5 == 0:
            k, v = x.values(s, past[s] + r)
            assert off(BF16, f64(q[at]), k, v, oracle.sees(r, past[s], parents[s]), x.scale, f64(out[at])) <= 1.0
        else:
            assert torch.isnan(out[at]).all()


@pytest.mark.parametrize("kw", BOTH)
def test_offsets_that_begin_behind_rows_of_no_sequence(kw):
    heads, kw = _split(kw)
    rows, past = [4, 9], [700, 33]
    x = Cache(BF16, heads, 2, 800, 16, **kw)
    x.fill([p + r for p, r in zip(past, rows)])
    q = x.queries(20)
    parents = [tree(r, "heap") for r in rows]
    out = x.attend(q, past, rows, [[-1] * 5, *parents], cu_rows=ints([5, 9, 18]))
    assert int(x.status) == 0
    x.check(q[5:18], out[5:18], past, rows, parents)
    assert torch.isnan(out[:5]).all() and torch.isnan(out[18:]).all()


def test_append_behind_rows_of_no_sequence():
    x = Cache(BF16, 2, 2, 64, 16, latent=128, rope=16)
    proj, q = torch.randn(9, 144, device="cuda").bfloat16(), torch.randn(9, 2, 16, device="cuda").bfloat16()
    qo = torch.full_like(q, 7.0)
    cp.cp_latent_append(x.desc, cp.qk_prep(0), proj[:, :128], proj[:, 128:], x.x, ints([5, 20]), 2, 9, 64,
                        cu_rows=ints([2, 5, 8]), q_rope=q, q_out=qo, block_table=x.table, dev_status=x.status)
    assert int(x.status) == 0
    assert torch.equal(x.at(x.x, 0, 5, 3)[:, 0], proj[2:5]) and torch.equal(x.at(x.x, 1, 20, 3)[:, 0], proj[5:8])
    assert int((~torch.isnan(x.x)).any(-1).sum()) == 6
    assert torch.equal(qo[2:8], q[2:8]) and (qo[:2] == 7.0).all() and (qo[8:] == 7.0).all()


@pytest.mark.parametrize("c,heads,page", [(512, 16, 0), (384, 40, 16), (128, 5, 64)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_non_finite_latents_under_a_causal_mask(c, heads, page, value):
    """In the call's own rows: the rows that see it.  In the context: its sequence, and no other."""
    rows, past = [30, 11], [100, 300]
    x = Cache(BF16, heads, 2, 400, page, latent=c, rope=32)
    x.fill([p + r for p, r in zip(past, rows)])
    q = x.queries(41)
    clean = x.attend(q, past, rows)
    x.check(q, clean, past, rows)
    for s, at, first in ((0, 100, 0), (0, 127, 27), (0, 129, 29), (0, 40, 0), (1, 305, 35), (1, 250, 30)):
        kept = x.at(x.x, s, at, 1).clone()
        bad = kept.clone()
        bad[..., c - 1] = value
        x.put(x.x, s, at, bad)
        out = x.attend(q, past, rows)
        x.put(x.x, s, at, kept)
        end = 30 if s == 0 else 41
        assert torch.equal(out[:first], clean[:first]) and torch.equal(out[end:], clean[end:])
        assert (~torch.isfinite(out[first:end].float())).any(-1).all()


def test_expanded_offsets_that_begin_behind_rows_and_keys_of_no_sequence():
    heads, dn, r, dv, t, n = 9, 64, 32, 128, 400, 900
    g = torch.Generator().manual_seed(1)
    q = torch.randn(t, heads, dn + r, generator=g).to(F16).cuda()
    k, v = torch.randn(n, heads, dn, generator=g).to(F16).cuda(), torch.randn(n, heads, dv, generator=g).to(F16).cuda()
    kr = torch.randn(n, r, generator=g).to(F16).cuda()
    cr, ck = [7, 207, 390], [11, 500, 890]
    for x in (k, v, kr):
        x[:11] = x[890:] = float("nan")
    out, status = torch.full((t, heads, dv), 7.0, dtype=F16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    desc = cp.latent_desc(F16, 1, heads, 128, r, nope_dim=dn, v_dim=dv, capacity=1)
    cp.cp_latent_chunk_attn(desc, q, k, kr, v, out, 2, t, n, cu_rows=ints(cr), cu_keys=ints(ck), dev_status=status)
    assert int(status) == 0 and (out[:7] == 7.0).all() and (out[390:] == 7.0).all()
    for s in range(2):
        a, b, i, j = cr[s], cr[s + 1], ck[s], ck[s + 1]
        keys = np.concatenate([f64(k[i:j]), np.broadcast_to(f64(kr[i:j])[:, None], (j - i, heads, r))], -1)
        see = np.arange(j - i) <= (j - i - (b - a) + np.arange(b - a))[:, None]
        assert off(F16, f64(q[a:b]), keys, f64(v[i:j]), see, (dn + r) ** -0.5, f64(out[a:b])) <= 1.0
