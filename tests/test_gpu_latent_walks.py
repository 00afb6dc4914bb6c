"""Long walks over the keys: scores whose maximum rises, falls or stays from tile to tile, so that outputs are rescaled
while a CTA has a unit; all heads of calls whose CTAs have several items; and calls one behind another.  Against 64 bits."""
import math

import numpy as np
import pytest
import torch

import chunked_prefill_causal_cp_gb300 as cp
from latent_util import Cache, cu, f64, half_step, ints, tree
from oracle import latent as oracle

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
SMS, START = 152, 4  # CTAs that share a call's tiles of keys; a unit counts as so many tiles more
RISES = (-9.0, 0.0, 3.0, 9.0, 30.0)  # of a pair's scores at each step, in powers of two


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from chunked_prefill_causal_cp_gb300 import _build
    _build.build()


def off(dtype, q, k, v, see, scale, got):
    """The largest error of `got` [R, H, V] in units of its tolerance; q [R, H, K], k [n, G, K], v [n, G, V], see [R, n].
    As oracle.attention, in 64 bits on the GPU."""
    q, k, v = (x.double() for x in (q, k, v))
    groups = k.shape[1]
    x = q.unflatten(1, (groups, -1)).permute(1, 2, 0, 3)  # [G, H / G, R, K]
    kt, vt = k.permute(1, 2, 0)[:, None], v.permute(1, 0, 2)[:, None]
    hide = ~torch.from_numpy(see).to(q.device)
    s = (x @ kt * scale).masked_fill(hide, -math.inf)
    p = torch.softmax(s, -1)
    p = p.masked_fill(hide.all(-1)[:, None], 0.0)  # rows that see nothing
    ref, mag, big = p @ vt, p @ vt.abs(), (x.abs() @ kt.abs()).amax(-1, keepdim=True) * scale
    ref, mag, big = (y.permute(2, 0, 1, 3).flatten(1, 2).cpu().numpy() for y in (ref, mag, big))
    tol = oracle.tolerance(half_step(dtype), ref, mag, big, q.shape[2], k.shape[0], dtype == F16, float(v.abs().max()))
    err = np.abs(f64(got) - ref)
    assert np.isfinite(err).all()
    return float((err / tol).max())


def steps_of(n, tile):
    """Steps up to each of n positions: one every third tile, and one more at the last."""
    j = torch.arange(n)
    return (j // tile // 3 + (j // tile == (n - 1) // tile)).float()


def rising(x, q, channel, tile, lens, seed):
    """Plants scores that change by RISES at every step: position's steps into `channel` of the keys, what a step is worth
    into that of the queries.  Steps are whole numbers below 256, exact in both types."""
    for s, n in enumerate(lens):
        rows = x.at(x.arrays[0], s, 0, n).clone()
        rows[..., channel] = steps_of(n, tile).to(x.dtype).cuda()[:, None]
        x.put(x.arrays[0], s, 0, rows)
    worth = torch.tensor(RISES)[torch.randint(0, len(RISES), q.shape[:2], generator=torch.Generator().manual_seed(seed))]
    q[..., channel] = (worth / (x.scale * math.log2(math.e))).to(x.dtype).cuda()


def check(x, q, out, past, rows, parents):
    r0 = 0
    for s, (p, r) in enumerate(zip(past, rows)):
        k = x.at(x.arrays[0], s, 0, p + r)
        v = k[..., :x.latent] if x.latent else x.at(x.v, s, 0, p + r)
        see = oracle.sees(r, p, None if parents is None else parents[s])
        assert off(x.dtype, q[r0:r0 + r], k, v, see, x.scale, out[r0:r0 + r]) <= 1.0, s
        r0 += r


@pytest.mark.parametrize("dtype,c,r,heads,seqs,rows,page,kind", [
    (BF16, 512, 64, 32, 12, 16, 0, "heap"), (F16, 512, 64, 20, 12, 13, 64, None), (BF16, 512, 0, 16, 60, 1, 16, None),
    (F16, 384, 48, 16, 60, 1, 32, None), (BF16, 384, 16, 40, 12, 20, 0, "random"), (BF16, 256, 32, 128, 10, 5, 128, None),
    (F16, 128, 16, 40, 12, 17, 16, "heap"), (BF16, 128, 64, 8, 60, 3, 0, "star")])
def test_latent_maxima_that_rise_along_a_walk(dtype, c, r, heads, seqs, rows, page, kind):
    past = [500 + (7919 * (i + 3)) % 5501 for i in range(seqs)]
    lens = [p + rows for p in past]
    units = -(-rows * heads // 64)
    assert sum(units * (START + -(-n // 64)) for n in lens) > 10 * SMS  # tiles of a CTA: rises of each kind among them
    x = Cache(dtype, heads, seqs, 6100, page, latent=c, rope=r, scale=0.05)
    x.fill(lens)
    q = x.queries(seqs * rows)
    rising(x, q, c + r - 1 if r else 0, 64, lens, seed=c + r)
    parents = kind and [tree(rows, kind, s) for s in range(seqs)]
    out = x.attend(q, past, [rows] * seqs, parents, uniform=True)
    assert int(x.status) == 0
    check(x, q, out, past, [rows] * seqs, parents)


@pytest.mark.parametrize("dtype,heads,kv,d,seqs,rows,page,lone", [
    (BF16, 32, 8, 128, 12, 16, 16, True), (F16, 32, 8, 64, 12, 30, 0, True), (BF16, 5, 5, 64, 24, 20, 64, True),
    (F16, 32, 8, 128, 12, 61, 0, False), (BF16, 6, 2, 64, 24, 100, 32, False), (BF16, 48, 6, 128, 10, 128, 128, False)])
def test_tree_maxima_that_rise_along_a_walk(dtype, heads, kv, d, seqs, rows, page, lone):
    past = [500 + (7919 * (i + 3)) % 5501 for i in range(seqs)]
    lens = [p + rows for p in past]
    of = 128 // (heads // kv)  # tokens of a Q tile
    tiles, two = -(-rows // of), -(-rows // (2 * of))
    assert (4 * two > 3 * tiles) == lone
    assert sum((tiles if lone else two) * kv * (START + -(-n // 128)) for n in lens) > 10 * SMS
    x = Cache(dtype, heads, seqs, 6200, page, kv=kv, d=d)
    x.fill(lens)
    q = x.queries(seqs * rows)
    rising(x, q, 0, 128, lens, seed=rows)
    parents = [tree(rows, "heap" if s % 2 else "random", s) for s in range(seqs)]
    out = x.attend(q, past, [rows] * seqs, parents, uniform=True)
    assert int(x.status) == 0
    check(x, q, out, past, [rows] * seqs, parents)


@pytest.mark.parametrize("dtype,heads,dn,r,dv", [
    (BF16, 40, 128, 64, 128), (F16, 90, 64, 32, 64), (BF16, 60, 128, 0, 64), (BF16, 200, 128, 64, 128),
    (F16, 201, 64, 32, 64), (BF16, 210, 128, 16, 64), (F16, 195, 64, 0, 128), (BF16, 220, 64, 0, 64)])
@pytest.mark.parametrize("rise", [False, True])
def test_expanded_chunks_every_head(dtype, heads, dn, r, dv, rise):
    """Several lone Q tiles a CTA, and heads enough for pairs of them: every head, with maxima that rise along the keys
    and without."""
    rows, keys = [1, 300, 37, 128, 2], [1, 300, 700, 257, 1300]
    g = torch.Generator().manual_seed(heads)
    t, n = sum(rows), sum(keys)
    q = torch.randn(t, heads, dn + r, generator=g).to(dtype).cuda()
    kv = torch.randn(n, heads, dn + dv, generator=g).to(dtype).cuda()
    k, v = kv[..., :dn], kv[..., dn:]
    kr = torch.randn(n, r, generator=g).to(dtype).cuda() if r else None
    scale = (dn + r) ** -0.5
    if rise:
        level = torch.cat([steps_of(m, 128) * 2 for m in keys]).to(dtype).cuda()
        if r:
            kr[:, r - 1] = level
        else:
            k[..., dn - 1] = level[:, None]
        worth = torch.tensor(RISES)[torch.randint(0, len(RISES), (t, heads), generator=g)]
        q[..., dn + r - 1] = (worth / (scale * math.log2(math.e))).to(dtype).cuda()
    out = torch.full((t, heads, dv), float("nan"), dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    desc = cp.latent_desc(dtype, 1, heads, 512, r, nope_dim=dn, v_dim=dv, capacity=1)
    cp.cp_latent_chunk_attn(desc, q, k, kr, v, out, len(rows), t, n, cu_rows=cu(rows), cu_keys=cu(keys), dev_status=status)
    assert int(status) == 0
    whole = k if kr is None else torch.cat([k, kr[:, None].expand(n, heads, r)], -1)
    r0 = k0 = 0
    for a, m in zip(rows, keys):
        see = np.arange(m) <= (m - a + np.arange(a))[:, None]
        assert off(dtype, q[r0:r0 + a], whole[k0:k0 + m], v[k0:k0 + m], see, scale, out[r0:r0 + a]) <= 1.0
        r0, k0 = r0 + a, k0 + m


@pytest.mark.parametrize("heads,rows,steps,page", [(4, 16, 40, 0), (4, 100, 12, 16), (32, 64, 16, 64)])
def test_lengths_that_grow_behind_one_another(heads, rows, steps, page):
    """Calls that advance the lengths themselves, enqueued without a wait: each takes its tiles, and merges its parts, by
    the lengths that the one before left.  The first grids are smaller than the merge's, which runs on other SMs too."""
    past = [0, 37]
    x = Cache(BF16, heads, 2, rows * steps + 64, page, latent=512, rope=64)
    x.fill([p + rows * steps for p in past])
    t = 2 * rows
    q = x.queries(steps * t).unflatten(0, (steps, t))
    out = torch.full((steps, t, heads, 512), float("nan"), dtype=BF16, device="cuda")
    ws = torch.full((cp.cp_workspace_size_latent(x.desc, t, rows * steps + 64, 2),), 255, dtype=torch.uint8, device="cuda")
    lens = ints(past)
    torch.cuda.synchronize()
    for i in range(steps):
        cp.cp_latent_attn(x.desc, q[i], x.x, lens, 2, t, rows * steps + 64, out[i], ws, block_table=x.table, commit=True,
                          dev_status=x.status)
    assert lens.tolist() == [p + rows * steps for p in past] and int(x.status) == 0
    for i in range(steps):
        check(x, q[i], out[i], [p + rows * i for p in past], [rows] * 2, None)


def test_drafts_one_behind_another_against_the_definition():
    """A draft's rows in, its attention, the accepted path to its places and the lengths' advance, 20 times without a wait;
    every round against 64 bits over the rows that each sequence must hold by then."""
    n, rows, rounds, past = 4, 9, 20, [0, 300, 1000, 63]
    path, count, parents = [0, 2, 7], [1, 3, 2, 0], tree(9, "heap")
    g = torch.Generator().manual_seed(7)
    q = torch.randn(rounds, n * rows, 8, 64, generator=g).to(F16).cuda()
    new = torch.randn(rounds, 2, n * rows, 2, 64, generator=g).to(F16).cuda()
    x = Cache(F16, 8, n, 1200, 16, kv=2, d=64)
    x.fill(past)
    held = [[x.at(a, s, 0, p).clone() for a in x.arrays] for s, p in enumerate(past)]
    lens, out = ints(past), torch.full((rounds, n * rows, 8, 64), float("nan"), dtype=F16, device="cuda")
    ws = torch.full((cp.cp_workspace_size_tree(x.desc, n * rows, 1200, n),), 255, dtype=torch.uint8, device="cuda")
    par, places, counts = ints(parents * n), ints([path] * n), ints(count)
    torch.cuda.synchronize()
    for i in range(rounds):
        cp.cp_kv_append(x.desc, new[i, 0], new[i, 1], rows, x.k, x.v, lens, 1150, x.table, x.status)
        cp.cp_tree_attn(x.desc, q[i], x.k, x.v, lens, par, n, n * rows, 1200, out[i], ws, block_table=x.table,
                        dev_status=x.status)
        cp.cp_tree_commit(x.desc, x.k, x.v, places, counts, lens, n, 3, 1200, block_table=x.table, dev_status=x.status)
    assert lens.tolist() == [p + rounds * c for p, c in zip(past, count)] and int(x.status) == 0
    for i in range(rounds):
        for s in range(n):
            at = slice(s * rows, (s + 1) * rows)
            k, v = (torch.cat([a, b[at]]) for a, b in zip(held[s], new[i]))
            see = oracle.sees(rows, held[s][0].shape[0], parents)
            assert off(F16, q[i, at], k, v, see, x.scale, out[i, at]) <= 1.0, (i, s)
            held[s] = [torch.cat([a, b[at][path[:count[s]]]]) for a, b in zip(held[s], new[i])]
    for s in range(n):
        for a, b in zip(x.arrays, held[s]):
            assert torch.equal(x.at(a, s, 0, b.shape[0]), b)
