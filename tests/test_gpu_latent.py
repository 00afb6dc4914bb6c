"""GPU parity of latent caches and of drafted trees over both kinds of cache: the append's rows, attention of single
tokens, chunks and trees, and the expanded form, against 64 bits."""
import numpy as np
import pytest
import torch

import chunked_prefill_causal_cp_gb300 as cp
from latent_util import Cache, cu, f64, half_step, ints, off, tree
from oracle import latent as oracle

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from chunked_prefill_causal_cp_gb300 import _build
    _build.build()


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("c,r,rot,inter,page,heads", [(512, 64, 64, False, 0, 32), (512, 64, 32, True, 64, 3),
                                                      (256, 48, 48, False, 16, 11), (384, 16, 16, True, 32, 16),
                                                      (128, 32, 0, False, 0, 1), (256, 0, 0, False, 128, 4)])
def test_append_rows(dtype, c, r, rot, inter, page, heads):
    rows, past = [1, 77, 5], [140, 0, 63]
    t = sum(rows)
    x = Cache(dtype, heads, 3, 256, page, latent=c, rope=r)
    g = torch.Generator().manual_seed(1)
    proj = (torch.randn(t, c + r + 8, generator=g) * 2).to(dtype).cuda()
    q = torch.randn(t, heads, r + 16, generator=g).to(dtype).cuda()
    wide = torch.full((t, heads, c + r), 5.0, dtype=dtype, device="cuda")
    w = (1 + 0.3 * torch.randn(c, generator=g)).to(dtype).cuda()
    freq = (500.0 ** (-torch.arange(0, max(rot, 2), 2) / max(rot, 1))).float().cuda()
    call = dict(inv_freq=freq, cu_rows=cu(rows), block_table=x.table, dev_status=x.status)
    cp.cp_latent_append(x.desc, cp.qk_prep(rot, inter, 1e-5), proj[:, :c], proj[:, c:c + r] if r else None, x.x, ints(past),
                        3, t, 256, weight=w, q_rope=q[..., 16:] if r else None, q_out=wide[..., c:] if r else None, **call)
    assert int(x.status) == 0
    u = half_step(dtype)
    pos = np.concatenate([np.arange(p, p + n) for n, p in zip(rows, past)])
    want = oracle.norm(f64(proj[:, :c]), f64(w), 1e-5)
    keys, kmag = oracle.rotate(f64(proj[:, None, c:c + r]), pos, f64(freq), rot, inter)
    got = np.concatenate([f64(x.at(x.x, s, p, n))[:, 0] for s, (n, p) in enumerate(zip(rows, past))])
    # One rounding to the type, and fp32 work: 16 + 5 sums, a root, three products below 2^-18; angles within 2^-25, and
    # sines and products three fp32 roundings.
    assert (np.abs(got[:, :c] - want) <= (u + 2.0 ** -18) * np.abs(want) + 2.0 ** -25).all()
    assert (np.abs(got[:, c:] - keys[:, 0]) <= u * np.abs(keys[:, 0]) + 2.0 ** -21 * kmag[:, 0] + 2.0 ** -25).all()
    if r:
        ref, mag = oracle.rotate(f64(q[..., 16:]), pos, f64(freq), rot, inter)
        assert (np.abs(f64(wide[..., c:]) - ref) <= u * np.abs(ref) + 2.0 ** -21 * mag + 2.0 ** -25).all()
        assert torch.equal(wide[..., c + rot:], q[..., 16 + rot:])  # channels that are not rotated, bit for bit
        assert (wide[..., :c] == 5.0).all()
    written = torch.zeros_like(x.x, dtype=torch.bool)
    for s, (n, p) in enumerate(zip(rows, past)):
        for e in range(p, p + n):
            written[(s, e) if not page else (int(x.table[s, e // page]), e % page)] = True
    assert torch.equal(torch.isnan(x.x), ~written)  # nothing else in the cache

    # Without a weight the latent is a copy; positions of their own turn the keys only; queries in place.
    y = Cache(dtype, heads, 3, 256, page, latent=c, rope=r)
    own = ints([(7 * i) % 90 for i in range(t)])
    q2 = q[..., 16:].clone()
    cp.cp_latent_append(y.desc, cp.qk_prep(rot, inter, 1e-5), proj[:, :c], proj[:, c:c + r] if r else None, y.x, ints(past),
                        3, t, 256, positions=own, q_rope=q2 if r else None, q_out=q2 if r else None, **call)
    got = torch.cat([y.at(y.x, s, p, n)[:, 0] for s, (n, p) in enumerate(zip(rows, past))])
    assert torch.equal(got[:, :c], proj[:, :c])
    keys, kmag = oracle.rotate(f64(proj[:, None, c:c + r]), f64(own), f64(freq), rot, inter)
    assert (np.abs(f64(got[:, c:]) - keys[:, 0]) <= u * np.abs(keys[:, 0]) + 2.0 ** -21 * kmag[:, 0] + 2.0 ** -25).all()
    if r:
        ref, mag = oracle.rotate(f64(q[..., 16:]), f64(own), f64(freq), rot, inter)
        assert (np.abs(f64(q2) - ref) <= u * np.abs(ref) + 2.0 ** -21 * mag + 2.0 ** -25).all()


def test_append_of_many_rows_and_far_positions():
    """Several heads' blocks a warp, and positions where 32-bit angles would be lost."""
    c, r, heads, t = 128, 64, 40, 6000
    x = Cache(BF16, heads, 1, t, latent=c, rope=r)
    g = torch.Generator().manual_seed(2)
    proj = torch.randn(t, c + r, generator=g).bfloat16().cuda()
    q = torch.randn(t, heads, r, generator=g).bfloat16().cuda()
    pos = torch.randint(0, 2 ** 31 - 1, (t,), generator=g).int().cuda()
    freq = (10000.0 ** (-torch.arange(0, r, 2) / r)).float().cuda()
    qo = torch.empty_like(q)
    cp.cp_latent_append(x.desc, cp.qk_prep(r), proj[:, :c], proj[:, c:], x.x, ints([0]), 1, t, t, inv_freq=freq,
                        positions=pos, q_rope=q, q_out=qo, dev_status=x.status)
    for got, src in ((x.x[0, :, None, c:], proj[:, None, c:]), (qo, q)):
        ref, mag = oracle.rotate(f64(src), f64(pos), f64(freq), r, False)
        assert (np.abs(f64(got) - ref) <= half_step(BF16) * np.abs(ref) + 2.0 ** -21 * mag + 2.0 ** -25).all()
    assert torch.equal(x.x[0, :, :c], proj[:, :c]) and int(x.status) == 0


def test_append_out_of_bounds_and_padded_batch():
    x = Cache(BF16, 2, 3, 32, 16, latent=128, rope=16)
    x.table[0, 1] = 1000
    proj = torch.randn(14, 144, device="cuda").bfloat16()
    q = torch.randn(14, 2, 16, device="cuda").bfloat16()
    qo = torch.full_like(q, 7.0)
    cp.cp_latent_append(x.desc, cp.qk_prep(0), proj[:, :128], proj[:, 128:], x.x, ints([14, 30, -3]), 3, 14, 32,
                        cu_rows=ints([0, 4, 8, 12]), q_rope=q, q_out=qo, block_table=x.table, dev_status=x.status)
    assert int(x.status) == cp.CP_DEV_BOUNDS
    wrote = (~torch.isnan(x.x)).any(-1).nonzero().tolist()
    table = x.table.cpu()
    want = [[int(table[s, p // 16]), p % 16] for s, p in ((0, 14), (0, 15), (1, 30), (1, 31), (2, 0))]
    assert sorted(wrote) == sorted(want)
    assert torch.equal(qo[:12], q[:12]) and (qo[12:] == 7.0).all()


# ------------------------------------------------------------------ attention over both kinds of cache

LATENT = [dict(latent=512, rope=64), dict(latent=128, rope=0), dict(latent=256, rope=16), dict(latent=384, rope=48)]


@pytest.mark.parametrize("dtype,shape,heads,page", [(BF16, LATENT[0], 16, 0), (F16, LATENT[0], 5, 16), (BF16, LATENT[1], 1, 32),
                                                    (F16, LATENT[2], 40, 64), (BF16, LATENT[3], 128, 128)])
def test_latent_rows_that_follow_one_another(dtype, shape, heads, page):
    rows, past = [1, 3, 1, 17, 2], [0, 63, 700, 64, 1]
    x = Cache(dtype, heads, 5, 1100, page, **shape)
    x.fill([p + r for p, r in zip(past, rows)])
    q = x.queries(sum(rows))
    out = x.attend(q, past, rows)
    assert int(x.status) == 0
    x.check(q, out, past, rows)


@pytest.mark.parametrize("past", [0, 1, 62, 63, 64, 127, 128, 1023, 2047, 2048, 5000])
def test_latent_single_tokens_at_every_kind_of_length(past):
    x = Cache(BF16, 32, 2, past + 130, latent=512, rope=64)
    x.fill([past + 1, past // 2 + 1])
    q = x.queries(2)
    out = x.attend(q, [past, past // 2], [1, 1], uniform=True)
    assert int(x.status) == 0
    x.check(q, out, [past, past // 2], [1, 1])


@pytest.mark.parametrize("seqs,rows,heads", [(1, 1, 8), (1, 1, 64), (1, 1, 128), (1, 16, 8), (3, 4, 32), (1, 100, 5)])
def test_latent_equal_rows_that_fill_their_tiles(seqs, rows, heads):
    past = [316, 0, 1500][:seqs]
    x = Cache(F16, heads, seqs, 1700, latent=256, rope=32)
    x.fill([p + rows for p in past])
    q = x.queries(seqs * rows)
    out = x.attend(q, past, [rows] * seqs, uniform=True)
    assert int(x.status) == 0
    x.check(q, out, past, [rows] * seqs)


@pytest.mark.parametrize("dtype,kw", [(BF16, dict(heads=32, kv=8, d=128)), (F16, dict(heads=6, kv=2, d=64, page=16)),
                                      (BF16, dict(heads=64, kv=1, d=128, page=64)), (F16, dict(heads=5, kv=5, d=128, page=128)),
                                      (BF16, dict(heads=14, kv=2, d=64)), (F16, dict(heads=16, latent=512, rope=64, page=32)),
                                      (BF16, dict(heads=7, latent=256, rope=32))])
@pytest.mark.parametrize("kind", ["random", "heap", "star", "forest", "chain"])
def test_trees(dtype, kw, kind):
    kw = dict(kw)
    heads, page = kw.pop("heads"), kw.pop("page", 0)
    rows, past = [33, 1, 128, 16], [300, 0, 61, 1030]
    x = Cache(dtype, heads, 4, 1200, page, **kw)
    x.fill([p + r for p, r in zip(past, rows)])
    q = x.queries(sum(rows))
    parents = [tree(r, kind, seed=s) for s, r in enumerate(rows)]
    out = x.attend(q, past, rows, parents)
    assert int(x.status) == 0
    x.check(q, out, past, rows, parents)


def test_a_chain_is_a_chunk():
    """A tree without branches sees what rows that follow one another see, bit for bit."""
    rows, past = [9, 40], [100, 70]
    x = Cache(BF16, 8, 2, 256, latent=256, rope=64)
    x.fill([p + r for p, r in zip(past, rows)])
    q = x.queries(sum(rows))
    a = x.attend(q, past, rows)
    b = x.attend(q, past, rows, [tree(r, "chain") for r in rows])
    assert torch.equal(a, b)


BOTH = [dict(heads=16, latent=512, rope=64), dict(heads=8, kv=2, d=128)]


@pytest.mark.parametrize("kw", BOTH)
def test_a_rows_bits_are_its_own_and_the_sizes(kw):
    """The same whatever the bounds, rows given as equal or ragged, and the other sequences' values."""
    heads, kw = kw["heads"], {k: v for k, v in kw.items() if k != "heads"}
    n, rows = 12, 13
    past = [0, 5000, 64, 700, 1, 2100, 333, 4096, 90, 17, 3000, 250]
    x = Cache(BF16, heads, n, 5200, 16, **kw)
    x.fill([p + rows for p in past])
    q = x.queries(n * rows)
    parents = [tree(rows, "random", s) for s in range(n)]
    out = x.attend(q, past, [rows] * n, parents, uniform=True)
    x.check(q, out, past, [rows] * n, parents)
    assert torch.equal(out, x.attend(q, past, [rows] * n, parents, max_ctx=5200))
    assert torch.equal(out, x.attend(q, past, [rows] * n, parents))
    for s in (0, 1, 5, 11):
        at = slice(s * rows, (s + 1) * rows)
        other = -q
        other[at] = q[at]
        assert torch.equal(x.attend(other, past, [rows] * n, parents)[at], out[at])
    assert int(x.status) == 0


@pytest.mark.parametrize("kw", BOTH)
def test_wide_trees_over_long_contexts(kw):
    """Trees of several tiles of rows, their keys over many SMs."""
    heads, kw = kw["heads"], {k: v for k, v in kw.items() if k != "heads"}
    past, rows = [5000, 0, 9001], [61, 128, 100]
    x = Cache(BF16, heads, 3, 9200, 16, **kw)
    x.fill([p + r for p, r in zip(past, rows)])
    q = x.queries(sum(rows))
    parents = [tree(r, k, s) for s, (r, k) in enumerate(zip(rows, ("heap", "random", "chain")))]
    x.check(q, x.attend(q, past, rows, parents), past, rows, parents)
    assert int(x.status) == 0


@pytest.mark.parametrize("kw", BOTH)
def test_many_short_sequences(kw):
    """More tiles of rows than SMs, few of which are split; some sequences without context, one-row ones among them."""
    heads, kw = kw["heads"], {k: v for k, v in kw.items() if k != "heads"}
    seqs = 333
    past = [(7919 * (i + 3)) % 301 if i % 7 else 0 for i in range(seqs)]
    rows = [1 + (5 * i) % 7 for i in range(seqs)]
    x = Cache(BF16, heads, seqs, 320, 16, **kw)
    x.fill([p + r for p, r in zip(past, rows)])
    q = x.queries(sum(rows))
    parents = [tree(r, "random", s) for s, r in enumerate(rows)]
    x.check(q, x.attend(q, past, rows, parents), past, rows, parents)
    assert int(x.status) == 0


@pytest.mark.parametrize("kw", BOTH)
@pytest.mark.parametrize("seqs", [1, 2, 40])
def test_long_contexts_of_few_and_many_sequences(kw, seqs):
    """Splits of every size: one sequence over all SMs, many sequences of several items each."""
    heads, kw = kw["heads"], {k: v for k, v in kw.items() if k != "heads"}
    past = [(7919 * (i + 3)) % 9001 for i in range(seqs)]
    rows = [1 + (5 * i) % 23 for i in range(seqs)]
    x = Cache(F16, heads, seqs, 9100, 64, **kw)
    x.fill([p + r for p, r in zip(past, rows)])
    q = x.queries(sum(rows))
    parents = [tree(r, "heap") for r in rows]
    out = x.attend(q, past, rows, parents)
    assert int(x.status) == 0
    x.check(q, out, past, rows, parents)


@pytest.mark.parametrize("kw", BOTH)
def test_large_scores(kw):
    """Scores that span hundreds of powers of two, their maximum in the last tile."""
    heads, kw = kw["heads"], {k: v for k, v in kw.items() if k != "heads"}
    x = Cache(F16, heads, 1, 600, 16, scale=3.0, **kw)
    x.fill([577])
    q = x.queries(6)
    parents = [tree(6, "heap")]
    out = x.attend(q, [571], [6], parents)
    x.check(q, out, [571], [6], parents)


@pytest.mark.parametrize("kw", BOTH)
def test_non_finite_values_reach_the_rows_that_see_them(kw):
    heads, kw = kw["heads"], {k: v for k, v in kw.items() if k != "heads"}
    rows, past = 20, 120  # the nodes' slots end inside a tile, and span two
    parents = [tree(rows, "heap")]
    see = oracle.sees(rows, past, parents[0])
    x = Cache(BF16, heads, 1, 400, 16, **kw)
    x.fill([past + rows])
    q = x.queries(rows)
    clean = x.attend(q, [past], [rows], parents)
    for node, value in ((0, float("inf")), (7, float("nan")), (19, float("-inf")), (8, float("nan"))):
        y = Cache(BF16, heads, 1, 400, 16, **kw)
        y.fill([past + rows])
        for a in y.arrays[-1:]:  # V, or the latent
            r = y.at(a, 0, past + node, 1).clone()
            r[..., 3] = value
            y.put(a, 0, past + node, r)
        out = y.attend(q, [past], [rows], parents)
        hit = torch.from_numpy(see[:, past + node]).cuda()
        assert torch.equal(out[~hit], clean[~hit])
        assert (~torch.isfinite(out[hit].float())).any(-1).all()


@pytest.mark.parametrize("kw", BOTH)
def test_bad_lengths_pages_and_parents(kw):
    heads, kw = kw["heads"], {k: v for k, v in kw.items() if k != "heads"}
    rows, past = [4, 4, 4, 4], [90, 10, 40, 30]
    x = Cache(BF16, heads, 4, 128, 16, **kw)
    x.fill([p + r for p, r in zip(past, rows)])
    q = x.queries(16)
    parents = [tree(4, "heap")] * 4
    want = x.attend(q, past, rows, parents)
    x.check(q, want, past, rows, parents)
    for lens, left in (([-1, 10, 40, 30], 0), ([90, 10, 2000, 30], 2), ([90, 125, 40, 30], 1)):
        x.status.zero_()
        out = x.attend(q, ints(lens), rows, parents, max_ctx=128)
        assert int(x.status) == cp.CP_DEV_BOUNDS
        for s in range(4):
            part = out[4 * s:4 * s + 4]
            assert torch.isnan(part).all() if s == left else torch.equal(part, want[4 * s:4 * s + 4])
    x.status.zero_()
    keep = x.table.clone()
    x.table[2, 1] = x.pages
    out = x.attend(q, past, rows, parents)
    assert int(x.status) == cp.CP_DEV_BOUNDS
    x.table.copy_(keep)
    for s in (0, 1, 3):
        assert torch.equal(out[4 * s:4 * s + 4], want[4 * s:4 * s + 4])
    for bad in (3, 7, -2, 2 ** 30, -2 ** 31):
        x.status.zero_()
        out = x.attend(q, past, rows, [[-1, 0, 0, bad], *parents[1:]])
        assert int(x.status) == cp.CP_DEV_BOUNDS
        assert torch.equal(out[4:], want[4:]) and torch.equal(out[:3], want[:3])
        x.check(q, out, past, rows, [[-1, 0, 0, -1], *parents[1:]])  # counts as a child of the context
    # Sequences without rows, and one of more than a tree's.
    x.status.zero_()
    out = x.attend(q, [90, 0, 10, 40, 30], [4, 0, 4, 4, 4], parents, block_table=x.table[[0, 0, 1, 2, 3]].contiguous(),
                   max_ctx=128) if x.page else None
    assert int(x.status) == cp.CP_DEV_BOUNDS and torch.equal(out, want)


@pytest.mark.parametrize("kw", BOTH)
def test_padded_batch_and_oversized_tree(kw):
    heads, kw = kw["heads"], {k: v for k, v in kw.items() if k != "heads"}
    x = Cache(BF16, heads, 2, 256, 0, **kw)
    x.fill([100, 240])
    rows, past = [5, 129], [90, 100]
    q = x.queries(140)  # 134 rows and six of padding
    parents = [tree(5, "heap"), tree(129, "heap")]
    out = x.attend(q, past, rows, parents, max_ctx=256)
    assert int(x.status) == cp.CP_DEV_BOUNDS
    assert torch.isnan(out[5:]).all()
    x.check(q[:5], out[:5], past[:1], rows[:1], parents[:1])
    x.status.zero_()
    out = x.attend(q, past, [5, 128], [parents[0], parents[1][:128]], max_ctx=256)
    assert int(x.status) == 0 and torch.isnan(out[133:]).all()
    x.check(q, out, past, [5, 128], [parents[0], parents[1][:128]])


def test_latent_commit_advances_lengths():
    rows, past = [1, 4], [30, 7]
    x = Cache(BF16, 4, 2, 64, latent=128, rope=16)
    x.fill([p + r for p, r in zip(past, rows)])
    q, lens = x.queries(5), ints(past)
    out = x.attend(q, lens, rows, commit=True, max_ctx=40)
    assert lens.tolist() == [31, 11]
    x.check(q, out, past, rows)
    lens = ints(past)
    x.attend(x.queries(2), lens, [1, 1], uniform=True, commit=True, max_ctx=40)
    assert lens.tolist() == [31, 8]


@pytest.mark.parametrize("page", [0, 16])
def test_steps_one_behind_another(page):
    """Append, attention and the lengths' advance, 40 steps without a wait, the workspace and the lengths shared: bit for
    bit what the same steps give with a wait after each call."""
    n, heads, steps, past = 5, 32, 40, [0, 700, 61, 2000, 127]
    g = torch.Generator().manual_seed(5)
    rows = torch.randn(steps, n, 512 + 64, generator=g).to(BF16).cuda()
    q = torch.randn(steps, n, heads, 512 + 64, generator=g).to(BF16).cuda()
    kept = []
    for wait in (lambda: None, torch.cuda.synchronize):
        x = Cache(BF16, heads, n, 2100, page, latent=512, rope=64)
        x.fill(past)
        lens, out = ints(past), torch.full((steps, n, heads, 512), float("nan"), dtype=BF16, device="cuda")
        ws = torch.full((cp.cp_workspace_size_latent(x.desc, n, 2100, n),), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for i in range(steps):
            call = dict(block_table=x.table, dev_status=x.status)
            cp.cp_latent_append(x.desc, cp.qk_prep(rot_dim=0), rows[i, :, :512], rows[i, :, 512:], x.x, lens, n, n, 2100, **call)
            wait()
            cp.cp_latent_attn(x.desc, q[i], x.x, lens, n, n, 2100, out[i], ws, commit=True, **call)
            wait()
        assert lens.tolist() == [p + steps for p in past] and int(x.status) == 0
        x.check(q[-1], out[-1], [p + steps - 1 for p in past], [1] * n)
        kept.append(out)
    assert torch.equal(*kept)


def test_trees_one_behind_another():
    """A draft's rows in, its attention, the accepted path to its places and the lengths' advance, 20 times without a wait."""
    n, rows, rounds, past = 4, 9, 20, [0, 300, 1000, 63]
    parents = tree(rows, "heap")
    g = torch.Generator().manual_seed(6)
    q = torch.randn(rounds, n * rows, 8, 64, generator=g).to(F16).cuda()
    new = torch.randn(rounds, 2, n * rows, 2, 64, generator=g).to(F16).cuda()
    path = ints([[0, 2, 7]] * n)
    count, par = ints([1, 3, 2, 0]), ints(parents * n)
    kept = []
    for wait in (lambda: None, torch.cuda.synchronize):
        x = Cache(F16, 8, n, 1200, 16, kv=2, d=64)
        x.fill(past)
        lens, out = ints(past), torch.full((rounds, n * rows, 8, 64), float("nan"), dtype=F16, device="cuda")
        ws = torch.full((cp.cp_workspace_size_tree(x.desc, n * rows, 1200, n),), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for i in range(rounds):
            cp.cp_kv_append(x.desc, new[i, 0], new[i, 1], rows, x.k, x.v, lens, 1150, x.table, x.status)
            wait()
            cp.cp_tree_attn(x.desc, q[i], x.k, x.v, lens, par, n, n * rows, 1200, out[i], ws, block_table=x.table,
                            dev_status=x.status)
            wait()
            cp.cp_tree_commit(x.desc, x.k, x.v, path, count, lens, n, 3, 1200, block_table=x.table, dev_status=x.status)
            wait()
        assert lens.tolist() == [p + rounds * c for p, c in zip(past, count.tolist())] and int(x.status) == 0
        kept.append(out)
    assert torch.equal(*kept) and torch.isfinite(kept[0].float()).all()


@pytest.mark.parametrize("kw", BOTH)
def test_capture_replay_and_two_streams(kw):
    """A captured call reads its buffers' present contents; calls on two streams keep apart with workspaces of their own."""
    heads, kw = kw["heads"], {k: v for k, v in kw.items() if k != "heads"}
    rows, past = [12, 7], [3000, 100]
    x = Cache(BF16, heads, 2, 3200, 64, **kw)
    x.fill([p + r + 40 for p, r in zip(past, rows)])
    parents = [tree(r, "heap") for r in rows]
    q, lens, cr = x.queries(19), ints(past), cu(rows)
    par = ints([p for y in parents for p in y])
    size = (cp.cp_workspace_size_latent if x.latent else cp.cp_workspace_size_tree)(x.desc, 19, 3200, 2)
    ws = [torch.empty(max(size, 16), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [x.empty_out(19) for _ in range(2)]

    def call(i):
        args = dict(cu_rows=cr, block_table=x.table, dev_status=x.status)
        if x.latent:
            cp.cp_latent_attn(x.desc, q, x.x, lens, 2, 19, 3200, outs[i], ws[i], parents=par, commit=False, **args)
        else:
            cp.cp_tree_attn(x.desc, q, x.k, x.v, lens, par, 2, 19, 3200, outs[i], ws[i], **args)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(0)
    torch.cuda.current_stream().wait_stream(s)
    x.check(q, outs[0], past, rows, parents)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(0)
    now = [2990, 64]
    lens.copy_(ints(now))
    q.copy_(x.queries(19, seed=9))
    par.copy_(ints(tree(12, "random", 5) + tree(7, "star")))
    outs[0].fill_(float("nan"))
    for _ in range(3):
        g.replay()
    x.check(q, outs[0], now, rows, [tree(12, "random", 5), tree(7, "star")])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                call(i)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and int(x.status) == 0


def test_latent_offsets_past_32_bits():
    """A cache whose last slots lie past 2^32 bytes."""
    c, r, page = 512, 64, 64
    pages = 2 ** 32 // (page * 576 * 2) + 40
    x = Cache(BF16, 8, 1, 128, page, latent=c, rope=r)
    big = torch.full((pages, page, 576), float("nan"), dtype=BF16, device="cuda")
    x.desc.num_pages = x.pages = pages
    x.x = big
    x.arrays = [big]
    x.table = ints([[pages - 1, pages - 20, 3]])
    x.desc.max_blocks = 3
    x.fill([150])
    q = x.queries(4)
    out = x.attend(q, [146], [4])
    x.check(q, out, [146], [4])
    assert int(x.status) == 0
    cap = 2 ** 32 // (576 * 2) + 700
    y = Cache(F16, 4, 2, cap, latent=c, rope=r)  # the second sequence lies past 2^32
    y.fill([10, 300])
    q = y.queries(2)
    out = y.attend(q, [9, 299], [1, 1], uniform=True, max_ctx=400)
    y.check(q, out, [9, 299], [1, 1])


# ------------------------------------------------------------------ expanded form

def _expanded(dtype, heads, dn, r, dv, rows, keys, seed=0, uniform=False, fused=True, scale=0.0, poison=None):
    g = torch.Generator().manual_seed(seed)
    t, n = sum(rows), sum(keys)
    q = torch.randn(t, heads, dn + r, generator=g).to(dtype).cuda()
    kv = torch.randn(n, heads, dn + dv, generator=g).to(dtype).cuda()
    kr = torch.randn(n, r + 8, generator=g).to(dtype).cuda()[:, :r] if r else None
    k, v = kv[..., :dn], kv[..., dn:]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    if poison:
        poison(k, kr, v)
    out = torch.full((t, heads, dv), float("nan"), dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    desc = cp.latent_desc(dtype, 1, heads, 512, r, nope_dim=dn, v_dim=dv, capacity=1, scale=scale)
    cp.cp_latent_chunk_attn(desc, q, k, kr, v, out, len(rows), t, n, cu_rows=None if uniform else cu(rows),
                            cu_keys=None if uniform else cu(keys), dev_status=status)
    return q, k, kr, v, out, status


def _check_expanded(dtype, q, k, kr, v, out, rows, keys, scale=0.0):
    r0 = k0 = 0
    scale = scale or q.shape[2] ** -0.5
    if q.shape[1] > 40:  # of many heads, some
        q, k, v, out = (x[:, 1::61] for x in (q, k, v, out))
    for r, n in zip(rows, keys):
        kk = f64(k[k0:k0 + n])
        if kr is not None:
            kk = np.concatenate([kk, np.broadcast_to(f64(kr[k0:k0 + n])[:, None], (n, kk.shape[1], kr.shape[1]))], -1)
        see = np.arange(n) <= (n - r + np.arange(r))[:, None]
        assert off(dtype, f64(q[r0:r0 + r]), kk, f64(v[k0:k0 + n]), see, scale, f64(out[r0:r0 + r])) <= 1.0
        r0, k0 = r0 + r, k0 + n


@pytest.mark.parametrize("dtype,heads,dn,r,dv", [(BF16, 4, 128, 64, 128), (F16, 3, 64, 32, 64), (BF16, 1, 128, 16, 64),
                                                 (F16, 2, 64, 0, 128), (BF16, 5, 64, 48, 64),
                                                 # several lone Q tiles a CTA, then heads enough for pairs of them
                                                 (BF16, 40, 128, 64, 128), (F16, 90, 64, 32, 64), (BF16, 60, 128, 0, 64),
                                                 (BF16, 200, 128, 64, 128), (F16, 201, 64, 32, 64), (BF16, 210, 128, 16, 64),
                                                 (F16, 195, 64, 0, 128), (BF16, 220, 64, 0, 64)])
def test_expanded_chunks(dtype, heads, dn, r, dv):
    rows, keys = [1, 300, 37, 128, 2], [1, 300, 700, 257, 129]
    q, k, kr, v, out, status = _expanded(dtype, heads, dn, r, dv, rows, keys)
    assert int(status) == 0
    _check_expanded(dtype, q, k, kr, v, out, rows, keys)


@pytest.mark.parametrize("rows,keys", [(1, 1), (127, 127), (128, 128), (129, 129), (255, 400), (257, 1025), (64, 64)])
@pytest.mark.parametrize("heads", [2, 130, 260])
def test_expanded_equal_rows(rows, keys, heads):
    q, k, kr, v, out, status = _expanded(BF16, heads, 128, 64, 128, [rows] * 3, [keys] * 3, uniform=True, fused=False, scale=0.3)
    assert int(status) == 0
    _check_expanded(BF16, q, k, kr, v, out, [rows] * 3, [keys] * 3, scale=0.3)


@pytest.mark.parametrize("heads", [2, 70, 260])
def test_expanded_rows_that_see_nothing(heads):
    """More rows than keys: the first rows see none and get zeros; a sequence without keys gets zeros throughout."""
    rows, keys = [300, 5, 140], [10, 0, 139]
    q, k, kr, v, out, status = _expanded(F16, heads, 64, 32, 64, rows, keys)
    assert int(status) == 0
    assert (out[:290] == 0).all() and (out[300:305] == 0).all() and (out[305] == 0).all()
    _check_expanded(F16, q, k, kr, v, out, rows, keys)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("heads", [2, 80, 310])
def test_expanded_non_finite_values(value, heads):
    """A value that is not finite reaches the rows that see its key, and neither the earlier ones nor the sequence before."""
    rows, keys = [150, 300], [150, 333]
    clean = _expanded(BF16, heads, 128, 64, 128, rows, keys)[4]
    for at in (150 + 33, 150 + 40, 150 + 200, 482):
        def poison(k, kr, v):
            v[at, 1, 5] = value
        out = _expanded(BF16, heads, 128, 64, 128, rows, keys, poison=poison)[4]
        first = max(0, at - 150 - 33) + 150  # the first row that sees it
        assert torch.equal(out[:first], clean[:first]) and torch.equal(out[:, 0], clean[:, 0])
        assert (~torch.isfinite(out[first:, 1].float())).any(-1).all()
    # In a key: the rows that see it, and no other; an infinite score of -inf weighs nothing.
    def poison_k(k, kr, v):
        kr[150 + 60, 3] = value
    q, _, _, _, out, _ = _expanded(BF16, heads, 128, 64, 128, rows, keys, poison=poison_k)
    first = 150 + 60 - 33
    assert torch.equal(out[:first], clean[:first])
    lost = ~torch.isfinite(out[first:].float()).all(-1)
    assert lost.all() if value != value else torch.equal(lost, q[first:, :, 128 + 3] > 0)


@pytest.mark.parametrize("heads", [2, 100, 520])
def test_expanded_bad_offsets_and_padding(heads):
    rows, keys = [40, 60, 50], [80, 90, 70]
    t, n = 150, 240
    q, k, kr, v, want, _ = _expanded(BF16, heads, 128, 64, 128, rows, keys)
    desc = cp.latent_desc(BF16, 1, heads, 512, 64, capacity=1)
    for cr, ck, skipped in (([0, 40, 100, 150], [0, 80, 80 - 1, 240], {1}), ([0, 40, 100, 150], [0, 80, 170, 241], {2}),
                            ([0, 40, 40, 150], [0, 80, 170, 240], None), ([0, 40, 100, 100], [0, 80, 170, 240], {2})):
        out = torch.full_like(want, 7.0)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        cp.cp_latent_chunk_attn(desc, q, k, kr, v, out, 3, t, n, cu_rows=ints(cr), cu_keys=ints(ck), dev_status=status)
        assert int(status) == cp.CP_DEV_BOUNDS
        if skipped:
            for s, (a, b) in enumerate(((0, 40), (40, 100), (100, 150))):
                if s in skipped:
                    assert (out[a:b] == 7.0).all()
                elif ck[s] == [0, 80, 170][s] and ck[s + 1] == [80, 170, 240][s]:
                    assert torch.equal(out[a:b], want[a:b])
    out = torch.full_like(want, 7.0)  # a padded batch
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cp.cp_latent_chunk_attn(desc, q, k, kr, v, out, 2, t, n, cu_rows=ints([0, 40, 100]), cu_keys=ints([0, 80, 170]),
                            dev_status=status)
    assert int(status) == 0 and torch.equal(out[:100], want[:100]) and (out[100:] == 7.0).all()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("page", [0, 32])
def test_a_latent_layer_from_prompt_to_accepted_draft(page):
    """One layer of a latent model: a prompt in chunks (append, expansion of the cached latents, expanded attention), a
    drafted tree (append at the nodes' depths, absorbed attention), the accepted path's commit, and the next token; each
    step against 64 bits from what the cache then holds, and the two forms against one another."""
    dt, heads, c, r, dn, dv = BF16, 8, 256, 32, 64, 64
    g = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w_k, w_v = (rnd(c, heads, dn) / c ** 0.5).to(dt).cuda(), (rnd(c, heads, dv) / c ** 0.5).to(dt).cuda()
    weight = (1 + 0.1 * rnd(c)).to(dt).cuda()
    freq = (10000.0 ** (-torch.arange(0, r, 2) / r)).float().cuda()
    x = Cache(dt, heads, 1, 512, page, latent=c, rope=r, nope_dim=dn, v_dim=dv)
    prep, lens, scale = cp.qk_prep(r), ints([0]), (dn + r) ** -0.5
    extra = dict(block_table=x.table, dev_status=x.status)

    def project(t):
        return rnd(t, c + r).to(dt).cuda(), rnd(t, heads, dn + r).to(dt).cuda()

    def append(proj, q, positions=None):
        t = q.shape[0]
        cp.cp_latent_append(x.desc, prep, proj[:, :c], proj[:, c:], x.x, lens, 1, t, 512, weight=weight, inv_freq=freq,
                            positions=positions, q_rope=q[..., dn:], q_out=q[..., dn:], **extra)

    past = 0
    for t in (200, 113):  # the prompt's chunks
        proj, q = project(t)
        append(proj, q)
        held = x.at(x.x, 0, 0, past + t)[:, 0]
        keys = (held[:, :c].float() @ w_k.float().flatten(1)).to(dt).unflatten(1, (heads, dn))
        values = (held[:, :c].float() @ w_v.float().flatten(1)).to(dt).unflatten(1, (heads, dv))
        out = torch.empty(t, heads, dv, dtype=dt, device="cuda")
        cp.cp_latent_chunk_attn(x.desc, q, keys, held[:, c:], values, out, 1, t, past + t, dev_status=x.status)
        _check_expanded(dt, q, keys, held[:, c:], values, out, [t], [past + t])
        # The absorbed form of the last rows: the same attention with the maps on the other side.  Its queries, latents'
        # mixture and product are rounded to 16 bits once more: three half steps of values of order one.
        wide = torch.empty(4, heads, c + r, dtype=dt, device="cuda")
        wide[..., :c] = torch.einsum("thd,chd->thc", q[-4:, :, :dn].float(), w_k.float()).to(dt)
        wide[..., c:] = q[-4:, :, dn:]
        got = x.attend(wide, [past + t - 4], [4])
        x.check(wide, got, [past + t - 4], [4])
        both = torch.einsum("thc,chd->thd", got.float(), w_v.float())
        assert (both - out[-4:].float()).abs().max() < 8 * half_step(dt) * max(1.0, float(out[-4:].abs().max()))
        past += t
        lens += t
    parents = tree(21, "heap")
    depth = [0] * 21
    for i, p in enumerate(parents):
        depth[i] = depth[p] + 1 if p >= 0 else 0
    proj, q = project(21)
    append(proj, q, positions=ints([past + e for e in depth]))
    wide = torch.randn(21, heads, c + r, generator=g).to(dt).cuda()
    out = x.attend(wide, [past], [21], [parents])
    x.check(wide, out, [past], [21], [parents])
    path = [0, 2, 8]
    kept = x.at(x.x, 0, past, 21)[path].clone()
    cp.cp_latent_tree_commit(x.desc, x.x, ints([path + [-1]]), ints([3]), lens, 1, 4, 512, **extra)
    assert lens.tolist() == [past + 3] and torch.equal(x.at(x.x, 0, past, 3), kept)
    proj, q = project(1)
    append(proj, q)
    wide = torch.randn(1, heads, c + r, generator=g).to(dt).cuda()
    out = x.attend(wide, lens, [1], uniform=True, commit=True, max_ctx=512)
    x.check(wide, out, [past + 3], [1])
    assert lens.tolist() == [past + 4] and int(x.status) == 0
