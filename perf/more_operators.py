"""Operators of latent caches and of drafted trees, as a user's program calls them:

  latent_append  norm of the latents, rotary position of the shared keys and the queries, rows into a latent cache
  latent         attention over a latent cache (absorbed form): single tokens, short chunks, drafted trees
  expanded       attention of prompt chunks over keys and values expanded from the latents
  tree           attention of a drafted tree's nodes over a K/V cache
  commit         the accepted path's rows moved to their places in a K/V or latent cache

`run` computes them in elementary torch operations, or with `own` set through
this package's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
THETA = 10000.0


# ------------------------------------------------------------------ cases

def case_of(name, op, dtype, heads, **kw):
    """A case: `seqs` sequences of `rows` rows (`ragged`: each has some fewer than the one before), their cached
    lengths spread over [past_lo, past_hi]; page 0 is a contiguous cache.  A latent cache holds `latent` + `rope`
    channels a token for all heads, a K/V cache kv heads of d.  branch 0: rows follow one another; else node i of a
    drafted tree is a child of node (i - 1) // branch."""
    c = dict(op=op, dtype=dtype, heads=heads, kv=0, d=0, latent=0, rope=0, nope=0, vdim=0, seqs=1, rows=1, ragged=False,
             past_lo=0, past_hi=0, page=0, branch=0, interleaved=False, accept=0)
    if name:
        c["name"] = name
    c.update(kw)
    return c


def listed():
    return [
        # The smallest call: one sequence's next token.
        case_of("latent_append_token", "latent_append", "bf16", 32, latent=512, rope=64, nope=128, past_lo=1024, past_hi=1024),
        # A full budget of prompt tokens into a paged latent cache.
        case_of("latent_append_chunk", "latent_append", "bf16", 32, latent=512, rope=64, nope=128, seqs=4, rows=2048,
                past_lo=100, past_hi=6000, page=64),
        # One sequence decodes one token over a short context: latency.
        case_of("latent_token", "latent", "bf16", 32, latent=512, rope=64, past_lo=1024, past_hi=1024),
        # A batch of long conversations decodes a token each: the cache's bytes.
        case_of("latent_decode", "latent", "bf16", 32, latent=512, rope=64, seqs=32, past_lo=12000, past_hi=40000, page=64),
        # Drafted trees of three conversations, a smaller model.
        case_of("latent_tree", "latent", "f16", 16, latent=256, rope=32, seqs=3, rows=27, ragged=True, past_lo=100,
                past_hi=9000, page=16, branch=3),
        # A prompt's last few tokens for many heads over a long cached prefix.
        case_of("latent_chunk", "latent", "bf16", 64, latent=512, rope=64, seqs=2, rows=45, past_lo=8000, past_hi=16000),
        # Short prompts of different lengths, some after a cached prefix.
        case_of("expanded_ragged", "expanded", "f16", 8, nope=64, rope=32, vdim=64, seqs=5, rows=333, ragged=True,
                past_lo=0, past_hi=1500),
        # One launch of a deep prompt chunk: the tensor cores.
        case_of("expanded_chunk", "expanded", "bf16", 32, nope=128, rope=64, vdim=128, rows=8128, past_lo=8128, past_hi=8128),
        # One conversation's drafted tree over a short context: latency.
        case_of("tree_one", "tree", "bf16", 32, kv=8, d=128, rows=16, past_lo=1024, past_hi=1024, branch=2),
        # A batch's drafted trees over a paged cache: the cache's bytes.
        case_of("tree_batch", "tree", "bf16", 32, kv=8, d=128, seqs=24, rows=61, past_lo=4000, past_hi=24000, page=16, branch=4),
        # One conversation's accepted path in a latent cache.
        case_of("commit_one", "commit", "bf16", 32, latent=512, rope=64, rows=32, accept=5, past_lo=1024, past_hi=1024),
        # A batch's accepted paths in a paged K/V cache.
        case_of("commit_batch", "commit", "bf16", 32, kv=8, d=128, seqs=64, rows=61, accept=8, past_lo=512, past_hi=4000, page=16),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["latent_append", "latent", "latent", "expanded", "tree", "tree", "commit"])
    dtype = rng.choice(["bf16", "f16"])
    kw = dict(page=rng.choice([0, 16, 32, 64, 128]), ragged=rng.random() < 0.5, seqs=_spread(rng, 1, 32))
    kw["past_lo"] = _spread(rng, 1, 4000) - 1
    kw["past_hi"] = kw["past_lo"] + _spread(rng, 1, 16000) - 1
    if op in ("latent_append", "latent"):
        kw.update(latent=rng.choice([128, 256, 512]), rope=rng.choice([16, 32, 64]))
    if op == "latent_append":
        heads = _spread(rng, 1, 64)
        kw.update(nope=rng.choice([64, 128]), rows=_spread(rng, 1, 8192 // kw["seqs"]), interleaved=rng.random() < 0.4, past_hi=min(kw["past_hi"], 8000))
        kw["past_lo"] = min(kw["past_lo"], kw["past_hi"])
    elif op == "latent":
        heads = _spread(rng, 1, 128)
        kw["branch"] = rng.choice([0, 0, 2, 3, 4])
        kw["rows"] = _spread(rng, 1, max(1, min(100, 1024 // (kw["seqs"] * max(1, heads // 8)))))
        if rng.random() < 0.4:  # plain decoding
            kw.update(rows=1, branch=0)
    elif op == "expanded":
        heads = _spread(rng, 1, 32)
        kw.update(nope=rng.choice([64, 128]), rope=rng.choice([16, 32, 64]), vdim=rng.choice([64, 128]), page=0,
                  seqs=_spread(rng, 1, 8))
        kw["rows"] = _spread(rng, 2, 4096 // kw["seqs"])
        kw["past_hi"] = min(kw["past_hi"], 8000)
        kw["past_lo"] = min(kw["past_lo"], kw["past_hi"])
    else:
        kw.update(kv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]), branch=rng.choice([1, 2, 3, 4]),
                  rows=_spread(rng, 2, 100), seqs=_spread(rng, 1, 24))
        heads = kw["kv"] * rng.choice([1, 2, 3, 4, 8])
        if op == "commit":
            kw["accept"] = _spread(rng, 1, min(12, kw["rows"] - 1))
            if rng.random() < 0.4:
                kw.update(kv=0, d=0, latent=rng.choice([128, 256, 512]), rope=rng.choice([16, 32, 64]))
    return case_of("", op, dtype, heads, **kw)


def layout(c):
    """Rows and cached lengths of the case's sequences, and a bound on their sum."""
    n = c["seqs"]
    rows = [max(1, c["rows"] - (c["rows"] // 9 + 1) * (i % 8)) if c["ragged"] else c["rows"] for i in range(n)]
    span = c["past_hi"] - c["past_lo"]
    past = [c["past_lo"] + (span * ((i * 37) % n)) // max(1, n - 1) for i in range(n)]
    return rows, past, max(r + p for r, p in zip(rows, past))


def parent_of(c, i):
    return (i - 1) // c["branch"] if i and c["branch"] else i - 1


def accepted(c, r):
    """The path of up to `accept` nodes that is taken of a tree of r: its first node and the last ones, so that no
    row is moved to another's place."""
    k = min(c["accept"], max(1, r // 2))
    return [0] + [r - k + 1 + i for i in range(k - 1)]


def work(c):
    rows, past, _ = layout(c)
    t, h, d, lat, rope = sum(rows), c["heads"], c["d"], c["latent"], c["rope"]
    es = 2
    keys = sum(r + p for r, p in zip(rows, past))
    depth = []  # nodes on the way to node i, itself among them
    for i in range(max(rows)):
        p = parent_of(c, i)
        depth.append(1 + (depth[p] if p >= 0 else 0))
    seen = sum(r * p + sum(depth[:r]) for r, p in zip(rows, past))
    if c["op"] == "latent_append":
        return {"bytes": 2 * t * (lat + rope + h * rope) * es, "flops": t * (4 * lat + 4 * rope * (h + 1))}
    if c["op"] == "latent":
        return {"bytes": (keys * (lat + rope) + t * h * (2 * lat + rope)) * es, "flops": 2 * seen * h * (2 * lat + rope)}
    if c["op"] == "expanded":
        dn, dv = c["nope"], c["vdim"]
        return {"bytes": (t * h * (dn + rope + dv) + keys * (h * (dn + dv) + rope)) * es,
                "flops": 2 * seen * h * (dn + rope + dv)}
    if c["op"] == "tree":
        return {"bytes": 2 * (c["kv"] * keys + t * h) * d * es, "flops": 4 * seen * h * d}
    moved = sum(len(accepted(c, r)) - 1 for r in rows)
    row = lat + rope if lat else 2 * c["kv"] * d
    return {"bytes": 2 * moved * row * es + 4 * sum(len(accepted(c, r)) + 2 for r in rows), "flops": 0}


# ------------------------------------------------------------------ inputs

class Inputs:
    """What a user's program has in hand before the call."""


def prepare(c, seed):
    dev, dt, op = "cuda", DTYPES[c["dtype"]], c["op"]
    h, d, lat, rope, page = c["heads"], c["d"], c["latent"], c["rope"], c["page"]
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=gen, device=dev, dtype=dt)

    st = Inputs()
    st.case, st.dtype = c, dt
    st.rows, st.past, st.max_ctx = layout(c)
    n, t = len(st.rows), sum(st.rows)
    st.n, st.t = n, t
    starts = [sum(st.rows[:i]) for i in range(n + 1)]
    st.cu_rows = torch.tensor(starts, dtype=torch.int32, device=dev)
    st.uniform = len(set(st.rows)) == 1
    st.lens = torch.tensor(st.past, dtype=torch.int32, device=dev)
    st.parents = None
    if c["branch"]:
        st.parents = torch.tensor([parent_of(c, i) for r in st.rows for i in range(r)], dtype=torch.int32, device=dev)

    if op == "expanded":  # keys and values of whole contexts, as one product with the latents gives them
        keys = [r + p for r, p in zip(st.rows, st.past)]
        st.keys = keys
        st.cu_keys = torch.tensor([sum(keys[:i]) for i in range(n + 1)], dtype=torch.int32, device=dev)
        st.nk = sum(keys)
        st.q = randn(t, h, c["nope"] + rope)
        kv = randn(st.nk, h, c["nope"] + c["vdim"])
        st.k_nope, st.v = kv[..., :c["nope"]], kv[..., c["nope"]:]
        st.k_rope = randn(st.nk, rope)
        st.out = torch.zeros(t, h, c["vdim"], dtype=dt, device=dev)
        if own:
            import chunked_prefill_causal_cp_gb300 as cp
            st.desc = cp.latent_desc(dt, n, h, 512, rope, nope_dim=c["nope"], v_dim=c["vdim"], capacity=st.max_ctx)
        return st

    # The cache: contiguous at a capacity with room to spare, or pages dealt at random.
    st.cap = -(-(st.max_ctx + 64) // 128) * 128
    st.table = None
    if page:
        st.blocks = st.cap // page
        need = [-(-(r + p) // page) for r, p in zip(st.rows, st.past)]
        st.pages = sum(need)
        perm = torch.randperm(st.pages, generator=host).tolist()
        first = [sum(need[:i]) for i in range(n)]
        st.table = torch.tensor([perm[f:f + k] + [-1] * (st.blocks - k) for f, k in zip(first, need)], dtype=torch.int32, device=dev)
    lead, slots_ = ((st.pages,), page) if page else ((n,), st.cap)
    empty = op == "latent_append"
    if lat:
        st.cache = torch.zeros(*lead, slots_, lat + rope, dtype=dt, device=dev) if empty else randn(*lead, slots_, lat + rope)
    else:
        st.k_cache, st.v_cache = randn(*lead, c["kv"], slots_, d), randn(*lead, c["kv"], slots_, d)
    if op == "latent_append":
        st.proj = randn(t, lat + rope)  # one projection gives the latents and the shared keys
        st.weight = (1 + 0.2 * randn(lat).float()).to(dt)
        st.inv_freq = (THETA ** (-torch.arange(0, rope, 2, device=dev, dtype=torch.float64) / rope)).float()
        st.q = randn(t, h, c["nope"] + rope)  # the queries' projection, with the channels to rotate behind the others
        st.q_out = torch.zeros(t, h, lat + rope, dtype=dt, device=dev)[..., lat:]  # behind the absorbed queries' place
    elif op == "latent":
        st.q = randn(t, h, lat + rope)
        st.scale = 1 / math.sqrt(lat // 4 + rope)  # of the heads that the queries were absorbed from
        st.out = torch.zeros(t, h, lat, dtype=dt, device=dev)
    elif op == "tree":
        st.q = randn(t, h, d)
        st.scale = 1 / math.sqrt(d)
        st.out = torch.zeros(t, h, d, dtype=dt, device=dev)
    elif op == "commit":
        paths = [accepted(c, r) for r in st.rows]
        st.most = max(len(p) for p in paths)
        st.path = torch.tensor([p + [-1] * (st.most - len(p)) for p in paths], dtype=torch.int32, device=dev)
        st.count = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=dev)
    if own:
        import chunked_prefill_causal_cp_gb300 as cp
        kind = dict(kind=cp.CP_CACHE_PAGED, page_size=page, num_pages=st.pages, max_blocks=st.blocks) if page else \
            dict(kind=cp.CP_CACHE_CONTIG, capacity=st.cap)
        if lat:
            st.desc = cp.latent_desc(dt, n, h, lat, rope, scale=st.scale if op == "latent" else 0.0, **kind)
        else:
            st.desc = cp.layer_desc(dt, n, h, c["kv"], d, **kind)
        st.call = dict(block_table=st.table)
        if op != "commit":
            st.call["cu_rows"] = None if st.uniform else st.cu_rows
        if op == "latent_append":
            st.prep = cp.qk_prep(rope, interleaved=c["interleaved"], eps=EPS)
        elif op == "latent":
            st.ws = torch.empty(max(16, cp.cp_workspace_size_latent(st.desc, t, st.max_ctx, n)), dtype=torch.uint8, device=dev)
        elif op == "tree":
            st.ws = torch.empty(max(16, cp.cp_workspace_size_tree(st.desc, t, st.max_ctx, n)), dtype=torch.uint8, device=dev)
    return st


# ------------------------------------------------------------------ one pass

def places(st):
    """Where each of the call's rows lives: two indexes of the cache, and its position."""
    seq = torch.repeat_interleave(torch.arange(st.n, device=st.lens.device), (st.cu_rows[1:] - st.cu_rows[:-1]).long(),
                                  output_size=st.t)
    pos = st.lens[seq].long() + torch.arange(st.t, device=seq.device) - st.cu_rows[seq].long()
    if st.table is None:
        return seq, pos, pos
    page = st.case["page"]
    return st.table[seq, pos // page].long(), pos % page, pos


def rotated(x, pos, inv_freq, interleaved):
    """Rotation of [t, heads, r] in 32 bits (angles in 64), rounded once."""
    u = pos.double()[:, None] * inv_freq.double()
    cos, sin = torch.cos(u).float()[:, None], torch.sin(u).float()[:, None]
    y = x.float()
    z, r = torch.empty_like(y), x.shape[-1]
    lo, hi = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    a, b = y[..., lo], y[..., hi]
    z[..., lo], z[..., hi] = a * cos - b * sin, b * cos + a * sin
    return z.to(x.dtype)


def padded(st, rows):
    """Indexes [s, r] of the sequences' rows, those past a sequence's own clamped, and which are real."""
    i = torch.arange(rows, device=st.lens.device)
    at = st.cu_rows[:-1].long()[:, None] + i
    return at.clamp(max=st.t - 1), i < (st.cu_rows[1:] - st.cu_rows[:-1])[:, None]


def hidden(st, at, keys):
    """[s, r, keys]: what a row does not see."""
    s, r = at.shape
    i = torch.arange(r, device=at.device)
    if st.parents is None:
        return torch.arange(keys, device=at.device) > st.lens.long()[:, None, None] + i[:, None]
    p = st.parents[at].long()
    reach = torch.eye(r, device=at.device).expand(s, r, r).clone()
    reach += (p[..., None] == i).float()
    for _ in range(max(1, (r - 1).bit_length())):
        reach = (torch.matmul(reach, reach) > 0).float()
    own_key = torch.arange(keys, device=at.device) - st.lens.long()[:, None]  # [s, keys]
    among = torch.gather(reach > 0, 2, own_key.clamp(0, r - 1)[:, None].expand(s, r, keys))
    return ~torch.where((own_key < 0)[:, None], torch.ones_like(among), among & (own_key < r)[:, None])


def softmax_(p):
    p -= p.amax(-1, keepdim=True)
    p.exp_()
    p /= p.sum(-1, keepdim=True)
    return p


def gathered(st, x):
    """The first max_ctx positions of every sequence of a cache array, rows past a sequence's own as zeros:
    [s, max_ctx, ...] or [s, kv, max_ctx, d]."""
    heads = x.dim() == 4
    if st.table is None:
        y = x[:, :, :st.max_ctx] if heads else x[:, :st.max_ctx]
    else:
        b = -(-st.max_ctx // st.case["page"])
        y = x[st.table[:, :b].long().clamp(min=0)]  # [s, b, (kv,) page, d]
        y = y.transpose(1, 2).flatten(2, 3)[:, :, :st.max_ctx] if heads else y.flatten(1, 2)[:, :st.max_ctx]
    held = st.lens + (st.cu_rows[1:] - st.cu_rows[:-1])
    gone = torch.arange(st.max_ctx, device=x.device) >= held[:, None]
    return y.float().masked_fill(gone[:, None, :, None] if heads else gone[..., None], 0)


def run(st):
    c, op = st.case, st.case["op"]
    if own:
        import chunked_prefill_causal_cp_gb300 as cp
        if op == "latent_append":
            lat = c["latent"]
            cp.cp_latent_append(st.desc, st.prep, st.proj[:, :lat], st.proj[:, lat:], st.cache, st.lens, st.n, st.t,
                                st.max_ctx, weight=st.weight, inv_freq=st.inv_freq, q_rope=st.q[..., c["nope"]:],
                                q_out=st.q_out, **st.call)
            return st.cache, st.q_out
        if op == "latent":
            cp.cp_latent_attn(st.desc, st.q, st.cache, st.lens, st.n, st.t, st.max_ctx, st.out, st.ws,
                              parents=st.parents, commit=False, **st.call)
            return st.out
        if op == "expanded":
            cp.cp_latent_chunk_attn(st.desc, st.q, st.k_nope, st.k_rope, st.v, st.out, st.n, st.t, st.nk,
                                    cu_rows=st.cu_rows, cu_keys=st.cu_keys)
            return st.out
        if op == "tree":
            cp.cp_tree_attn(st.desc, st.q, st.k_cache, st.v_cache, st.lens, st.parents, st.n, st.t, st.max_ctx, st.out,
                            st.ws, **st.call)
            return st.out
        if c["latent"]:
            cp.cp_latent_tree_commit(st.desc, st.cache, st.path, st.count, st.lens, st.n, st.most, st.max_ctx,
                                     commit=False, **st.call)
            return st.cache
        cp.cp_tree_commit(st.desc, st.k_cache, st.v_cache, st.path, st.count, st.lens, st.n, st.most, st.max_ctx,
                          commit=False, **st.call)
        return st.k_cache, st.v_cache

    if op == "latent_append":
        i, j, pos = places(st)
        lat = c["latent"]
        y = st.proj[:, :lat].float()
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * st.weight.float()
        k = rotated(st.proj[:, None, lat:], pos, st.inv_freq, c["interleaved"])[:, 0]
        st.cache[i, j] = torch.cat([y.to(st.dtype), k], -1)
        return st.cache, rotated(st.q[..., c["nope"]:], pos, st.inv_freq, c["interleaved"])

    if op == "commit":
        e = torch.arange(st.most, device=st.lens.device)
        seq, e = torch.nonzero(e < st.count[:, None], as_tuple=True)
        src, dst = (st.lens[seq] + st.path[seq, e]).long(), (st.lens[seq] + e).long()
        if st.table is None:
            at = lambda p: (seq, p)  # noqa: E731
        else:
            at = lambda p: (st.table[seq, p // c["page"]].long(), p % c["page"])  # noqa: E731
        (i, j), (k, l) = at(src), at(dst)
        if c["latent"]:
            st.cache[k, l] = st.cache[i, j]
            return st.cache
        st.k_cache[k, :, l], st.v_cache[k, :, l] = st.k_cache[i, :, j], st.v_cache[i, :, j]
        return st.k_cache, st.v_cache

    if op == "expanded":
        out = []
        r0 = k0 = 0
        for r, n in zip(st.rows, st.keys):
            q = st.q[r0:r0 + r].float().transpose(0, 1) / math.sqrt(c["nope"] + c["rope"])  # [h, r, ..]
            p = torch.matmul(q[..., :c["nope"]], st.k_nope[k0:k0 + n].float().permute(1, 2, 0))
            p += torch.matmul(q[..., c["nope"]:], st.k_rope[k0:k0 + n].float().T)
            ar = torch.arange(n, device=q.device)
            p.masked_fill_(ar > ar[n - r:, None], -math.inf)
            out.append(torch.matmul(softmax_(p), st.v[k0:k0 + n].float().transpose(0, 1)).transpose(0, 1).to(st.dtype))
            del p
            r0, k0 = r0 + r, k0 + n
        return torch.cat(out)

    at, real = padded(st, max(st.rows))
    hide = hidden(st, at, st.max_ctx)
    q = st.q[at].float() * st.scale  # [s, r, h, ..]
    s, r, h, _ = q.shape
    if op == "latent":
        x = gathered(st, st.cache)
        p = torch.matmul(q.flatten(1, 2), x.transpose(1, 2)).unflatten(1, (r, h))
        p.masked_fill_(hide[:, :, None], -math.inf)
        o = torch.matmul(softmax_(p).flatten(1, 2), x[..., :c["latent"]]).unflatten(1, (r, h))
    else:
        k, v, kv = gathered(st, st.k_cache), gathered(st, st.v_cache), c["kv"]
        q = q.unflatten(2, (kv, h // kv)).transpose(1, 2).flatten(2, 3)  # [s, kv, r g, d]
        p = torch.matmul(q, k.transpose(2, 3)).unflatten(2, (r, h // kv))
        p.masked_fill_(hide[:, None, :, None], -math.inf)
        o = torch.matmul(softmax_(p).flatten(2, 3), v).unflatten(2, (r, h // kv)).transpose(1, 2).flatten(2, 3)
    return o[real].to(st.dtype)


# ------------------------------------------------------------------ in 64 bits

def exact(c, seed):
    """The definition, in 64 bits, sequence by sequence and head by head."""
    st = prepare(c, seed)
    f64, op, lat, rope, page = torch.float64, c["op"], c["latent"], c["rope"], c["page"]
    dev = st.lens.device

    def slots(s, first, count):  # of positions of sequence s: (index, slot)
        pos = torch.arange(first, first + count, device=dev)
        if not page:
            return torch.full_like(pos, s), pos
        return st.table[s].long()[torch.div(pos, page, rounding_mode="floor")], pos.remainder(page)

    if op == "commit":
        arrays = [x.to(f64) for x in ([st.cache] if lat else [st.k_cache.transpose(1, 2), st.v_cache.transpose(1, 2)])]
        for s in range(st.n):
            path = accepted(c, st.rows[s])
            i, j = slots(s, st.past[s], max(path) + 1)
            for x in arrays:
                moved = x[i[path], j[path]].clone()
                x[i[:len(path)], j[:len(path)]] = moved
        return arrays[0] if lat else tuple(x.transpose(1, 2).contiguous() for x in arrays)

    if op == "latent_append":
        cache, q_out = st.cache.to(f64), torch.empty(st.t, c["heads"], rope, dtype=f64, device=dev)
        y = st.proj.to(f64)
        norm = y[:, :lat] * (y[:, :lat].pow(2).sum(-1, keepdim=True) / lat + EPS).rsqrt() * st.weight.to(f64)
        r0 = 0
        for s, (r, p) in enumerate(zip(st.rows, st.past)):
            turn = torch.polar(torch.ones((), dtype=f64, device=dev),
                               torch.outer(torch.arange(p, p + r, device=dev, dtype=f64), st.inv_freq.to(f64)))

            def turned(x):  # [r, heads, rope]
                if c["interleaved"]:
                    z = torch.complex(x[..., 0::2].contiguous(), x[..., 1::2].contiguous()) * turn[:, None]
                    return torch.stack([z.real, z.imag], -1).flatten(-2)
                z = torch.complex(*(u.contiguous() for u in x.chunk(2, -1))) * turn[:, None]
                return torch.cat([z.real, z.imag], -1)

            i, j = slots(s, p, r)
            cache[i, j, :lat] = norm[r0:r0 + r]
            cache[i, j, lat:] = turned(y[r0:r0 + r, None, lat:])[:, 0]
            q_out[r0:r0 + r] = turned(st.q[r0:r0 + r, :, c["nope"]:].to(f64))
            r0 += r
        return cache, q_out

    out = torch.empty(st.out.shape, dtype=f64, device=dev)
    r0 = k0 = 0
    for s, (r, p) in enumerate(zip(st.rows, st.past)):
        n = p + r
        see = torch.zeros(r, n, dtype=torch.bool)
        see[:, :p] = True
        for i in range(r):  # a row sees what its parent sees, and itself
            up = parent_of(c, i)
            if up >= 0:
                see[i] = see[up]
            see[i, p + i] = True
        see = see.to(dev)
        if op != "expanded":
            i, j = slots(s, 0, n)
        for h in range(c["heads"]):
            q = st.q[r0:r0 + r, h].to(f64)
            if op == "expanded":
                k = torch.cat([st.k_nope[k0:k0 + n, h], st.k_rope[k0:k0 + n]], -1).to(f64)
                v, scale = st.v[k0:k0 + n, h].to(f64), (c["nope"] + rope) ** -0.5
            elif op == "latent":
                if h == 0:
                    k = st.cache[i, j].to(f64)
                    v, scale = k[:, :lat], st.scale
            else:
                g = h // (c["heads"] // c["kv"])
                if h % (c["heads"] // c["kv"]) == 0:
                    k, v, scale = st.k_cache[i, g, j].to(f64), st.v_cache[i, g, j].to(f64), st.scale
            score = torch.where(see, torch.mm(q, k.T) * scale, -math.inf)
            out[r0:r0 + r, h] = torch.mm(torch.softmax(score, -1), v)
        r0, k0 = r0 + r, k0 + n
    return out
