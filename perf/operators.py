"""Operators around the attention of a chunk, as a user's program calls them:

  rope         norm of every query and key head and rotary position, one pass
  rope_append  the same, with the keys and values put into their cache slots
  append       new rows into a cache held in 4 bits, and their values read back
  attn         causal attention of a call's rows over a cache held in 4 bits
  step         append + attention of a token-budget step over a cache held in 4 bits

`run` computes them in elementary torch operations, or with `own` set through
this package's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GROUP = 32  # channels that share a scale in the 4-bit cache
EPS = 1e-6


# ------------------------------------------------------------------ cases

def case_of(name, op, dtype, hq, hkv, d, **kw):
    """A case: one-row sequences (`ones`), then `chunks` sequences of up to `rows`
    rows, their cached lengths spread over [past_lo, past_hi]; page 0 is a
    contiguous cache."""
    c = dict(op=op, dtype=dtype, hq=hq, hkv=hkv, d=d, ones=0, chunks=0, rows=1, past_lo=0, past_hi=0, page=0,
             rot=0, interleaved=False, theta=10000.0, fused_qkv=False, norm=True)
    if name:
        c["name"] = name
    c.update(kw)
    return c


def listed():
    return [
        # The smallest call: one sequence decodes one token.
        case_of("rope_token", "rope", "bf16", 32, 8, 128, ones=1, past_lo=1024, past_hi=1024, rot=128),
        # A ragged step of a model that rotates part of its channels, in adjacent pairs, read from a fused projection.
        case_of("rope_ragged", "rope", "f16", 16, 4, 64, ones=29, chunks=3, rows=251, past_lo=5, past_hi=4000, rot=32,
                interleaved=True, fused_qkv=True),
        # A full budget of prompt tokens, far into a long document, read from a fused projection.
        case_of("rope_chunk", "rope", "bf16", 32, 8, 128, chunks=4, rows=2048, past_lo=90000, past_hi=120000, rot=128,
                theta=500000.0, fused_qkv=True),
        # A prompt chunk of a long prompt into a paged cache.
        case_of("rope_append_paged", "rope_append", "bf16", 32, 8, 128, chunks=4, rows=512, past_lo=100, past_hi=3400,
                page=16, rot=128, fused_qkv=True),
        # The fp32 example's prompt of 1000 tokens into a contiguous cache, no norm.
        case_of("rope_append_f32", "rope_append", "f32", 8, 8, 64, chunks=1, rows=1000, rot=64, norm=False),
        # A ragged step's rows into a paged 4-bit cache.
        case_of("append_q4_ragged", "append", "f16", 8, 8, 64, ones=30, chunks=3, rows=333, past_lo=0, past_hi=2000, page=16),
        # A full budget of prompt tokens into a contiguous 4-bit cache.
        case_of("append_q4_chunk", "append", "bf16", 32, 8, 128, chunks=4, rows=2048, past_lo=0, past_hi=6000),
        # One sequence decodes one token over a short context: latency.
        case_of("attn_q4_token", "attn", "bf16", 32, 8, 128, ones=1, past_lo=1024, past_hi=1024),
        # A few long conversations decode: the cache's bytes.
        case_of("attn_q4_long", "attn", "bf16", 32, 8, 128, ones=4, past_lo=100000, past_hi=100000, page=128),
        # One launch of a deep prompt chunk: the tensor cores.
        case_of("attn_q4_chunk", "attn", "bf16", 32, 8, 128, chunks=1, rows=8128, past_lo=8128, past_hi=8128),
        # Several short conversations decode a token each, append included.
        case_of("step_q4_decode", "step", "f16", 16, 16, 64, ones=7, past_lo=100, past_hi=2000, page=64),
        # A step of 64 running decodes and a prompt's chunk at a budget of 2048 tokens.
        case_of("step_q4_mixed", "step", "bf16", 32, 8, 128, ones=64, chunks=1, rows=1984, past_lo=512, past_hi=8191, page=16),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_append", "append", "attn", "step"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8])
    rope = op.startswith("rope")
    dtype = rng.choice(["bf16", "f16", "f32"] if rope else ["bf16", "f16"])
    kw = dict(page=rng.choice([0, 16, 32, 64, 128]))
    shape = rng.choice(["ones", "chunk", "mixed"])
    if shape != "chunk":
        kw["ones"] = _spread(rng, 1, 64)
    if shape != "ones":
        kw["chunks"] = _spread(rng, 1, 4)
        kw["rows"] = _spread(rng, 2, 2048 // kw["chunks"])
    kw["past_lo"] = _spread(rng, 1, 2000) - 1
    kw["past_hi"] = kw["past_lo"] + _spread(rng, 1, 6000) - 1
    if op == "attn" and shape == "ones":  # a few long contexts
        kw["ones"] = min(kw["ones"], 6)
        kw["past_hi"] = kw["past_lo"] + _spread(rng, 1, 60000) - 1
    if rope:
        kw["rot"] = rng.choice([d, d, d // 2, 16, 48])
        kw["interleaved"] = rng.random() < 0.3
        kw["theta"] = rng.choice([10000.0, 500000.0])
        kw["fused_qkv"] = rng.random() < 0.5
        kw["norm"] = rng.random() < 0.8
    return case_of("", op, dtype, hkv * group, hkv, d, **kw)


def layout(c):
    """Rows and cached lengths of the case's sequences, and a bound on their sum."""
    n = c["ones"] + c["chunks"]
    # Equal rows when every sequence has a chunk; beside one-row sequences the chunks get shorter one by one.
    rows = [1] * c["ones"] + [max(2, c["rows"] - 37 * i) if c["ones"] else c["rows"] for i in range(c["chunks"])]
    span = c["past_hi"] - c["past_lo"]
    past = [c["past_lo"] + (span * ((i * 37) % n)) // max(1, n - 1) for i in range(n)]
    return rows, past, max(r + p for r, p in zip(rows, past))


def work(c):
    rows, past, _ = layout(c)
    t, d, es = sum(rows), c["d"], 4 if c["dtype"] == "f32" else 2
    hq, hkv = c["hq"], c["hkv"]
    q4 = d // 2 + d // GROUP * 4  # bytes of a row held in 4 bits
    keys = sum(r + p for r, p in zip(rows, past))
    seen = sum(r * p + r * (r + 1) // 2 for r, p in zip(rows, past))
    norm = 2 * hkv * t * d  # 2 hkv rows of d channels for each token
    if c["op"] == "rope":
        return {"bytes": 2 * t * (hq + hkv) * d * es, "flops": 8 * t * (hq + hkv) * d}
    if c["op"] == "rope_append":
        return {"bytes": 2 * t * (hq + 2 * hkv) * d * es, "flops": 8 * t * (hq + hkv) * d}
    if c["op"] == "append":  # rows in, codes out and in again, values out
        return {"bytes": norm * es * 2 + 2 * 2 * hkv * t * q4, "flops": 8 * norm}
    attn = {"bytes": 2 * hkv * keys * q4 + 2 * t * hq * d * es, "flops": 4 * seen * hq * d}
    if c["op"] == "attn":
        return attn
    return {"bytes": attn["bytes"] + norm * es * 2 + 2 * hkv * t * q4, "flops": attn["flops"] + 8 * norm}


# ------------------------------------------------------------------ inputs

def quantized(x):
    """Rows of d channels -> (codes uint8 [..., d / 2], params [..., d / 32, 2]) of the 4-bit cache."""
    g = x.unflatten(-1, (-1, GROUP)).float()
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    step = ((hi - lo) / 15).to(x.dtype)
    above = step.float() > (hi - lo) / 15  # cut toward zero
    step = torch.where(above, (step.view(torch.int16) - 1).view(x.dtype), step)
    s = step.float()
    c = torch.where(s > 0, ((g - lo) / s).round().clamp(max=15), torch.zeros_like(g)).to(torch.int32)
    c = c.flatten(-2).unflatten(-1, (-1, 4, 2))  # [words, 4, 2]: channels 8w + 2i, 8w + 2i + 1
    at = 4 * torch.arange(4, device=x.device, dtype=torch.int32)
    half = (c << at[:, None]).sum(-2, dtype=torch.int32)  # [words, 2]: the two 16-bit halves
    b = torch.stack([half & 255, half >> 8], -1).flatten(-3).to(torch.uint8)
    return b, torch.cat([step, lo.to(x.dtype)], -1)


def values(codes, params):
    """What the cache's codes stand for, in the params' type."""
    b = codes.unflatten(-1, (-1, 2, 2)).int()
    half = b[..., 0] | (b[..., 1] << 8)  # [words, 2]
    at = 4 * torch.arange(4, device=codes.device, dtype=torch.int32)
    c = ((half[..., None, :] >> at[:, None]) & 15).flatten(-3).unflatten(-1, (-1, GROUP)).float()
    s, m = params[..., 0:1].float(), params[..., 1:2].float()
    return (m + c * s).to(params.dtype).flatten(-2)


class Inputs:
    """What a user's program has in hand before the call."""


def prepare(c, seed):
    dev, dt, d = "cuda", DTYPES[c["dtype"]], c["d"]
    hq, hkv = c["hq"], c["hkv"]
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    st = Inputs()
    st.case, st.dtype = c, dt
    st.rows, st.past, st.max_ctx = layout(c)
    n, t = len(st.rows), sum(st.rows)
    st.n, st.t = n, t
    starts = [sum(st.rows[:i]) for i in range(n + 1)]
    st.cu_rows = torch.tensor(starts, dtype=torch.int32, device=dev)
    st.uniform = len(set(st.rows)) == 1
    st.lens = torch.tensor(st.past, dtype=torch.int32, device=dev)
    st.seq = torch.repeat_interleave(torch.arange(n, device=dev), torch.tensor(st.rows, device=dev))
    st.at = torch.arange(t, device=dev) - st.cu_rows[st.seq].long()  # a row's place within its sequence
    rope = c["op"].startswith("rope")

    # Projections: queries, keys (some channels larger, as models have them) and values.
    wide = 1.0 + 3.0 * (torch.rand(hkv, d, generator=gen, device=dev) < 0.06)
    if c["fused_qkv"]:
        qkv = randn(t, (hq + 2 * hkv) * d).to(dt)
        st.q = qkv[:, :hq * d].unflatten(1, (hq, d))
        st.k = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        st.v = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        st.k.mul_(wide.to(dt))
    else:
        st.q = randn(t, hq, d).to(dt)
        st.k = (randn(t, hkv, d) * wide).to(dt)
        st.v = randn(t, hkv, d).to(dt)
    if rope:
        rot = c["rot"]
        st.inv_freq = (c["theta"] ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / max(rot, 1))).float()
        st.q_weight = (1 + 0.2 * randn(d)).to(dt) if c["norm"] else None
        st.k_weight = (1 + 0.2 * randn(d)).to(dt) if c["norm"] else None
        st.q_out = torch.zeros(t, hq, d, dtype=dt, device=dev)
        st.k_out = torch.zeros(t, hkv, d, dtype=dt, device=dev)

    # The cache: contiguous at a capacity with room to spare, or pages dealt at random.
    st.cap = -(-(st.max_ctx + 64) // 128) * 128
    st.table = None
    page = c["page"]
    if page:
        st.blocks = st.cap // page
        need = [-(-(r + p) // page) for r, p in zip(st.rows, st.past)]
        st.pages = sum(need)
        perm = torch.randperm(st.pages, generator=host).tolist()
        first = [sum(need[:i]) for i in range(n)]
        st.table = torch.tensor([perm[f:f + k] + [-1] * (st.blocks - k) for f, k in zip(first, need)], dtype=torch.int32, device=dev)
        planes = (st.pages, hkv, page)
    else:
        planes = (n, hkv, st.cap)
    if c["op"] == "rope_append":
        st.k_cache = torch.zeros(*planes, d, dtype=dt, device=dev)
        st.v_cache = torch.zeros(*planes, d, dtype=dt, device=dev)
    elif not rope:
        held = c["op"] != "append"  # an attention finds the earlier rows there
        k = randn(*planes, d).mul_(wide[:, None]).to(dt) if held else torch.zeros(*planes, d, dtype=dt, device=dev)
        st.k_codes, st.k_params = quantized(k)
        del k
        v = randn(*planes, d).to(dt) if held else torch.zeros(*planes, d, dtype=dt, device=dev)
        st.v_codes, st.v_params = quantized(v)
        del v
        if c["op"] == "attn":  # the call's own rows are in the cache already
            write_rows(st, *quantized(st.k), *quantized(st.v))
        st.out = torch.zeros(t, hq, d, dtype=dt, device=dev)
    if own:
        import chunked_prefill_causal_cp_gb300 as cp
        kind = dict(kind=cp.CP_CACHE_PAGED, page_size=page, num_pages=st.pages, max_blocks=st.blocks) if page else \
            dict(kind=cp.CP_CACHE_CONTIG, capacity=st.cap)
        st.desc = cp.layer_desc(dt, n, hq, hkv, d, **kind)
        st.call = dict(cu_rows=None if st.uniform else st.cu_rows)
        if rope:
            st.prep = cp.qk_prep(c["rot"], interleaved=c["interleaved"], eps=EPS)
        else:
            st.call["block_table"] = st.table
            st.cache = cp.q4_cache(st.k_codes, st.v_codes, st.k_params, st.v_params)
            st.ws = torch.empty(max(16, cp.cp_workspace_size_q4(st.desc, t, st.max_ctx, n)), dtype=torch.uint8, device=dev)
            st.k_back, st.v_back = torch.zeros_like(st.k), torch.zeros_like(st.v)
    return st


def slots(st):
    """Where each of the call's rows lives: two indexes of the cache's first and third dimension."""
    pos = st.lens[st.seq].long() + st.at
    if st.table is None:
        return st.seq, pos
    page = st.case["page"]
    return st.table[st.seq, pos // page].long(), pos % page


def write_rows(st, k_codes, k_params, v_codes, v_params):
    i, j = slots(st)
    st.k_codes[i, :, j], st.k_params[i, :, j] = k_codes, k_params
    st.v_codes[i, :, j], st.v_params[i, :, j] = v_codes, v_params


# ------------------------------------------------------------------ one pass

def rotated(x, w, pos, inv_freq, c):
    """Norm and rotation of [t, heads, d], in 32 bits (angles in 64), rounded once."""
    y = x.float()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
    u = pos.double()[:, None] * inv_freq.double()
    cos, sin = torch.cos(u).float()[:, None], torch.sin(u).float()[:, None]
    z, rot = y.clone(), c["rot"]
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = y[..., lo], y[..., hi]
    z[..., lo], z[..., hi] = a * cos - b * sin, b * cos + a * sin
    return z.to(x.dtype)


def attention(q, k, v, past, scale):
    """Rows [s, r, hq, d] at positions past[s] + i over keys [s, hkv, n, d], causal."""
    s, r, hq, d = q.shape
    hkv, n = k.shape[1], k.shape[2]
    q = (q.float() * scale).unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [s, hkv, g r, d]
    p = torch.matmul(q, k.float().transpose(2, 3))
    last = past[:, None] + torch.arange(r, device=q.device)  # [s, r]: the last key a row sees
    hide = (torch.arange(n, device=q.device) > last[..., None]).repeat(1, hq // hkv, 1)[:, None]
    p.masked_fill_(hide, -math.inf)
    p -= p.amax(-1, keepdim=True)
    p.exp_()
    norm = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.float()) / norm
    return o.unflatten(2, (hq // hkv, r)).permute(0, 3, 1, 2, 4).flatten(2, 3)


def gathered(st, first, count, x):
    """The first max_ctx positions of sequences first .. first + count - 1 of a cache array: [s, hkv, n, ...]."""
    if st.table is None:
        return x[first:first + count, :, :st.max_ctx]
    b = -(-st.max_ctx // st.case["page"])
    y = x[st.table[first:first + count, :b].long().clamp(min=0)]  # [s, b, hkv, page, ...]
    return y.transpose(1, 2).flatten(2, 3)[:, :, :st.max_ctx]


def attended(st, first, count, r):
    """Attention of sequences that all have up to r rows; rows past a sequence's own are dropped."""
    at = st.cu_rows[first:first + count].long()[:, None] + torch.arange(r, device=st.q.device)
    real = torch.arange(r, device=st.q.device) < torch.tensor(st.rows[first:first + count], device=st.q.device)[:, None]
    k = values(gathered(st, first, count, st.k_codes), gathered(st, first, count, st.k_params))
    v = values(gathered(st, first, count, st.v_codes), gathered(st, first, count, st.v_params))
    held = (st.lens + (st.cu_rows[1:] - st.cu_rows[:-1]))[first:first + count, None, None, None]
    gone = torch.arange(st.max_ctx, device=st.q.device)[:, None] >= held
    k, v = k.masked_fill(gone, 0), v.masked_fill(gone, 0)
    o = attention(st.q[at.clamp(max=st.t - 1)], k, v, st.lens[first:first + count].long(), 1 / math.sqrt(st.case["d"]))
    return o[real].to(st.dtype)


def attended_all(st):
    ones, n = st.case["ones"], st.n
    parts = [attended(st, 0, ones, 1)] if ones else []
    parts += [attended(st, ones, n - ones, max(st.rows))] if n > ones else []
    return torch.cat(parts)


def run(st):
    c, op = st.case, st.case["op"]
    if own:
        import chunked_prefill_causal_cp_gb300 as cp
        if op == "rope":
            cp.cp_qk_norm_rope(st.desc, st.prep, st.q, st.k, st.q_out, st.k_out, st.n, st.t, q_weight=st.q_weight,
                               k_weight=st.k_weight, inv_freq=st.inv_freq, seqlens_k=st.lens, **st.call)
            return st.q_out, st.k_out
        if op == "rope_append":
            cp.cp_qk_norm_rope_append(st.desc, st.prep, st.q, st.k, st.v, st.q_out, st.k_cache, st.v_cache, st.lens, st.n,
                                      st.t, st.max_ctx, q_weight=st.q_weight, k_weight=st.k_weight,
                                      inv_freq=st.inv_freq, block_table=st.table, **st.call)
            return st.q_out, st.k_cache, st.v_cache
        if op == "append":
            cp.cp_kv_append_q4(st.desc, st.k, st.v, st.cache, st.lens, st.n, st.t, st.max_ctx, **st.call)
        if op == "attn":
            cp.cp_chunk_attn_q4(st.desc, st.q, st.cache, st.lens, st.n, st.t, st.max_ctx, st.out, st.ws, commit=False, **st.call)
            return st.out
        if op == "step":
            cp.cp_mixed_step_q4(st.desc, st.q, st.k, st.v, st.cache, st.lens, st.n, st.t, st.max_ctx, st.out, st.ws,
                                commit=False, **st.call)
        # The values that the rows now stand for.
        cp.cp_kv_read_q4(st.desc, st.cache, st.lens, st.n, st.t, st.max_ctx, st.k_back, st.v_back, **st.call)
        back = st.k_back, st.v_back
        return back if op == "append" else (st.out, *back)

    if op.startswith("rope"):
        pos = st.lens[st.seq].long() + st.at
        q, k = rotated(st.q, st.q_weight, pos, st.inv_freq, c), rotated(st.k, st.k_weight, pos, st.inv_freq, c)
        if op == "rope":
            return q, k
        i, j = slots(st)
        st.k_cache[i, :, j], st.v_cache[i, :, j] = k, st.v
        return q, st.k_cache, st.v_cache
    if op != "attn":
        write_rows(st, *quantized(st.k), *quantized(st.v))
        i, j = slots(st)
        back = values(st.k_codes[i, :, j], st.k_params[i, :, j]), values(st.v_codes[i, :, j], st.v_params[i, :, j])
        if op == "append":
            return back
    out = attended_all(st)
    return out if op == "attn" else (out, *back)


# ------------------------------------------------------------------ in 64 bits

def exact(c, seed):
    """The definition, in 64 bits, sequence by sequence."""
    st = prepare(c, seed)
    f64, d, dt = torch.float64, c["d"], DTYPES[c["dtype"]]
    bounds = st.cu_rows.tolist()
    seqs = [(s, bounds[s], bounds[s + 1], int(st.lens[s])) for s in range(len(bounds) - 1)]

    def place(s, p):  # of position p of sequence s
        if not c["page"]:
            return s, p
        return int(st.table[s, p // c["page"]]), p % c["page"]

    if c["op"].startswith("rope"):
        def turn(x, w):
            y = x.to(f64)
            if w is not None:
                y = y * (y.pow(2).sum(-1, keepdim=True) / d + EPS).rsqrt() * w.to(f64)
            z = y.clone()
            for s, r0, r1, past in seqs:
                angle = torch.outer(torch.arange(past, past + r1 - r0, device=x.device, dtype=f64), st.inv_freq.to(f64))
                for i in range(c["rot"] // 2):
                    a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + c["rot"] // 2)
                    co, si = angle[:, i, None].cos(), angle[:, i, None].sin()
                    z[r0:r1, :, a] = y[r0:r1, :, a] * co - y[r0:r1, :, b] * si
                    z[r0:r1, :, b] = y[r0:r1, :, a] * si + y[r0:r1, :, b] * co
            return z

        q, k = turn(st.q, st.q_weight), turn(st.k, st.k_weight)
        if c["op"] == "rope":
            return q, k
        kc, vc = st.k_cache.to(f64), st.v_cache.to(f64)
        for s, r0, r1, past in seqs:
            for t in range(r0, r1):
                i, j = place(s, past + t - r0)
                kc[i, :, j], vc[i, :, j] = k[t], st.v[t].to(f64)
        return q, kc, vc

    def stands_for(x):  # of rows put into the cache
        g = x.to(f64).reshape(*x.shape[:-1], d // GROUP, GROUP)
        lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
        step = ((hi - lo) / 15).to(dt)
        bits = step.view(torch.int16)
        step = torch.where(step.to(f64) * 15 > hi - lo, (bits - 1).view(dt), step).to(f64)
        code = torch.where(step > 0, torch.round((g - lo) / step).clamp(0, 15), 0.0)
        return (lo + code * step).to(dt).to(f64).reshape(x.shape)

    def held(codes, params):  # [.., n, d] that a cache array stands for
        words = codes.contiguous().view(torch.int32)
        parts = [(words >> (4 * i + 16 * e)) & 15 for i in range(4) for e in range(2)]
        code = torch.stack(parts, -1).to(f64).reshape(*words.shape[:-1], d // GROUP, GROUP)
        p = params.to(f64)
        return (p[..., 1:2] + code * p[..., 0:1]).to(dt).to(f64).reshape(*words.shape[:-1], d)

    own_k, own_v = stands_for(st.k), stands_for(st.v)
    if c["op"] == "append":
        return own_k, own_v
    out = torch.empty(st.t, c["hq"], d, dtype=f64, device=st.q.device)
    for s, r0, r1, past in seqs:
        n = past + r1 - r0
        if c["page"]:
            b = st.table[s, :-(-n // c["page"])].long()
            flat = lambda x: x[b].transpose(0, 1).flatten(1, 2)[:, :n]  # noqa: E731
        else:
            flat = lambda x: x[s, :, :n]  # noqa: E731
        k, v = held(flat(st.k_codes), flat(st.k_params)), held(flat(st.v_codes), flat(st.v_params))
        if c["op"] == "step":
            k[:, past:], v[:, past:] = own_k[r0:r1].transpose(0, 1), own_v[r0:r1].transpose(0, 1)
        hide = torch.arange(n, device=k.device) > torch.arange(past, n, device=k.device)[:, None]
        for h in range(c["hq"]):
            g = h // (c["hq"] // c["hkv"])
            score = (st.q[r0:r1, h].to(f64) @ k[g].T / math.sqrt(d)).masked_fill_(hide, -math.inf)
            out[r0:r1, h] = torch.softmax(score, -1) @ v[g]
    return out if c["op"] == "attn" else (out, own_k, own_v)
