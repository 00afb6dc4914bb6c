"""GPU parity of the cache held in 4 bits: its stored bits against the fp32
restatement, what reads back, and attention over it against 64 bits."""
import numpy as np
import pytest
import torch

import chunked_prefill_causal_cp_gb300 as cp
from oracle import q4
from q4_util import Cache4, check_attention, f64

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from chunked_prefill_causal_cp_gb300 import _build
    _build.build()


def _ints(xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


def _cu(rows):
    return _ints([0, *np.cumsum(rows).tolist()])


def _awkward(dtype, t, hkv, d, seed):
    """Rows with groups that are flat, tiny, huge, of one sign, and not finite."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, hkv, d, generator=g)
    x[0] = 3.25
    x[1] = 0.0
    x[2] *= 1e-7 if dtype == F16 else 1e-39
    x[3] *= 9000.0 if dtype == F16 else 1e38
    x[4] = x[4].abs() + 2
    x[5] = -x[5].abs()
    x[6, :, 0] = 60000.0
    x[7, :, 5], x[7, :, 40] = float("nan"), float("inf")
    if dtype == F16:
        x[8, :, 0], x[8, :, 1] = 65504.0, -65504.0
    else:
        x[8, :, 0], x[8, :, 1] = 3e38, -3e38  # the range overflows fp32
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d,page", [(128, 0), (64, 16), (128, 64)])
def test_stored_bits_and_values_read_back(dtype, d, page):
    rows, past = [1, 200, 13, 64], [130, 0, 5, 64]
    t, hkv = sum(rows), 3
    c = Cache4(dtype, hkv, hkv, d, 4, 256, page)
    k, v = _awkward(dtype, t, hkv, d, 1).cuda(), _awkward(dtype, t, hkv, d, 2).cuda()
    cp.cp_kv_append_q4(c.desc, k, v, c.arg, _ints(past), 4, t, 256, cu_rows=_cu(rows), block_table=c.table,
                       dev_status=c.status)
    assert int(c.status) == 0
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    cp.cp_kv_read_q4(c.desc, c.arg, _ints(past), 4, t, 256, ko, vo, cu_rows=_cu(rows), block_table=c.table,
                     dev_status=c.status)
    assert int(c.status) == 0
    r0 = 0
    for s, (r, p) in enumerate(zip(rows, past)):
        for new, (codes, scale, lo), back in zip((k, v), c.rows(s, p + r), (ko, vo)):
            x = new[r0:r0 + r].float().cpu().numpy()
            wc, ws, wl = q4.store(x, dtype == BF16)
            fine = np.isfinite(ws)
            assert np.array_equal(np.isfinite(scale[p:]), fine)
            assert np.array_equal(scale[p:][fine], ws[fine]) and np.array_equal(lo[p:][fine], wl[fine])
            assert np.array_equal(codes[p:], wc)
            assert np.isnan(scale[:p]).all() and (codes[:p] == 15).all()  # unwritten slots as they were
            with np.errstate(invalid="ignore"):
                want = torch.from_numpy(q4.values(wc, ws, wl)).to(dtype)
            got = back[r0:r0 + r].cpu()
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            assert torch.equal(torch.nan_to_num(got.float()), torch.nan_to_num(want.float()))
            # No further from what was put in than half a step of the group (the cut scale: the top code 15/128 more).
            with np.errstate(invalid="ignore"):
                off = np.abs(f64(got) - x).reshape(r, hkv, -1, 32).max(-1)
                near = np.abs(x).reshape(r, hkv, -1, 32).max(-1) * torch.finfo(dtype).eps + 15 * 2.0 ** -24
                assert (off <= 0.62 * ws + near)[fine].all()
        r0 += r


def test_append_out_of_bounds_is_reported_and_skipped():
    c = Cache4(BF16, 2, 2, 64, 3, 32, page=16)
    c.table[0, 1] = 1000
    x = torch.randn(3 * 4, 2, 64, device="cuda").bfloat16()
    before = [y.clone() for y in (c.kc, c.vc)]
    cp.cp_kv_append_q4(c.desc, x, x, c.arg, _ints([14, 30, -3]), 3, 12, 32, block_table=c.table, dev_status=c.status)
    assert int(c.status) == cp.CP_DEV_BOUNDS
    ok = [(0, 14), (0, 15), (1, 30), (1, 31), (2, 0)]
    changed = (c.vc != before[1]).any(-1).any(1).nonzero().tolist()
    assert sorted(changed) == sorted([list(c.slot(s, p)) for s, p in ok])
    c.status.zero_()
    out = torch.full((12, 2, 64), 7.0, dtype=BF16, device="cuda")
    cp.cp_kv_read_q4(c.desc, c.arg, _ints([14, 30, -3]), 3, 12, 32, out, None, block_table=c.table, dev_status=c.status)
    assert int(c.status) == cp.CP_DEV_BOUNDS
    same = (out == 7.0).all(-1).all(-1).cpu().tolist()
    assert same == [False, False, True, True, False, False, True, True, True, True, True, False]


def _attend(c, rows, past, uniform=False, commit=False, seed=3, dtype=None):
    t = sum(rows)
    q = torch.randn(t, c.hq, c.d, generator=torch.Generator().manual_seed(seed)).to(c.dtype).cuda()
    out = torch.full_like(q, float("nan"))
    mc = max(p + r for p, r in zip(past, rows))
    lens = _ints(past)
    cp.cp_chunk_attn_q4(c.desc, q, c.arg, lens, len(rows), t, mc, out, c.workspace(t, mc), commit=commit,
                        cu_rows=None if uniform else _cu(rows), block_table=c.table, dev_status=c.status)
    assert int(c.status) == 0
    assert lens.tolist() == [p + (r if commit else 0) for p, r in zip(past, rows)]
    return q, out


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (16, 2), (16, 1)])
@pytest.mark.parametrize("page", [0, 32])
def test_single_rows(dtype, d, hq, hkv, page):
    """Decode rows: one key, and lengths at the edges of tiles, pages, warps and splits."""
    past = [0, 1, 15, 16, 63, 127, 128, 500, 511, 512, 513, 1023, 1024, 1530]
    c = Cache4(dtype, hq, hkv, d, len(past), 1600, page)
    c.fill([p + 1 for p in past])
    q, out = _attend(c, [1] * len(past), past, uniform=True)
    check_attention(c, q, out, past, [1] * len(past))


@pytest.mark.parametrize("rows,hq,hkv,dtype,page", [(2, 8, 2, BF16, 0), (4, 8, 2, F16, 16), (5, 2, 2, BF16, 64),
                                                    (16, 3, 3, F16, 0), (8, 4, 2, BF16, 128), (2, 16, 2, BF16, 32)])
def test_short_chunks(rows, hq, hkv, dtype, page):
    past = [0, 3, 120, 505, 511, 1019, 1024]
    for d in (64, 128):
        c = Cache4(dtype, hq, hkv, d, len(past), 1200, page)
        c.fill([p + rows for p in past])
        q, out = _attend(c, [rows] * len(past), past, uniform=True, commit=True)
        check_attention(c, q, out, past, [rows] * len(past))


@pytest.mark.parametrize("rows,past,hq,hkv,d,dtype,page", [
    ([17], [0], 4, 4, 64, BF16, 0),
    ([129], [127], 8, 2, 128, BF16, 0),
    ([300, 300], [0, 513], 4, 2, 128, F16, 16),
    ([65, 65, 65], [1000, 64, 1], 16, 1, 64, F16, 64),
    ([256], [256], 8, 1, 128, BF16, 128),
    ([511], [130], 4, 1, 128, F16, 32),
    ([1000], [1], 2, 1, 64, BF16, 0),
])
def test_chunks(rows, past, hq, hkv, d, dtype, page):
    c = Cache4(dtype, hq, hkv, d, len(rows), 1700, page)
    c.fill([p + r for p, r in zip(past, rows)])
    q, out = _attend(c, rows, past, uniform=True)
    check_attention(c, q, out, past, rows)


@pytest.mark.parametrize("dtype,d,hq,hkv,page", [(BF16, 128, 8, 2, 16), (F16, 64, 6, 6, 0), (BF16, 64, 16, 1, 128)])
def test_ragged_rows(dtype, d, hq, hkv, page):
    rows, past = [1, 40, 1, 2, 333, 1, 128], [700, 0, 0, 77, 129, 1024, 500]
    c = Cache4(dtype, hq, hkv, d, len(rows), 1100, page)
    c.fill([p + r for p, r in zip(past, rows)])
    q, out = _attend(c, rows, past, commit=True)
    check_attention(c, q, out, past, rows)


def test_scale_and_large_scores():
    """A given scale, and keys so large that one key takes each row."""
    c = Cache4(BF16, 4, 1, 128, 2, 400, scale=0.5)
    c.fill([400, 300], k_scale=8.0)
    q, out = _attend(c, [100, 100], [300, 200], uniform=True)
    check_attention(c, q, out, [300, 200], [100, 100])


def test_sequence_out_of_bounds_is_reported_and_left_alone():
    for r in (1, 40):
        c = Cache4(BF16, 4, 2, 64, 3, 128)
        c.fill([128] * 3)
        q = torch.randn(3 * r, 4, 64, device="cuda").bfloat16()
        out = torch.full_like(q, 5.0)
        cp.cp_chunk_attn_q4(c.desc, q, c.arg, _ints([20, 129 - r, -1]), 3, 3 * r, 128, out, c.workspace(3 * r, 128),
                            commit=False, dev_status=c.status)
        assert int(c.status) == cp.CP_DEV_BOUNDS
        assert (out[r:] == 5.0).all()
        check_attention(c, q[:r], out[:r], [20], [r])


def test_a_bad_page_is_reported_and_not_read():
    for r in (1, 40):
        c = Cache4(BF16, 4, 2, 64, 2, 128, page=16)
        c.fill([128] * 2)
        c.table[0, 2] = 10 ** 6
        q = torch.randn(2 * r, 4, 64, device="cuda").bfloat16()
        out = torch.empty_like(q)
        cp.cp_chunk_attn_q4(c.desc, q, c.arg, _ints([80, 60]), 2, 2 * r, 128, out, c.workspace(2 * r, 128),
                            commit=False, block_table=c.table, dev_status=c.status)
        assert int(c.status) == cp.CP_DEV_BOUNDS
        check_attention(c, q[r:], out[r:], [60], [r], seqs=[1])


def test_a_step_is_append_then_attention_in_fewer_calls():
    rows, past = [1, 1, 50, 1, 260], [100, 511, 30, 0, 200]
    t = sum(rows)
    g = torch.Generator().manual_seed(8)
    q, k, v = (torch.randn(t, h, 128, generator=g).bfloat16().cuda() for h in (8, 2, 2))
    outs, caches = [], []
    for fused in (False, True):
        c = Cache4(BF16, 8, 2, 128, 5, 520, page=16)
        c.fill(past)
        out, lens, ws = torch.empty_like(q), _ints(past), c.workspace(t, 512)
        kw = dict(cu_rows=_cu(rows), block_table=c.table, dev_status=c.status)
        if fused:
            cp.cp_mixed_step_q4(c.desc, q, k, v, c.arg, lens, 5, t, 512, out, ws, **kw)
        else:
            cp.cp_kv_append_q4(c.desc, k, v, c.arg, lens, 5, t, 512, **kw)
            cp.cp_chunk_attn_q4(c.desc, q, c.arg, lens, 5, t, 512, out, ws, **kw)
        assert int(c.status) == 0 and lens.tolist() == [p + r for p, r in zip(past, rows)]
        outs.append(out)
        caches.append(c)
    assert torch.equal(outs[0], outs[1])
    for a, b in zip(caches[0].arg.tensors, caches[1].arg.tensors):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    check_attention(caches[1], q, outs[1], past, rows)


def test_a_row_depends_on_its_own_sequence_only():
    rows, past = [1, 64, 1, 200], [900, 100, 33, 515]
    c = Cache4(BF16, 8, 2, 128, 4, 1000)
    c.fill([p + r for p, r in zip(past, rows)])
    q, out = _attend(c, rows, past)
    for i in range(4):
        r0 = sum(rows[:i])
        cache, desc, _ = c.view(i)
        o = torch.empty_like(q[r0:r0 + rows[i]])
        cp.cp_chunk_attn_q4(desc, q[r0:r0 + rows[i]], cache, _ints([past[i]]), 1, rows[i], 1000, o,
                            c.workspace(rows[i], 1000, 1), cu_rows=_cu([rows[i]]), commit=False)
        assert torch.equal(o, out[r0:r0 + rows[i]])


@pytest.mark.parametrize("dtype,hq,d", [(BF16, 8, 128), (F16, 4, 64)])
@pytest.mark.parametrize("rows,past", [(1, 300), (2, 127), (4, 510), (40, 100), (200, 77), (300, 0)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_non_finite_key_reaches_the_rows_that_see_it_only(dtype, hq, d, rows, past, value):
    hkv, at = hq // 2, past + rows // 2  # the key of a row in the middle of the call's
    n = past + rows
    outs = []
    for which in (None, "v", "k"):
        c = Cache4(dtype, hq, hkv, d, 1, 700)
        g = torch.Generator().manual_seed(7)
        k, v = (torch.randn(n, hkv, d, generator=g).to(dtype).cuda() for _ in range(2))
        if which:
            {"k": k, "v": v}[which][at, :, 3] = value
        cp.cp_kv_append_q4(c.desc, k, v, c.arg, _ints([0]), 1, n, n)
        outs.append(_attend(c, [rows], [past], uniform=True)[1])
    seen = at - past
    for out in outs[1:]:
        assert torch.equal(out[:seen], outs[0][:seen])
        assert (~torch.isfinite(out[seen:]).all(-1)).all()


def test_slots_past_four_billion_bytes():
    """The last sequence's codes start more than 2^32 bytes into the cache."""
    hq, hkv, d, n, cap = 8, 8, 128, 3, 2_900_001
    lead = (n, hkv, cap)
    kc, vc = (torch.empty(*lead, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    kp, vp = (torch.empty(*lead, d // 32, 2, dtype=BF16, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 32
    desc = cp.layer_desc(BF16, n, hq, hkv, d, capacity=cap)
    cache = cp.q4_cache(kc, vc, kp, vp)
    rows, past, small = [1, 40, 33], [0, 0, 0], Cache4(BF16, hq, hkv, d, n, 64)
    for r in (rows, [1, 1, 60]):
        t = sum(r)
        g = torch.Generator().manual_seed(t)
        q, k, v = (torch.randn(t, hkv, d, generator=g).bfloat16().cuda() for _ in range(3))
        outs = []
        for dsc, c, mc in ((desc, cache, cap), (small.desc, small.arg, 64)):
            out, lens, st = torch.empty_like(q), _ints(past), torch.zeros(1, dtype=torch.int32, device="cuda")
            ws = torch.empty(cp.cp_workspace_size_q4(dsc, t, mc, n), dtype=torch.uint8, device="cuda")
            cp.cp_mixed_step_q4(dsc, q, k, v, c, lens, n, t, mc, out, ws, cu_rows=_cu(r), dev_status=st)
            assert int(st) == 0 and lens.tolist() == r
            outs.append(out)
        assert torch.equal(outs[0], outs[1])
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        cp.cp_kv_read_q4(desc, cache, _ints(past), n, t, cap, ko, vo, cu_rows=_cu(r))
        k2, v2 = torch.empty_like(k), torch.empty_like(v)
        cp.cp_kv_read_q4(small.desc, small.arg, _ints(past), n, t, 64, k2, v2, cu_rows=_cu(r))
        assert torch.equal(ko, k2) and torch.equal(vo, v2)


def _step_buffers(rows, past, seed):
    c = Cache4(BF16, 8, 2, 128, len(rows), 700, page=32, seed=seed)
    c.fill(past, seed=seed)
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(sum(rows), h, 128, generator=g).bfloat16().cuda() for h in (8, 2, 2))
    return c, q, k, v


def test_captured_and_replayed_and_on_another_stream():
    """A step captured on a side stream, replayed on new inputs, equals the same steps made one by one."""
    rows, past = [1, 30, 1, 290], [512, 0, 77, 300]
    t, n = sum(rows), len(rows)
    c, q, k, v = _step_buffers(rows, past, 1)
    e, _, _, _ = _step_buffers(rows, past, 1)
    out, ref, lens, cu = torch.empty_like(q), torch.empty_like(q), _ints(past), _cu(rows)
    ws, ws2 = c.workspace(t, 600), c.workspace(t, 600)
    kw = dict(cu_rows=cu, commit=False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cp.cp_mixed_step_q4(c.desc, q, k, v, c.arg, lens, n, t, 600, out, ws, block_table=c.table, **kw)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cp.cp_mixed_step_q4(c.desc, q, k, v, c.arg, lens, n, t, 600, out, ws, block_table=c.table, **kw)
    for seed in (5, 6):
        g = torch.Generator().manual_seed(seed)
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        out.fill_(float("nan"))
        ws.fill_(255)
        graph.replay()
        cp.cp_mixed_step_q4(e.desc, q, k, v, e.arg, lens, n, t, 600, ref, ws2, block_table=e.table, **kw)
        assert torch.equal(out, ref)
        assert torch.equal(c.kc, e.kc) and torch.equal(c.vc, e.vc)
    check_attention(c, q, out, past, rows)


def test_two_calls_at_once_on_two_streams():
    rows, past = [1, 1, 200], [600, 44, 333]
    t, n = sum(rows), len(rows)
    sets = [_step_buffers(rows, past, s) for s in (3, 4)]
    outs, wss = [torch.empty_like(s[1]) for s in sets], [s[0].workspace(t, 640) for s in sets]
    lens, cu = [_ints(past), _ints(past)], _cu(rows)
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        for i, (c, q, k, v) in enumerate(sets):
            cp.cp_mixed_step_q4(c.desc, q, k, v, c.arg, lens[i], n, t, 640, outs[i], wss[i], cu_rows=cu,
                                block_table=c.table, commit=False, stream=streams[i])
    torch.cuda.synchronize()
    for (c, q, _, _), out in zip(sets, outs):
        check_attention(c, q, out, past, rows)


def test_rows_without_a_sequence_and_a_sequence_without_rows():
    """A listed sequence with no rows is reported; rows past the last sequence's stay as they were."""
    c = Cache4(BF16, 4, 2, 64, 3, 64)
    c.fill([40, 40, 40])
    q = torch.randn(45, 4, 64, device="cuda").bfloat16()
    out = torch.full_like(q, 3.0)
    cp.cp_chunk_attn_q4(c.desc, q, c.arg, _ints([10, 10, 10]), 3, 45, 64, out, c.workspace(45, 64), commit=False,
                        cu_rows=_ints([0, 20, 20, 41]), dev_status=c.status)
    assert int(c.status) == cp.CP_DEV_BOUNDS
    assert (out[41:] == 3.0).all()
    check_attention(c, q[:20], out[:20], [10], [20], seqs=[0])
    check_attention(c, q[20:41], out[20:41], [10], [21], seqs=[2])


def test_a_padded_batch():
    """total_rows past the last sequence's: the rows there go nowhere, in every call."""
    rows, past, t = [1, 30, 2], [40, 0, 17], 64
    n, cu, lens = sum(rows), _cu(rows), _ints(past)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(t, 8 * 64, generator=g).bfloat16().cuda()
    q, k, v = (y.unflatten(1, (-1, 64)) for y in x.split([4 * 64, 2 * 64, 2 * 64], 1))
    freq = torch.ones(32, device="cuda")
    c, e = (Cache4(BF16, 4, 2, 64, 3, 64, page=16) for _ in range(2))
    for y in (c, e):
        y.fill([p + 1 for p in past])
    got = []
    for cache, m in ((c, t), (e, n)):
        q2, k2 = torch.full((t, 4, 64), 3.0).bfloat16().cuda(), torch.full((t, 2, 64), 3.0).bfloat16().cuda()
        out, back = torch.full_like(q2, 3.0), torch.full_like(k2, 3.0)
        kw = dict(cu_rows=cu)
        cp.cp_qk_norm_rope(cache.desc, cp.qk_prep(64), q[:m], k[:m], q2, k2, 3, m, inv_freq=freq, seqlens_k=lens, **kw)
        kw.update(block_table=cache.table, dev_status=cache.status)
        cp.cp_mixed_step_q4(cache.desc, q2[:m], k2[:m], v[:m].contiguous(), cache.arg, lens, 3, m, 64, out,
                            cache.workspace(m, 64), commit=False, **kw)
        cp.cp_kv_read_q4(cache.desc, cache.arg, lens, 3, m, 64, None, back, **kw)
        qa, kc = torch.full_like(q2, 3.0), torch.full((cache.pages, 2, 16, 64), 3.0).bfloat16().cuda()
        vc = torch.full_like(kc, 3.0)
        cp.cp_qk_norm_rope_append(cache.desc, cp.qk_prep(64), q[:m], k[:m], v[:m], qa, kc, vc, lens, 3, m, 64,
                                  inv_freq=freq, **kw)
        assert int(cache.status) == 0
        got.append([q2, k2, out, back, qa, kc, vc, *(y.view(torch.uint8) for y in cache.arg.tensors)])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    for y in got[0][:5]:
        assert (y[n:] == 3.0).all()


def test_binding_refuses_wrong_tensors():
    c = Cache4(BF16, 4, 2, 64, 2, 64)
    c.fill([64, 64])
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    out, lens, ws = torch.empty_like(q), _ints([5, 5]), c.workspace(2, 64)
    good = dict(q=q, cache=c.arg, lens=lens, out=out, ws=ws, desc=c.desc)

    def call(**kw):
        a = {**good, **kw}
        cp.cp_chunk_attn_q4(a["desc"], a["q"], a["cache"], a["lens"], 2, 2, 64, a["out"], a["ws"], commit=False)

    call()
    bigger = cp.layer_desc(BF16, 3, 4, 2, 64, capacity=64)
    halves = torch.empty(2, 4, 128, device="cuda").bfloat16()[..., :64]
    for kw in (dict(q=q.half()), dict(q=q.cpu()), dict(q=q[:1]), dict(q=halves), dict(out=halves), dict(lens=lens.long()),
               dict(lens=lens[:1]), dict(ws=ws[:16]), dict(desc=bigger),
               dict(desc=cp.layer_desc(F16, 2, 4, 2, 64, capacity=64))):
        with pytest.raises(cp.CPError):
            call(**kw)
    x = torch.randn(4, 4, 64, device="cuda").bfloat16()
    kv = torch.randn(4, 2, 64, device="cuda").bfloat16()
    for bad in (x[:1].expand(4, 4, 64), x.transpose(0, 1), x[::2], x[..., :32]):
        with pytest.raises(cp.CPError):
            cp.cp_qk_norm_rope(c.desc, cp.qk_prep(0), bad, kv, torch.empty_like(x), torch.empty_like(kv), 1, 4, seqlens_k=lens)


def test_prompt_then_decode_with_norm_and_rotation():
    """The operators as they are used together: chunks of two prompts and then decode rows; every step norms and
    rotates its queries and keys, then appends and attends."""
    hq, hkv, d, n = 8, 2, 128, 2
    lens_total = [230, 150]
    g = torch.Generator().manual_seed(12)
    xs = [torch.randn(m, (hq + 2 * hkv) * d, generator=g).bfloat16().cuda() for m in lens_total]
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in range(2))
    freq = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
    c = Cache4(BF16, hq, hkv, d, n, 256, page=16)
    prep = cp.qk_prep(d)
    lens = _ints([0] * n)
    done, got = [0, 0], [[], []]
    plan = [[100, 60], [100, 60], [27, 27]] + [[1, 1]] * 3
    for rows in plan:
        t = sum(rows)
        x = torch.cat([xs[i][done[i]:done[i] + rows[i]] for i in range(n)])
        q, k, v = (y.unflatten(1, (-1, d)) for y in x.split([hq * d, hkv * d, hkv * d], 1))
        q2, k2 = torch.empty(t, hq, d, dtype=BF16, device="cuda"), torch.empty(t, hkv, d, dtype=BF16, device="cuda")
        out, cu = torch.empty_like(q2), _cu(rows)
        cp.cp_qk_norm_rope(c.desc, prep, q, k, q2, k2, n, t, q_weight=wq, k_weight=wk, inv_freq=freq, seqlens_k=lens,
                           cu_rows=cu)
        cp.cp_mixed_step_q4(c.desc, q2, k2, v.contiguous(), c.arg, lens, n, t, 256, out, c.workspace(t, 256), cu_rows=cu,
                            block_table=c.table, dev_status=c.status)
        r0 = 0
        for i in range(n):
            got[i].append((done[i], q2[r0:r0 + rows[i]], out[r0:r0 + rows[i]]))
            done[i] += rows[i]
            r0 += rows[i]
    assert int(c.status) == 0 and lens.tolist() == done == lens_total
    for i in range(n):
        for past, q, out in got[i]:
            check_attention(c, q, out, [past], [q.shape[0]], seqs=[i])
        # The keys in the cache are the normed and rotated ones: within half a step of 16 per group.
        x = xs[i][:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        want, _ = q4.norm_rope(f64(x), f64(wk), np.arange(lens_total[i]), f64(freq), d, False, 1e-6)
        k, _ = c.values(i, lens_total[i])
        span = np.ptp(want.reshape(-1, hkv, d // 32, 32), axis=-1)
        off = np.abs(k - want).reshape(-1, hkv, d // 32, 32).max(-1)
        assert (off <= 0.62 * span / 15 + 2.0 ** -7 * np.abs(want).max()).all()


@pytest.mark.parametrize("rows", [[0, 2], [2, 0], [1, 0, 2], [0, 0, 3, 1], [0, 0, 0, 2, 1, 0, 0], [1, 1, 1]])
@pytest.mark.parametrize("hq,hkv,d,dtype,page", [(8, 2, 128, BF16, 16), (4, 4, 64, F16, 0)])
def test_fewer_rows_than_sequences(rows, hq, hkv, d, dtype, page):
    """Listed sequences without rows are reported; every row of the others is computed, however few there are."""
    n, t = len(rows), sum(rows)
    past = [300, 40, 600, 17, 513, 5, 250][:n]
    g = torch.Generator().manual_seed(t)
    q, k, v = (torch.randn(t, h, d, generator=g).to(dtype).cuda() for h in (hq, hkv, hkv))
    outs = []
    for step in (False, True):
        c = Cache4(dtype, hq, hkv, d, n, 640, page)
        c.fill(past)
        out, lens, ws = torch.full_like(q, float("nan")), _ints(past), c.workspace(t, 640)
        kw = dict(cu_rows=_cu(rows), block_table=c.table, dev_status=c.status)
        if step:
            cp.cp_mixed_step_q4(c.desc, q, k, v, c.arg, lens, n, t, 640, out, ws, **kw)
        else:
            cp.cp_kv_append_q4(c.desc, k, v, c.arg, lens, n, t, 640, **kw)
            cp.cp_chunk_attn_q4(c.desc, q, c.arg, lens, n, t, 640, out, ws, **kw)
        assert int(c.status) == (cp.CP_DEV_BOUNDS if 0 in rows else 0)
        assert lens.tolist() == [p + r for p, r in zip(past, rows)]
        keep = [i for i in range(n) if rows[i]]
        check_attention(c, q, out, [past[i] for i in keep], [rows[i] for i in keep], seqs=keep)
        outs.append(out)
    assert torch.equal(*outs)


def test_fewer_rows_than_sequences_out_of_bounds():
    """A sequence whose rows do not all fit is left alone as a whole, its first row too."""
    c = Cache4(BF16, 4, 2, 64, 4, 128)
    c.fill([128] * 4)
    q = torch.randn(4, 4, 64, device="cuda").bfloat16()
    out = torch.full_like(q, 5.0)
    cp.cp_chunk_attn_q4(c.desc, q, c.arg, _ints([10, 127, 10, 30]), 4, 4, 128, out, c.workspace(4, 128), commit=False,
                        cu_rows=_ints([0, 0, 2, 2, 4]), dev_status=c.status)
    assert int(c.status) == cp.CP_DEV_BOUNDS
    assert (out[:2] == 5.0).all()
    check_attention(c, q[2:], out[2:], [30], [2], seqs=[3])
