"""GPU parity of the query/key norm and rotary position against the 64-bit
restatement, and of the form that appends into a cache against the form that
does not, followed by the append."""
import numpy as np
import pytest
import torch

import chunked_prefill_causal_cp_gb300 as cp
from oracle import q4
from q4_util import f64, half_step

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from chunked_prefill_causal_cp_gb300 import _build
    _build.build()


def _freqs(rot, theta=10000.0):
    return (theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().cuda()


def _desc(dtype, hq, hkv, d, batch=1, cap=64):
    return cp.layer_desc(dtype, batch, hq, hkv, d, cp.CP_CACHE_CONTIG, capacity=cap)


def _inputs(dtype, t, hq, hkv, d, seed, fused):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, (hq + 2 * hkv) * d, generator=g)
    x = (x * (1 + 3 * (torch.rand(x.shape[1], generator=g) < 0.1))).to(dtype).cuda()
    parts = x.split([hq * d, hkv * d, hkv * d], dim=1)
    q, k, v = (p.unflatten(1, (-1, d)) for p in parts)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(dtype).cuda() for _ in range(2)]
    return q, k, v, w


def _check(x, y, w, pos, freq, rot, inter, eps, dtype):
    """One rounding of the result (half a step), and fp32 before it: a sum of squares of d terms and its root
    (relative 2^-20 at most), and an angle within 2^-23 + 2^-22 of a sine's own error: 2^-19 (|a| + |b|) covers
    them."""
    ref, mag = q4.norm_rope(f64(x), None if w is None else f64(w), pos, freq, rot, inter, eps)
    tol = half_step(dtype) * np.abs(ref) + 2.0 ** -19 * mag + 1e-30
    if dtype == F16:
        tol = tol + 2.0 ** -25  # subnormal results
    err = np.abs(f64(y) - ref)
    assert np.isfinite(err).all() and (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (128, 128, True), (64, 64, False), (64, 32, True),
                                         (128, 48, False), (64, 16, False), (128, 80, True), (128, 0, False)])
def test_norm_and_rotation(dtype, d, rot, inter):
    for t, hq, hkv, norm, fused in [(1, 32, 8, True, False), (7, 5, 1, True, True), (33, 6, 3, False, True)]:
        q, k, _, w = _inputs(dtype, t, hq, hkv, d, t + d + rot, fused)
        w = w if norm else [None, None]
        freq = _freqs(rot)
        lens = torch.tensor([1000 + t], dtype=torch.int32, device="cuda")
        qo, ko = torch.empty(t, hq, d, dtype=dtype, device="cuda"), torch.empty(t, hkv, d, dtype=dtype, device="cuda")
        prep = cp.qk_prep(rot, inter, eps=1e-5)
        cp.cp_qk_norm_rope(_desc(dtype, hq, hkv, d), prep, q, k, qo, ko, 1, t, q_weight=w[0], k_weight=w[1],
                           inv_freq=freq if rot else None, seqlens_k=lens)
        pos = 1000 + t + np.arange(t)
        _check(q, qo, w[0], pos, f64(freq), rot, inter, 1e-5, dtype)
        _check(k, ko, w[1], pos, f64(freq), rot, inter, 1e-5, dtype)


def test_far_positions_are_exact():
    """Any int32 position, given one by one; large frequencies too."""
    pos = np.array([0, 1, -1, 4095, 2 ** 20 + 1, 123456789, 2 ** 31 - 1, -2 ** 31, -7654321], np.int64)
    t, d = len(pos), 128
    q, k, _, w = _inputs(F32, t, 4, 2, d, 3, False)
    freq = torch.cat([_freqs(96, 500000.0), torch.tensor([3.0, 7.5, -0.25, 1e-9, 0.0, 1e-30, 40.0, 2.0 ** -70,
                                                          -1e-6, 0.3, 0.7, 0.9, 1.0, 1.1, 2.2, 6.25]).cuda()])
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    cp.cp_qk_norm_rope(_desc(F32, 4, 2, d), cp.qk_prep(128), q, k, qo, ko, 1, t, q_weight=w[0], k_weight=w[1],
                       inv_freq=freq, positions=torch.from_numpy(pos).int().cuda())
    _check(q, qo, w[0], pos, f64(freq), 128, False, 1e-6, F32)
    _check(k, ko, w[1], pos, f64(freq), 128, False, 1e-6, F32)


def test_in_place_one_tensor_and_no_rows():
    t, hq, hkv, d = 50, 8, 2, 128
    q, k, _, w = _inputs(BF16, t, hq, hkv, d, 9, False)
    desc, prep, freq = _desc(BF16, hq, hkv, d), cp.qk_prep(128), _freqs(128)
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(q_weight=w[0], k_weight=w[1], inv_freq=freq, seqlens_k=lens)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    cp.cp_qk_norm_rope(desc, prep, q, k, qo, ko, 1, t, **kw)
    q2, k2 = q.clone(), k.clone()
    cp.cp_qk_norm_rope(desc, prep, q2, k2, q2, k2, 1, t, **kw)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    q3, k3 = torch.zeros_like(q), torch.zeros_like(k)
    cp.cp_qk_norm_rope(desc, prep, q, None, q3, None, 1, t, **kw)
    cp.cp_qk_norm_rope(desc, prep, None, k, None, k3, 1, t, stream=torch.cuda.current_stream(), **kw)
    assert torch.equal(q3, qo) and torch.equal(k3, ko)
    cp.cp_qk_norm_rope(desc, prep, q[:0], k[:0], q3[:0], k3[:0], 1, 0, **kw)


def test_ragged_rows_take_their_sequences_positions():
    rows, past = [1, 5, 1, 130, 2], [4000, 0, 17, 999, 250]
    t, hq, hkv, d = sum(rows), 12, 4, 64
    q, k, _, w = _inputs(F16, t, hq, hkv, d, 5, True)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device="cuda")
    lens = torch.tensor(past, dtype=torch.int32, device="cuda")
    qo, ko = (torch.empty(t, h, d, dtype=F16, device="cuda") for h in (hq, hkv))
    cp.cp_qk_norm_rope(_desc(F16, hq, hkv, d), cp.qk_prep(64, True), q, k, qo, ko, 5, t, q_weight=w[0], k_weight=w[1],
                       inv_freq=_freqs(64), seqlens_k=lens, cu_rows=cu)
    pos = np.concatenate([p + np.arange(r) for p, r in zip(past, rows)])
    _check(q, qo, w[0], pos, f64(_freqs(64)), 64, True, 1e-6, F16)
    _check(k, ko, w[1], pos, f64(_freqs(64)), 64, True, 1e-6, F16)


@pytest.mark.parametrize("dtype,d,hq,hkv,fused", [(BF16, 128, 32, 8, True), (F16, 64, 6, 2, False), (F32, 64, 4, 4, True),
                                                  (F32, 128, 3, 1, False)])
@pytest.mark.parametrize("kind", ["contig", "paged", "rolling"])
def test_append_is_the_two_calls(dtype, d, hq, hkv, fused, kind):
    n, r = 3, 37
    t, past = n * r, [0, 60, 91]
    q, k, v, w = _inputs(dtype, t, hq, hkv, d, 21, fused)
    table = None
    if kind == "paged":
        table = torch.randperm(30, generator=torch.Generator().manual_seed(2))[:27].reshape(3, 9).int().cuda()
        desc = cp.layer_desc(dtype, n, hq, hkv, d, cp.CP_CACHE_PAGED, page_size=16, num_pages=30, max_blocks=9)
        lead = (30, hkv, 16)
    else:
        cap = 130 if kind == "contig" else 70
        desc = cp.layer_desc(dtype, n, hq, hkv, d, getattr(cp, "CP_CACHE_" + kind.upper()), capacity=cap)
        lead = (n, hkv, cap)
    lens = torch.tensor(past, dtype=torch.int32, device="cuda")
    kw = dict(q_weight=w[0], k_weight=w[1], inv_freq=_freqs(d))
    prep = cp.qk_prep(d)
    nan = float("nan")
    caches = [torch.full((*lead, d), nan, dtype=dtype, device="cuda") for _ in range(4)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qa, qb, kb = (torch.empty(t, h, d, dtype=dtype, device="cuda") for h in (hq, hq, hkv))
    cp.cp_qk_norm_rope_append(desc, prep, q, k, v, qa, caches[0], caches[1], lens, n, t, 128, block_table=table,
                              dev_status=status, **kw)
    cp.cp_qk_norm_rope(desc, prep, q, k, qb, kb, n, t, seqlens_k=lens, **kw)
    cp.cp_kv_append(desc, kb, v.contiguous(), r, caches[2], caches[3], lens, 91, block_table=table, dev_status=status)
    bits = torch.int32 if dtype == F32 else torch.int16
    for a, b in ((qa, qb), (caches[0], caches[2]), (caches[1], caches[3])):
        assert torch.equal(a.view(bits), b.view(bits))
    assert int(status) == 0 and lens.tolist() == past


def test_append_reports_positions_out_of_bounds_and_touches_nothing_there():
    n, r, hq, hkv, d = 3, 4, 4, 2, 64
    t = n * r
    q, k, v, w = _inputs(BF16, t, hq, hkv, d, 4, False)
    desc = cp.layer_desc(BF16, n, hq, hkv, d, cp.CP_CACHE_PAGED, page_size=16, num_pages=4, max_blocks=2)
    table = torch.tensor([[0, 99], [1, 2], [-5, 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([14, 30, -3], dtype=torch.int32, device="cuda")  # page 99; past max_ctx; negative positions
    kc = torch.full((4, hkv, 16, d), float("nan"), dtype=BF16, device="cuda")
    vc, qo = torch.full_like(kc, float("nan")), torch.empty_like(q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cp.cp_qk_norm_rope_append(desc, cp.qk_prep(64), q, k, v, qo, kc, vc, lens, n, t, 32, q_weight=w[0], k_weight=w[1],
                              inv_freq=_freqs(64), block_table=table, dev_status=status)
    assert int(status) == cp.CP_DEV_BOUNDS
    written = ~torch.isnan(vc).all(-1).all(1)  # [page, slot]
    want = torch.zeros(4, 16, dtype=torch.bool)
    want[0, 14:] = True  # sequence 0: positions 14, 15
    want[2, 14:] = True  # sequence 1: positions 30, 31
    # sequence 2: position 0 is on page -5: nothing
    assert torch.equal(written.cpu(), want)
    pos = np.concatenate([np.arange(p, p + r) for p in (14, 30, -3)])
    _check(q, qo, w[0], pos, f64(_freqs(64)), 64, False, 1e-6, BF16)
    assert torch.equal(vc[2, :, 14:].transpose(0, 1), v[4:6])


def test_ring_with_more_rows_than_slots_keeps_the_newest():
    """Sequences without rows slip past the host's bound; the ring then takes the newest rows and reports."""
    hq, hkv, d, cap = 2, 2, 64, 4
    q, k, v, _ = _inputs(BF16, 6, hq, hkv, d, 6, False)
    desc = cp.layer_desc(BF16, 3, hq, hkv, d, cp.CP_CACHE_ROLLING, capacity=cap)
    kc = torch.full((3, hkv, cap, d), 9.0).bfloat16().cuda()
    vc, qo, status = torch.full_like(kc, 9.0), torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    cp.cp_qk_norm_rope_append(desc, cp.qk_prep(0), q, k, v, qo, kc, vc, torch.zeros(3, dtype=torch.int32, device="cuda"), 3,
                              6, 6, cu_rows=torch.tensor([0, 0, 0, 6], dtype=torch.int32, device="cuda"), dev_status=status)
    assert int(status) == cp.CP_DEV_BOUNDS and torch.equal(qo, q)
    assert (vc[:2] == 9.0).all()
    for pos in range(2, 6):
        assert torch.equal(vc[2, :, pos % cap], v[pos]) and torch.equal(kc[2, :, pos % cap], k[pos])


def test_angles_to_the_last_places():
    """(1, 0) turned by an angle is its cosine and sine: an ulp of the function's own (CUDA's bound for sincospif) and
    an angle within 2^-25, wherever in the turn it falls."""
    t, d = 4096, 128
    g = torch.Generator().manual_seed(31)
    pos = torch.randint(-2 ** 31, 2 ** 31, (t,), generator=g, dtype=torch.int64)
    pos[:2048] = torch.arange(2048)
    x = torch.zeros(t, 1, d)
    x[..., :d // 2] = 1
    x = x.cuda()
    freq = torch.cat([_freqs(64), torch.rand(32, generator=g).cuda() * 3])
    y = torch.empty_like(x)
    cp.cp_qk_norm_rope(_desc(F32, 1, 1, d), cp.qk_prep(d), x, None, y, None, 1, t, inv_freq=freq,
                       positions=pos.int().cuda())
    u = _reduced(pos.numpy(), f64(freq))
    for got, want, slope in ((y[:, 0, :d // 2], np.cos(u), np.sin(u)), (y[:, 0, d // 2:], np.sin(u), np.cos(u))):
        tol = np.spacing(np.abs(want).astype(np.float32)).astype(np.float64) + 2.0 ** -25 * np.abs(slope)
        off = np.abs(f64(got) - want)
        assert (off <= tol).all(), float((off / tol).max())


def _reduced(pos, freq):
    """pos * freq in [0, 2 pi), by whole-number arithmetic: a product of floats has no error in 64 bits, but whole turns
    taken off it there would."""
    two_pi = 0x6487ED5110B4611A62633145C06E0E68948127044533E63A0105DF  # 2 pi * 2^212
    out = np.empty((len(pos), len(freq)))
    for j, f in enumerate(freq.tolist()):
        num, den = f.as_integer_ratio()
        for i, p in enumerate(pos.tolist()):
            out[i, j] = ((p * num << 212) // den) % two_pi / 2 ** 212
    return out
