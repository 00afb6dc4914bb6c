"""GPU parity of the query/key norm and rotary position with many rows, where a
warp takes several blocks of a token's head rows, some of them uneven."""
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


def _check(x, y, w, pos, freq, rot, inter, dtype):
    """Half a step for the one rounding, and 2^-19 (|a| + |b|) for fp32 before it: a norm of d terms (relative 2^-20 at
    most) and an angle and its sine within 2^-22."""
    ref, mag = q4.norm_rope(f64(x), f64(w), pos, freq, rot, inter, 1e-6)
    tol = half_step(dtype) * np.abs(ref) + 2.0 ** -19 * mag + (2.0 ** -25 if dtype == F16 else 1e-30)
    err = np.abs(f64(y) - ref)
    assert np.isfinite(err).all() and (err <= tol).all(), float((err / tol).max())


# Rows and heads so that a warp takes 2 of 10 blocks, 4 of 10 (the last 2), all of them, and heads that do not fill one.
@pytest.mark.parametrize("dtype,t,hq,hkv,d,rot,inter", [
    (BF16, 700, 32, 8, 128, 128, False), (BF16, 1700, 32, 8, 128, 64, True), (BF16, 5003, 5, 1, 128, 128, False),
    (F16, 1301, 9, 3, 64, 64, False), (F16, 5003, 14, 7, 64, 32, True), (F32, 1700, 7, 1, 64, 64, True),
    (F32, 2503, 6, 3, 128, 48, False), (F32, 4865, 3, 3, 128, 128, False)])
def test_many_rows(dtype, t, hq, hkv, d, rot, inter):
    """Out of place from a fused projection, in place, and the form that appends, which is the plain form and the append."""
    g = torch.Generator().manual_seed(t + d)
    x = torch.randn(t, (hq + 2 * hkv) * d, generator=g).to(dtype).cuda()
    q, k, v = (y.unflatten(1, (-1, d)) for y in x.split([hq * d, hkv * d, hkv * d], dim=1))
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(dtype).cuda() for _ in range(2))
    freq = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
    desc = cp.layer_desc(dtype, 1, hq, hkv, d, cp.CP_CACHE_PAGED, page_size=64, num_pages=100, max_blocks=90)
    table = torch.randperm(100, generator=g)[:90].int().cuda()[None].contiguous()
    lens, prep = torch.tensor([333], dtype=torch.int32, device="cuda"), cp.qk_prep(rot, inter)
    kw = dict(q_weight=wq, k_weight=wk, inv_freq=freq, seqlens_k=lens)
    qo, ko = torch.empty(t, hq, d, dtype=dtype, device="cuda"), torch.empty(t, hkv, d, dtype=dtype, device="cuda")
    cp.cp_qk_norm_rope(desc, prep, q, k, qo, ko, 1, t, **kw)
    pos = 333 + np.arange(t)
    _check(q, qo, wq, pos, f64(freq), rot, inter, dtype)
    _check(k, ko, wk, pos, f64(freq), rot, inter, dtype)
    q2, k2 = q.contiguous(), k.contiguous()
    cp.cp_qk_norm_rope(desc, prep, q2, k2, q2, k2, 1, t, **kw)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    caches = [torch.zeros(100, hkv, 64, d, dtype=dtype, device="cuda") for _ in range(4)]
    q3, status = torch.empty_like(qo), torch.zeros(1, dtype=torch.int32, device="cuda")
    del kw["seqlens_k"]
    cp.cp_qk_norm_rope_append(desc, prep, q, k, v, q3, caches[0], caches[1], lens, 1, t, 90 * 64, block_table=table,
                              dev_status=status, **kw)
    cp.cp_kv_append(desc, ko, v.contiguous(), t, caches[2], caches[3], lens, 333, block_table=table, dev_status=status)
    assert int(status) == 0 and torch.equal(q3, qo)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
