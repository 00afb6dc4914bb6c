"""GPU parity of attention over a 4-bit cache at the lengths where the split path
changes its split size, beyond eight splits, and in calls of many sequences."""
import numpy as np
import pytest
import torch

import chunked_prefill_causal_cp_gb300 as cp
from q4_util import Cache4, check_attention

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


def _attend(c, q, rows, past, max_ctx, cu=None, table=None, arg=None, desc=None):
    out, n = torch.full_like(q, float("nan")), len(rows)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    desc = desc or c.desc
    ws = torch.full((cp.cp_workspace_size_q4(desc, sum(rows), max_ctx, n),), 255, dtype=torch.uint8, device="cuda")
    cp.cp_chunk_attn_q4(desc, q, arg or c.arg, _ints(past), n, sum(rows), max_ctx, out, ws, commit=False, cu_rows=cu,
                        block_table=c.table if table is None else table, dev_status=status)
    assert int(status) == 0
    return out


# 256 keys a split up to 2048, 512 up to 16384, 1024 beyond; a merge takes eight splits side by side.
ENDS = [1, 256, 257, 2047, 2048, 2049, 4097, 9000, 16383, 16384, 16385, 20011]


@pytest.mark.parametrize("rows,dtype,hq,hkv,d,page", [
    (1, BF16, 4, 1, 64, 0), (1, F16, 2, 2, 64, 16), (1, BF16, 16, 1, 128, 128), (1, F16, 4, 2, 128, 0),
    (4, BF16, 4, 1, 64, 16), (16, F16, 1, 1, 64, 0), (3, BF16, 2, 1, 128, 64), (2, BF16, 4, 1, 128, 0)])
def test_split_sizes(rows, dtype, hq, hkv, d, page):
    """Every regime of split sizes in one call, against 64 bits; and each sequence as in a call of its own, with bounds of
    its own, bit for bit."""
    past = [max(n - rows, 0) for n in ENDS]
    n = len(past)
    c = Cache4(dtype, hq, hkv, d, n, 20032, page)
    c.fill([p + rows for p in past])
    q = torch.randn(n * rows, hq, d, generator=torch.Generator().manual_seed(rows)).to(dtype).cuda()
    out = _attend(c, q, [rows] * n, past, 20032)
    check_attention(c, q, out, past, [rows] * n)
    for i in range(n):
        arg, desc, table = c.view(i)
        one = slice(i * rows, (i + 1) * rows)
        alone = _attend(c, q[one], [rows], past[i:i + 1], past[i] + rows, arg=arg, desc=desc,
                        table=None if table is None else table[i:i + 1])
        assert torch.equal(alone, out[one])


@pytest.mark.parametrize("dtype,hq,hkv,d,page", [(BF16, 4, 2, 64, 16), (F16, 8, 1, 128, 0)])
def test_many_sequences(dtype, hq, hkv, d, page):
    """Chunks far down a list of sequences, single rows around them."""
    n = 103
    rows = [1] * n
    for i, r in ((0, 5), (31, 2), (32, 70), (33, 17), (64, 129), (95, 3), (96, 260), (102, 40)):
        rows[i] = r
    past = [(37 * i) % 300 for i in range(n)]
    c = Cache4(dtype, hq, hkv, d, n, 600, page)
    c.fill([p + r for p, r in zip(past, rows)])
    q = torch.randn(sum(rows), hq, d, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    out = _attend(c, q, rows, past, 600, cu=_ints([0, *np.cumsum(rows).tolist()]))
    check_attention(c, q, out, past, rows)
