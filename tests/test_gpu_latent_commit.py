"""GPU tests of the lengths' advance behind attention over a latent cache: sequences that the call skips keep theirs."""
import pytest
import torch

import chunked_prefill_causal_cp_gb300 as cp
from latent_util import Cache, ints

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from chunked_prefill_causal_cp_gb300 import _build
    _build.build()


def _attend(x, q, lens, n, max_ctx, cu_rows):
    t = q.shape[0]
    out, ws = x.empty_out(t), torch.zeros(cp.cp_workspace_size_latent(x.desc, t, max_ctx, n), dtype=torch.uint8, device="cuda")
    cp.cp_latent_attn(x.desc, q, x.x, lens, n, t, max_ctx, out, ws, cu_rows=cu_rows, block_table=x.table, commit=True,
                      dev_status=x.status)
    return out


@pytest.mark.parametrize("page", [0, 16])
def test_equal_rows(page):
    """A negative length, and lengths whose rows pass the bound by one and by 2^31."""
    x = Cache(BF16, 4, 5, 128, page, latent=128, rope=16)
    x.fill([100] * 5)
    q, now = x.queries(10), [30, -1, 2 ** 31 - 1, 99, 98]
    lens = ints(now)
    out = _attend(x, q, lens, 5, 100, None)
    assert int(x.status) == cp.CP_DEV_BOUNDS
    assert torch.isnan(out[2:8]).all()
    assert lens.tolist() == [32, -1, 2 ** 31 - 1, 99, 100]
    for s in (0, 4):
        y = Cache(BF16, 4, 1, 128, latent=128, rope=16)
        y.put(y.x, 0, 0, x.at(x.x, s, 0, 100))
        y.check(q[2 * s:2 * s + 2], out[2 * s:2 * s + 2], [now[s]], [2])


def test_ragged_rows():
    """A sequence past the bound, one with a negative length, one without rows, a descending pair of offsets and rows past
    the total."""
    x = Cache(BF16, 4, 7, 128, latent=128, rope=16)
    x.fill([100] * 7)
    now = [30, 99, -7, 5, 40, 60, 7]
    lens = ints(now)
    out = _attend(x, x.queries(10), lens, 7, 100, ints([0, 2, 5, 6, 6, 4, 8, 11]))
    assert int(x.status) == cp.CP_DEV_BOUNDS
    assert lens.tolist() == [32, 99, -7, 5, 40, 64, 7]
    assert torch.isfinite(out[:2].float()).all() and torch.isnan(out[2:4]).all() and torch.isfinite(out[4:8].float()).all()
    assert torch.isnan(out[8:]).all()


def test_in_a_graph():
    x = Cache(BF16, 4, 2, 256, 16, latent=256, rope=0)
    x.fill([256, 256])
    lens, q = ints([100, 300]), x.queries(6)
    _attend(x, q, ints([0, 0]), 2, 200, None)
    out, ws = x.empty_out(6), torch.zeros(cp.cp_workspace_size_latent(x.desc, 6, 200, 2), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cp.cp_latent_attn(x.desc, q, x.x, lens, 2, 6, 200, out, ws, block_table=x.table, commit=True, dev_status=x.status)
    for want in ([103, 300], [106, 300]):
        g.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == want
