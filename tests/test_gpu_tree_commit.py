"""GPU tests of the accepted path's commit: the bytes of the cache against the definition."""
import numpy as np
import pytest
import torch

import chunked_prefill_causal_cp_gb300 as cp
from latent_util import Cache, ints

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from chunked_prefill_causal_cp_gb300 import _build
    _build.build()


def _commit(x, path, counts, lens, max_ctx, **kw):
    call = dict(block_table=x.table, dev_status=x.status)
    call.update(kw)
    n, most = path.shape
    if x.latent:
        cp.cp_latent_tree_commit(x.desc, x.x, path, counts, lens, n, most, max_ctx, **call)
    else:
        cp.cp_tree_commit(x.desc, x.k, x.v, path, counts, lens, n, most, max_ctx, **call)


def _bits(arrays):
    return [a.clone().view(torch.int32 if a.dtype == F32 else torch.int16) for a in arrays]


def _expect(x, path, counts, lens):
    """The cache's arrays after the commit of the sequences with a list of places."""
    want = [a.clone() for a in x.arrays]
    for s, (p, n, at) in enumerate(zip(path, counts, lens)):
        for a, w in zip(x.arrays, want):
            rows = torch.stack([x.at(a, s, at + e, 1)[0] for e in p[:n]]) if n else None
            if n:
                x.put(w, s, at, rows)
    return want


@pytest.mark.parametrize("dtype,kw", [(BF16, dict(kv=8, d=128)), (F16, dict(kv=3, d=64, page=16)), (F32, dict(kv=5, d=128, page=32)),
                                      (F32, dict(kv=2, d=64)), (BF16, dict(latent=512, rope=64, page=64)),
                                      (F16, dict(latent=128, rope=16))])
def test_paths_move(dtype, kw):
    kw = dict(kw)
    page = kw.pop("page", 0)
    heads = kw.get("kv", 4)
    g = np.random.default_rng(3)
    lens = [0, 5, 60, 127, 31, 250, 16]
    path = [[0, 1, 2], [], [0, 2, 3], list(range(1, 33)), [127], sorted(g.choice(128, 20, replace=False).tolist()), [3, 4, 5, 6, 7, 8, 9, 10, 11]]
    most = 40
    x = Cache(dtype, heads, 7, 400, page, **kw)
    x.fill([n + 128 for n in lens])
    want = _expect(x, path, [len(p) for p in path], lens)
    dev = ints(lens)
    _commit(x, ints([p + [9] * (most - len(p)) for p in path]), ints([len(p) for p in path]), dev, 400)
    assert dev.tolist() == [n + len(p) for n, p in zip(lens, path)]
    assert int(x.status) == 0
    for a, b in zip(_bits(x.arrays), _bits(want)):
        assert torch.equal(a, b)
    # Another layer of the same model: the same lengths, not advanced.
    y = Cache(dtype, heads, 7, 400, page, seed=0, **kw)
    y.fill([n + 128 for n in lens])
    dev = ints(lens)
    _commit(y, ints([p + [9] * (most - len(p)) for p in path]), ints([len(p) for p in path]), dev, 400, commit=False)
    assert dev.tolist() == lens
    for a, b in zip(_bits(y.arrays), _bits(want)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kw", [dict(kv=2, d=128), dict(latent=256, rope=32)])
def test_what_is_out_of_range_is_left_as_it_was(kw):
    heads = kw.get("kv", 4)
    x = Cache(BF16, heads, 8, 64, 16, **kw)
    x.fill([64] * 8)
    x.table[6, 1] = x.pages
    x.table[7, 3] = -1
    path = [[0, 2, 4], [2, 2, 3], [0, 3, 1], [-1, 1, 2], [0, 1, 60], [0, 1, 2], [0, 1, 9], [0, 2, 4]]
    counts, lens = [3, 3, 3, 3, 3, 4, 3, 3], [10, 10, 10, 10, 10, 10, 10, 10]
    before = _bits(x.arrays)
    want = _expect(x, [path[0]] + [[]] * 6 + [path[7]], [3, 0, 0, 0, 0, 0, 0, 3], lens)
    dev = ints(lens)
    _commit(x, ints(path), ints(counts), dev, 64)
    assert int(x.status) == cp.CP_DEV_BOUNDS
    assert dev.tolist() == [13, 10, 10, 10, 10, 10, 10, 13]  # the page that sequence 7 lacks is none of its own
    for a, b, c in zip(_bits(x.arrays), _bits(want), before):
        assert torch.equal(a, b) and not torch.equal(a, c)
    for bad in (([-1] * 8, lens), ([3] * 8, [-5] * 8), ([3] * 8, [2 ** 31 - 1] * 8), ([2 ** 31 - 1] * 8, lens)):
        x.status.zero_()
        now, dev = _bits(x.arrays), ints(bad[1])
        _commit(x, ints(path), ints(bad[0]), dev, 64)
        assert int(x.status) == cp.CP_DEV_BOUNDS and dev.tolist() == bad[1]
        for a, b in zip(_bits(x.arrays), now):
            assert torch.equal(a, b)


def test_commit_in_a_graph():
    x = Cache(BF16, 4, 2, 256, 16, kv=4, d=64)
    x.fill([256, 256])
    dev, path, counts = ints([20, 30]), ints([[0, 3, 5], [1, 2, 8]]), ints([3, 2])
    _commit(x, path, ints([0, 0]), dev, 256)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        _commit(x, path, counts, dev, 256)
    for p, c in (([[0, 3, 5], [1, 2, 8]], [3, 2]), ([[2, 4, 6], [0, 1, 3]], [1, 3])):
        at = dev.tolist()
        want = _expect(x, p, c, at)
        path.copy_(ints(p))
        counts.copy_(ints(c))
        g.replay()
        torch.cuda.synchronize()
        assert dev.tolist() == [a + b for a, b in zip(at, c)]
        for a, b in zip(_bits(x.arrays), _bits(want)):
            assert torch.equal(a, b)
