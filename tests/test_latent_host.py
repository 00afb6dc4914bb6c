"""Refusals of the latent cache's and the drafted trees' calls, made on the host before anything is enqueued, and the
64-bit restatement's own pins."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import chunked_prefill_causal_cp_gb300 as cp
from oracle import latent as oracle

FAKE = 1 << 20  # a 16-byte aligned non-null address; never dereferenced (the checks fail first)
INVALID, UNSUP, CAP, WS = (cp.CP_ERR_INVALID_ARG, cp.CP_ERR_UNSUPPORTED, cp.CP_ERR_CAPACITY, cp.CP_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def built():
    from chunked_prefill_causal_cp_gb300 import _build
    _build.build()


def _latent(**kw):
    base = dict(dtype=torch.bfloat16, batch=4, num_heads=16, latent_dim=512, rope_dim=64, kind=cp.CP_CACHE_CONTIG,
                capacity=1024)
    base.update(kw)
    return cp.latent_desc(**base)


def _layer(**kw):
    base = dict(dtype=torch.bfloat16, batch=4, num_q_heads=8, num_kv_heads=2, head_dim=128, kind=cp.CP_CACHE_CONTIG,
                capacity=1024)
    base.update(kw)
    return cp.layer_desc(**base)


PAGED = dict(kind=cp.CP_CACHE_PAGED, page_size=16, num_pages=64, max_blocks=8)


def _append(desc=None, prep=None, x=FAKE, xs=0, k=FAKE, ks=0, w=FAKE, freq=FAKE, pos=None, q=FAKE, qr=0, qh=0, qo=2 * FAKE,
            outr=0, outh=0, cu=None, n=4, t=8, cache=3 * FAKE, lens=FAKE, table=None, ctx=1024, st=None):
    desc, prep = desc or _latent(), prep or cp.qk_prep(64)
    return cp.lib().cp_latent_append(ctypes.byref(desc), ctypes.byref(prep), x, xs, k, ks, w, freq, pos, q, qr, qh, qo, outr,
                                     outh, cu, n, t, cache, lens, table, ctx, st, None)


BAD_LATENT = [(dict(dtype=torch.float32), UNSUP), (dict(kind=cp.CP_CACHE_ROLLING), UNSUP), (dict(latent_dim=100), UNSUP),
              (dict(latent_dim=640), UNSUP), (dict(latent_dim=0), INVALID), (dict(latent_dim=-128), INVALID),
              (dict(rope_dim=72), UNSUP), (dict(rope_dim=80), UNSUP), (dict(rope_dim=-16), INVALID), (dict(nope_dim=96), UNSUP),
              (dict(v_dim=256), UNSUP), (dict(nope_dim=0), INVALID), (dict(v_dim=-64), INVALID), (dict(num_heads=0), INVALID),
              (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
              (dict(kind=7), INVALID), (dict(capacity=0), INVALID), (dict(kind=cp.CP_CACHE_PAGED, page_size=24), UNSUP)]


def test_append_refusals():
    for kw, want in BAD_LATENT:
        assert _append(desc=_latent(**kw)) == want, kw
    assert _append(prep=cp.qk_prep(80)) == INVALID and _append(prep=cp.qk_prep(-16)) == INVALID
    assert _append(prep=cp.qk_prep(24)) == UNSUP and _append(prep=cp.QKPrep(64, 2, 1e-6)) == INVALID
    assert _append(prep=cp.qk_prep(64, eps=-1.0)) == INVALID and _append(prep=cp.qk_prep(64, eps=float("inf"))) == INVALID
    for f in ("x", "k", "cache", "lens", "freq"):
        assert _append(**{f: None}) == INVALID, f
    for f in ("x", "k", "w", "q", "qo", "cache"):
        assert _append(**{f: FAKE + 8}) == INVALID, f
    for f in ("freq", "pos", "cu", "lens", "table", "st"):
        assert _append(**{f: FAKE + 2}) == INVALID, f
    assert _append(q=None) == INVALID and _append(qo=None) == INVALID
    assert _append(xs=504) == INVALID and _append(xs=516) == INVALID and _append(xs=1 << 60) == UNSUP
    assert _append(ks=56) == INVALID and _append(ks=65) == INVALID
    assert _append(qh=56) == INVALID and _append(qh=68) == INVALID and _append(qr=16 * 64 - 8) == INVALID
    assert _append(outh=576, outr=16 * 576 - 8) == INVALID and _append(outh=1 << 55) == UNSUP
    assert _append(outh=(2 ** 63 - 1 >> 34) // 16 * 16) == UNSUP
    assert _append(qo=FAKE, outh=128) == INVALID  # in place with other strides
    assert _append(n=0) == INVALID and _append(t=-4) == INVALID and _append(n=3) == INVALID
    assert _append(n=5, t=10) == INVALID and _append(ctx=1025) == CAP and _append(ctx=0) == INVALID
    assert _append(desc=_latent(**PAGED), ctx=128) == INVALID and _append(desc=_latent(**PAGED), table=FAKE, ctx=129) == CAP
    assert _append(desc=_latent(num_heads=70000)) == UNSUP
    assert _append(t=0) == cp.CP_OK


def _attn(desc=None, q=FAKE, cache=FAKE, lens=FAKE, table=None, par=None, cu=None, n=4, t=8, ctx=1024, out=1 << 40, ws=FAKE,
          ws_bytes=1 << 50, commit=0, st=None):
    desc = desc or _latent()
    return cp.lib().cp_latent_attn(ctypes.byref(desc), q, cache, lens, table, par, cu, n, t, ctx, out, ws, ws_bytes, commit,
                                   st, None)


def _tree(desc=None, q=FAKE, k=FAKE, v=FAKE, lens=FAKE, table=None, par=FAKE, cu=None, n=4, t=8, ctx=1024, out=1 << 40,
          ws=FAKE, ws_bytes=1 << 50, st=None):
    desc = desc or _layer()
    return cp.lib().cp_tree_attn(ctypes.byref(desc), q, k, v, lens, table, par, cu, n, t, ctx, out, ws, ws_bytes, st, None)


@pytest.mark.parametrize("f,desc", [(_attn, _latent), (_tree, _layer)])
def test_attention_refusals(f, desc):
    for arg in ("q", "lens", "out"):
        assert f(**{arg: None}) == INVALID, arg
    for arg in ("q", "out"):
        assert f(**{arg: FAKE + 8}) == INVALID, arg
    for arg in ("lens", "table", "par", "cu", "st"):
        assert f(**{arg: FAKE + 2}) == INVALID, arg
    assert f(out=FAKE) == INVALID and f(out=FAKE + 16) == INVALID and f(q=FAKE + 16, out=FAKE) == INVALID
    assert f(n=0) == INVALID and f(t=-1) == INVALID and f(n=3) == INVALID and f(n=5, t=10) == INVALID
    assert f(ctx=1025) == CAP and f(ctx=0) == INVALID
    assert f(desc=desc(**PAGED), ctx=128) == INVALID and f(desc=desc(**PAGED), table=FAKE, ctx=129) == CAP
    big = dict(kind=cp.CP_CACHE_PAGED, page_size=128, num_pages=64, max_blocks=2 ** 24 - 1)
    assert f(desc=desc(**big), table=FAKE, ctx=2 ** 31 - 200) == UNSUP
    assert f(par=FAKE, n=1, t=129) == UNSUP  # a tree's most rows
    assert f(t=2 ** 30) == UNSUP
    assert f(ctx=1000, ws=None) == WS and f(ctx=1000, ws_bytes=64) == WS and f(ctx=1000, ws=FAKE + 8) == WS
    assert f(t=0) == cp.CP_OK


def test_attention_refusals_of_each():
    for kw, want in BAD_LATENT:
        assert _attn(desc=_latent(**kw)) == want, kw
    assert _attn(cache=None) == INVALID and _attn(cache=FAKE + 8) == INVALID
    assert _attn(par=FAKE, commit=1) == INVALID
    assert _tree(par=None) == INVALID and _tree(k=None) == INVALID and _tree(v=None) == INVALID
    assert _tree(k=FAKE + 8) == INVALID and _tree(v=FAKE + 4) == INVALID
    assert _tree(desc=_layer(dtype=torch.float32)) == UNSUP and _tree(desc=_layer(kind=cp.CP_CACHE_ROLLING)) == UNSUP
    assert _tree(desc=_layer(head_dim=96)) == UNSUP and _tree(desc=_layer(num_q_heads=130, num_kv_heads=2)) == UNSUP
    assert _tree(desc=_layer(num_q_heads=7)) == INVALID


def test_workspace_sizes():
    for size, desc in ((cp.cp_workspace_size_latent, _latent), (cp.cp_workspace_size_tree, _layer)):
        assert size(desc(dtype=torch.float32), 8, 1024, 4) == 0 and size(desc(kind=cp.CP_CACHE_ROLLING), 8, 1024, 4) == 0
        assert size(desc(), 0, 1024, 4) == 0 and size(desc(), 8, 0, 4) == 0 and size(desc(), 8, 1024, 0) == 0
        for t, n in ((1, 1), (4, 4), (60, 3), (1000, 2)):  # a size suffices for every smaller call
            top = size(desc(), t, 100000, n)
            for ctx in (1, 64, 65, 1000, 5000, 30000, 99999):
                for rows in {1, n, t // 2 + 1, t}:
                    assert size(desc(), min(rows, t), ctx, min(n, rows)) <= top


def _expanded(desc=None, q=FAKE, k=FAKE, kr=0, kh=0, r=FAKE, rr=0, v=FAKE, vr=0, vh=0, cu=None, ck=None, n=4, t=8, nk=16,
              out=1 << 40, st=None):
    desc = desc or _latent()
    return cp.lib().cp_latent_chunk_attn(ctypes.byref(desc), q, k, kr, kh, r, rr, v, vr, vh, cu, ck, n, t, nk, out, st, None)


def test_expanded_refusals():
    for kw, want in BAD_LATENT:
        assert _expanded(desc=_latent(**kw)) == want, kw
    for f in ("q", "k", "r", "v", "out"):
        assert _expanded(**{f: None}) == INVALID, f
        assert _expanded(**{f: FAKE + 8}) == INVALID, f
    assert _expanded(cu=FAKE) == INVALID and _expanded(ck=FAKE) == INVALID
    assert _expanded(cu=FAKE + 2, ck=FAKE) == INVALID and _expanded(cu=FAKE, ck=FAKE + 1) == INVALID
    assert _expanded(st=FAKE + 2) == INVALID
    assert _expanded(kh=120) == INVALID and _expanded(kh=129) == INVALID and _expanded(kr=16 * 128 - 8) == INVALID
    assert _expanded(vh=120) == INVALID and _expanded(vr=8) == INVALID and _expanded(rr=56) == INVALID
    assert _expanded(rr=1 << 60) == UNSUP and _expanded(kr=1 << 60) == UNSUP
    assert _expanded(n=0) == INVALID and _expanded(t=-1) == INVALID and _expanded(nk=-4) == INVALID
    assert _expanded(n=3, t=9) == INVALID and _expanded(n=3, t=8, nk=18) == INVALID
    assert _expanded(out=FAKE) == INVALID and _expanded(out=FAKE + 16) == INVALID
    assert _expanded(n=1, t=2 ** 30) == UNSUP and _expanded(n=1, nk=2 ** 31 - 100) == UNSUP
    assert _expanded(t=0) == cp.CP_OK


def _commit(latent, desc=None, k=FAKE, v=FAKE, path=FAKE, cnt=FAKE, lens=FAKE, table=None, n=4, most=3, ctx=1024, st=None):
    L = cp.lib()
    if latent:
        return L.cp_latent_tree_commit(ctypes.byref(desc or _latent()), k, path, cnt, lens, table, n, most, ctx, 1, st, None)
    return L.cp_tree_commit(ctypes.byref(desc or _layer()), k, v, path, cnt, lens, table, n, most, ctx, 1, st, None)


@pytest.mark.parametrize("latent", [True, False])
def test_commit_refusals(latent):
    make = _latent if latent else _layer
    f = lambda **kw: _commit(latent, **kw)  # noqa: E731
    assert f(desc=make(kind=cp.CP_CACHE_ROLLING)) == UNSUP
    for arg in ("k", "path", "cnt", "lens"):
        assert f(**{arg: None}) == INVALID, arg
    assert f(k=FAKE + 8) == INVALID
    for arg in ("path", "cnt", "lens", "table", "st"):
        assert f(**{arg: FAKE + 2}) == INVALID, arg
    if latent:
        for kw, want in BAD_LATENT:
            assert f(desc=_latent(**kw)) == want, kw
    else:
        assert f(v=None) == INVALID and f(v=FAKE + 4) == INVALID and f(desc=_layer(head_dim=80)) == UNSUP
    assert f(n=-1) == INVALID and f(most=-1) == INVALID and f(most=129) == UNSUP
    assert f(n=5) == INVALID and f(ctx=1025) == CAP and f(ctx=0) == INVALID
    assert f(desc=make(**PAGED), ctx=128) == INVALID and f(desc=make(**PAGED), table=FAKE, ctx=129) == CAP
    assert f(n=0) == cp.CP_OK and f(most=0) == cp.CP_OK


def test_binding_refuses_host_tensors():
    """CPU tensors are refused before the library is reached."""
    x = torch.zeros(8, 576, dtype=torch.bfloat16)
    lens = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: cp.cp_latent_append(_latent(), cp.qk_prep(0), x[:, :512], x[:, 512:], x, lens, 4, 8, 64),
                 lambda: cp.cp_latent_attn(_latent(), x, x, lens, 4, 8, 64, x, None),
                 lambda: cp.cp_latent_chunk_attn(_latent(), x, x, x, x, x, 4, 8, 8),
                 lambda: cp.cp_tree_attn(_layer(), x, x, x, lens, lens, 4, 8, 64, x, None),
                 lambda: cp.cp_tree_commit(_layer(), x, x, lens, lens, lens, 4, 1, 64),
                 lambda: cp.cp_latent_tree_commit(_latent(), x, lens, lens, lens, 4, 1, 64)):
        with pytest.raises(cp.CPError) as e:
            call()
        assert e.value.status == INVALID


_STRIDED = """
import torch
import chunked_prefill_causal_cp_gb300 as cp
torch._C._cuda_getDevice = lambda: 0
D = torch.bfloat16
def at(t, shape):
    class T:  # a stand-in with a device index: the check reads nothing else of the GPU
        dtype, shape_ = t.dtype, t.shape
        shape = property(lambda s: t.shape)
        def __getattr__(s, n): return getattr(t, n)
        def get_device(s): return 0
    return cp._rows3_arg("x", T(), D, *shape, 0) if len(shape) == 3 else cp._rows2_arg("x", T(), D, *shape, 0)
x = torch.zeros(6, 4, 80, dtype=D)
p = x.data_ptr()
assert at(x, (6, 4, 80)) == (p, 320, 80)
assert at(x[..., 16:], (6, 4, 64)) == (p + 32, 320, 80)
assert at(x[:1, :, 16:], (1, 4, 64)) == (p + 32, 320, 80)
assert at(x[:, :1, 16:], (6, 1, 64))[1:] == (320, 64)
assert at(x[:, 0], (6, 80)) == (p, 320) and at(x[:1, 0, 8:40], (1, 32)) == (p + 16, 32)
assert at(x[::2], (3, 4, 80)) == (p, 640, 80)
assert at(x[:0], (0, 4, 80))[1:] == (320, 80) and at(x[:0, 0], (0, 80))[1:] == (80,)
bad = [(x, (6, 4, 64)), (x.transpose(0, 1), (4, 6, 80)), (x[..., ::2], (6, 4, 40)), (x[:, :1].expand(6, 4, 80), (6, 4, 80)),
       (x[:1].expand(6, 4, 80), (6, 4, 80)), (x.float(), (6, 4, 80)), (x[:1, 0].expand(6, 80), (6, 80)), (x[0].T, (80, 4)),
       (x[:, 0, ::2], (6, 40)), (x[:, 0], (6, 64))]
for t, shape in bad:
    try:
        at(t, shape)
    except cp.CPError as e:
        assert e.status == cp.CP_ERR_INVALID_ARG
    else:
        raise AssertionError((t.shape, t.stride(), shape))
"""


def test_binding_takes_slices_of_wider_rows_and_refuses_other_strides():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _STRIDED], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_restatement_of_what_rows_see():
    see = oracle.sees(5, 2, [-1, 0, 0, 2, -1])
    want = ["1110000", "1111000", "1110100", "1110110", "1100001"]
    assert see.astype(int).tolist() == [[int(c) for c in w] for w in want]
    assert np.array_equal(oracle.sees(4, 3), np.arange(7) <= 3 + np.arange(4)[:, None])
    g = np.random.default_rng(0)
    q, k, v = g.normal(size=(3, 4, 8)), g.normal(size=(6, 2, 8)), g.normal(size=(6, 2, 5))
    out, mag, big = oracle.attention(q, k, v, oracle.sees(3, 3), 0.5)
    for i in range(3):
        for h in range(4):
            w = np.array([np.exp(0.5 * float(q[i, h] @ k[j, h // 2])) for j in range(4 + i)])
            assert np.allclose(out[i, h], (w[:, None] * v[:4 + i, h // 2]).sum(0) / w.sum())
    assert (mag >= np.abs(out) - 1e-12).all() and (big > 0).all()
