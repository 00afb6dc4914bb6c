"""Refusals of the query/key preparation and of the 4-bit cache's calls, made on
the host before anything is enqueued, and the 64-bit restatement's own pins."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import chunked_prefill_causal_cp_gb300 as cp
from oracle import q4

FAKE = 1 << 20  # a 16-byte aligned non-null address; never dereferenced (the checks fail first)
INVALID, UNSUP, CAP, WS = (cp.CP_ERR_INVALID_ARG, cp.CP_ERR_UNSUPPORTED, cp.CP_ERR_CAPACITY, cp.CP_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def built():
    from chunked_prefill_causal_cp_gb300 import _build
    _build.build()


def _desc(**kw):
    base = dict(dtype=torch.bfloat16, batch=4, num_q_heads=8, num_kv_heads=2, head_dim=128,
                kind=cp.CP_CACHE_CONTIG, capacity=1024)
    base.update(kw)
    return cp.layer_desc(**base)


def _paged(**kw):
    return _desc(kind=cp.CP_CACHE_PAGED, page_size=16, num_pages=64, max_blocks=8, **kw)


def _cache(**kw):
    p = dict(k_codes=FAKE, v_codes=FAKE, k_params=FAKE, v_params=FAKE)
    p.update(kw)
    return cp.Q4Cache(*(p[f] for f, _ in cp.Q4Cache._fields_))


def _rope(desc=None, prep=None, q=FAKE, qs=0, k=2 * FAKE, ks=0, freq=FAKE, pos=None, lens=FAKE, cu=None, n=1, t=8,
          qo=3 * FAKE, ko=4 * FAKE, wq=FAKE):
    desc, prep = desc or _desc(), prep or cp.qk_prep(128)
    return cp.lib().cp_qk_norm_rope(ctypes.byref(desc), ctypes.byref(prep), q, qs, k, ks, wq, FAKE, freq, pos, lens, cu,
                                    n, t, qo, ko, None)


def test_rope_refusals():
    assert _rope(prep=cp.qk_prep(130)) == INVALID
    assert _rope(prep=cp.qk_prep(-16)) == INVALID
    assert _rope(prep=cp.qk_prep(24)) == UNSUP
    assert _rope(prep=cp.qk_prep(128, eps=-1.0)) == INVALID
    assert _rope(prep=cp.qk_prep(128, eps=float("nan"))) == INVALID
    assert _rope(prep=cp.QKPrep(128, 2, 1e-6)) == INVALID
    assert _rope(desc=_desc(head_dim=96)) == UNSUP
    assert _rope(freq=None) == INVALID
    assert _rope(freq=FAKE + 2) == INVALID
    assert _rope(q=None) == INVALID and _rope(qo=None) == INVALID and _rope(ko=None) == INVALID
    assert _rope(q=FAKE + 8) == INVALID and _rope(wq=FAKE + 2) == INVALID and _rope(ko=4 * FAKE + 2) == INVALID
    assert _rope(qs=1000) == INVALID  # less than the row
    assert _rope(qs=1025) == INVALID  # not whole 16-byte pieces
    assert _rope(ks=1 << 62) == UNSUP
    assert _rope(lens=None) == INVALID
    assert _rope(n=0) == INVALID and _rope(t=-1) == INVALID
    assert _rope(n=3, t=8) == INVALID  # equal rows: 8 / 3
    assert _rope(qo=FAKE + 16) == INVALID  # overlaps its input, not in place
    assert _rope(qo=FAKE, qs=2048) == INVALID  # in place, but strided
    assert _rope(qo=2 * FAKE) == INVALID  # over k
    assert _rope(ko=3 * FAKE + 16) == INVALID  # over q_out
    assert _rope(t=0) == cp.CP_OK and _rope(q=None, qo=None, k=None, ko=None) == cp.CP_OK


def _append(desc=None, q=FAKE, k=2 * FAKE, v=3 * FAKE, vs=0, cu=None, n=4, t=8, qo=4 * FAKE, kc=FAKE, lens=FAKE, table=None,
            max_ctx=1024):
    desc, prep = desc or _desc(), cp.qk_prep(128)
    return cp.lib().cp_qk_norm_rope_append(ctypes.byref(desc), ctypes.byref(prep), q, 0, k, 0, v, vs, FAKE, FAKE, FAKE,
                                           None, cu, n, t, qo, kc, FAKE, lens, table, max_ctx, None, None)


def test_rope_append_refusals():
    assert _append(k=None) == INVALID and _append(v=None) == INVALID and _append(kc=None) == INVALID
    assert _append(lens=None) == INVALID and _append(q=None, qo=None) == INVALID
    assert _append(kc=FAKE + 4) == INVALID and _append(v=3 * FAKE + 4) == INVALID and _append(vs=8) == INVALID
    assert _append(max_ctx=1025) == CAP and _append(max_ctx=0) == INVALID
    assert _append(n=5, t=10) == INVALID  # more sequences than the cache has
    assert _append(desc=_paged(), table=None, max_ctx=128) == INVALID
    assert _append(desc=_paged(), table=FAKE, max_ctx=129) == CAP
    ring = _desc(kind=cp.CP_CACHE_ROLLING, capacity=64)
    assert _append(desc=ring, n=1, t=65, max_ctx=10 ** 6) == CAP
    assert _append(desc=ring, n=2, t=66, cu=FAKE, max_ctx=10 ** 6) == CAP  # one of them may have 65
    assert _append(qo=2 * FAKE) == INVALID and _append(qo=FAKE + 32) == INVALID
    assert _append(t=0) == cp.CP_OK


def _q4(call, desc=None, cache=None, n=4, t=8, cu=None, lens=FAKE, table=None, max_ctx=1024, x=FAKE, out=FAKE, ws=FAKE,
        ws_bytes=1 << 40):
    desc, cache = desc or _desc(), cache or _cache()
    d, c = ctypes.byref(desc), ctypes.byref(cache)
    L = cp.lib()
    if call == "append":
        return L.cp_kv_append_q4(d, x, FAKE, cu, n, t, c, lens, table, max_ctx, None, None)
    if call == "read":
        return L.cp_kv_read_q4(d, c, lens, table, cu, n, t, max_ctx, x, out, None, None)
    if call == "attn":
        return L.cp_chunk_attn_q4(d, x, c, lens, table, cu, n, t, max_ctx, out, ws, ws_bytes, 1, None, None)
    return L.cp_mixed_step_q4(d, x, FAKE, FAKE, c, table, cu, lens, n, t, max_ctx, out, ws, ws_bytes, 1, None, None)


@pytest.mark.parametrize("call", ["append", "read", "attn", "step"])
def test_q4_refusals(call):
    f = lambda **kw: _q4(call, **kw)  # noqa: E731
    assert f(desc=_desc(dtype=torch.float32)) == UNSUP
    assert f(desc=_desc(kind=cp.CP_CACHE_ROLLING)) == UNSUP
    assert f(desc=_desc(head_dim=80)) == UNSUP
    for field, _ in cp.Q4Cache._fields_:
        assert f(cache=_cache(**{field: None})) == INVALID
        assert f(cache=_cache(**{field: FAKE + 8})) == INVALID
    assert f(n=0) == INVALID and f(t=-4) == INVALID and f(n=3, t=8) == INVALID
    assert f(n=5, t=10) == INVALID
    assert f(lens=None) == INVALID
    assert f(x=FAKE + 2) == INVALID
    assert f(max_ctx=1025) == CAP and f(max_ctx=0) == INVALID
    assert f(desc=_paged(), max_ctx=128) == INVALID
    assert f(desc=_paged(), table=FAKE, max_ctx=129) == CAP
    assert f(t=0) == cp.CP_OK
    if call != "read":
        assert f(x=None) == INVALID
    if call in ("attn", "step"):
        assert f(out=None) == INVALID
        assert f(desc=_desc(num_q_heads=6, num_kv_heads=2)) == UNSUP
        assert f(desc=_desc(num_q_heads=32, num_kv_heads=1)) == UNSUP


def test_workspace_is_asked_for_and_has_to_be_there():
    d = _desc()
    need = cp.cp_workspace_size_q4(d, 8, 1024, 4)
    for call in ("attn", "step"):
        assert _q4(call, ws=None) == WS and _q4(call, ws_bytes=need - 1) == WS and _q4(call, ws=FAKE + 8) == WS
        assert _q4(call, t=4, n=2, ws_bytes=255) == WS
    # What suffices for some bounds suffices for every call within them.
    sizes = {(t, m, n): cp.cp_workspace_size_q4(d, t, m, n) for t in (1, 4, 7, 16, 700) for n in (1, 2, 4)
             for m in (1, 256, 257, 1024, 2048, 2049, 16384, 16385, 40000)}
    for (t, m, n), size in sizes.items():
        for (t2, m2, n2), size2 in sizes.items():
            assert t2 > t or m2 > m or n2 > n or size2 <= size
    for bad in (_desc(dtype=torch.float32), _desc(kind=cp.CP_CACHE_ROLLING), _desc(num_q_heads=6), _desc(head_dim=96)):
        assert cp.cp_workspace_size_q4(bad, 8, 1024, 4) == 0
    assert cp.cp_workspace_size_q4(d, 0, 1024, 4) == 0 and cp.cp_workspace_size_q4(d, 8, 0, 4) == 0
    huge = _paged(batch=0)
    assert cp.cp_workspace_size_q4(huge, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1) > 2 ** 40
    assert _q4("attn", desc=_desc(capacity=2 ** 31 - 1), max_ctx=2 ** 31 - 2) == UNSUP


def test_a_step_refuses_missing_rows_before_it_starts():
    d, c = _desc(), _cache()
    for k, v in ((None, FAKE), (FAKE, None), (FAKE + 2, FAKE)):
        assert cp.lib().cp_mixed_step_q4(ctypes.byref(d), FAKE, k, v, ctypes.byref(c), None, None, FAKE, 4, 8, 1024, FAKE,
                                         FAKE, 1 << 40, 1, None, None) == INVALID


def test_binding_refuses_tensors_that_are_not_what_the_call_takes():
    """Types, sizes and strides, checked on CPU tensors' way out: none of them reaches the library."""
    x = torch.zeros(8, 8, 128, dtype=torch.bfloat16)
    kv = torch.zeros(8, 2, 128, dtype=torch.bfloat16)
    for q, k in ((x, kv), (x.float(), kv), (x[:4], kv)):
        with pytest.raises(cp.CPError) as e:
            cp.cp_qk_norm_rope(_desc(), cp.qk_prep(0), q, k, x, kv, 1, 8)
        assert e.value.status == INVALID
    with pytest.raises(cp.CPError):
        cp.q4_cache(torch.zeros(1, 2, 16, 64, dtype=torch.uint8), torch.zeros(1, 2, 16, 64, dtype=torch.uint8),
                    torch.zeros(1, 2, 16, 4, 2, dtype=torch.bfloat16), torch.zeros(1, 2, 16, 4, 2, dtype=torch.bfloat16))


def test_store_pins():
    """Values worked out by hand."""
    x = np.zeros((1, 32), np.float32)
    x[0, :16] = np.arange(16)
    c, s, m = q4.store(x, True)
    assert s[0, 0] == 1.0 and m[0, 0] == 0.0 and c[0, :16].tolist() == list(range(16)) and not c[0, 16:].any()
    x[0, :] = -2.0
    c, s, m = q4.store(x, False)
    assert s[0, 0] == 0.0 and m[0, 0] == -2.0 and not c.any()
    x[0, 1] = -2.0 + 15 * 0.3  # the scale is cut: 0.298828125 in bf16, 0.2998046875 in fp16
    c, s, m = q4.store(x, True)
    assert s[0, 0] == 0.298828125 and c[0, 1] == 15
    x[0, 2] = -2.0 + 2.5 * 0.298828125  # ties go to the even code
    assert q4.store(x, True)[0][0, 2] == 2
    b = np.array([[0x21, 0x43, 0x65, 0x87]], np.uint8)  # a word 0x87654321
    assert q4.unpack(b)[0].tolist() == [1, 5, 2, 6, 3, 7, 4, 8]


def test_norm_rope_pins():
    x = np.zeros((2, 1, 64))
    x[:, 0, 0], x[:, 0, 1] = 3.0, 4.0
    y, _ = q4.norm_rope(x, np.ones(64), [0, 1], np.array([np.pi / 2] * 8), 16, True, 0.0)
    r = np.sqrt(25 / 64)
    assert np.allclose(y[0, 0, :2], [3 / r, 4 / r]) and np.allclose(y[1, 0, :2], [-4 / r, 3 / r])
    y, _ = q4.norm_rope(x, None, [0, 1], np.array([np.pi / 2] * 8), 16, False, 0.0)
    assert np.allclose(y[1, 0, [0, 8, 1, 9]], [0, 3, 0, 4])


HUGE_ROWS = """
import ctypes, sys
import chunked_prefill_causal_cp_gb300 as cp
d, p = cp.layer_desc(cp.CP_BF16, 1, 4, 1, 128, capacity=64), cp.qk_prep(0)
at = [i << 50 for i in range(1, 5)]
for t in (2 ** 31 - 1, 2 ** 31 - 4863, 2 ** 31 - 4864):
    s = cp.lib().cp_qk_norm_rope(ctypes.byref(d), ctypes.byref(p), at[0], 0, at[1], 0, None, None, None, at[0], None, None,
                                 1, t, at[2], at[3], None)
    assert s == cp.CP_ERR_CUDA, s
"""


def test_any_number_of_rows_is_answered_with_a_status():
    """In a process of its own, as a fault on the host would end it, and without a GPU, as its buffers are none."""
    env = {**os.environ, "CUDA_VISIBLE_DEVICES": ""}
    r = subprocess.run([sys.executable, "-c", HUGE_ROWS], env=env, cwd=os.path.dirname(os.path.dirname(__file__)),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr)


class On:
    """A CPU tensor that says it is on another device."""

    def __init__(self, t, dev):
        self.t, self.dev, self.is_cuda = t, dev, dev >= 0

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.dev


def test_a_cache_lies_on_one_device():
    codes, params = torch.zeros(1, 2, 16, 64, dtype=torch.uint8), torch.zeros(1, 2, 16, 4, 2, dtype=torch.bfloat16)
    make = lambda devs: cp.q4_cache(*(On(t.clone(), dev) for t, dev in zip((codes, codes, params, params), devs)))  # noqa: E731
    cache = make((1, 1, 1, 1))
    desc = _desc(batch=1, capacity=16)
    assert cp._q4_arg("call", desc, cache, 1)
    for dev in (0, 2, -1):
        with pytest.raises(cp.CPError):
            cp._q4_arg("call", desc, cache, dev)
    for other in range(4):
        with pytest.raises(cp.CPError) as e:
            make([0 if i == other else 1 for i in range(4)])
        assert e.value.status == INVALID


def test_without_a_tensor_among_the_rows_the_current_device_is_the_calls(monkeypatch):
    """Raw handles for the rows and tensors for the rest: those have to be where the call launches."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    assert cp._device("call", FAKE, None) == 1
    lens = torch.zeros(4, dtype=torch.int32)
    assert cp._arg("call", On(lens, 1), torch.int32, 4, cp._device("call", FAKE)) == lens.data_ptr()
    with pytest.raises(cp.CPError):
        cp._arg("call", On(lens, 0), torch.int32, 4, cp._device("call", FAKE))


def test_whole_number_arguments_lie_on_their_own_boundaries():
    """Lengths, offsets, positions, page ids and status off a 4-byte boundary: a load there would be a fault on the GPU."""
    L, odd = cp.lib(), FAKE + 2
    desc, paged, prep, cache = _desc(), _paged(), cp.qk_prep(128), _cache()
    q, k, v, qo, ko = (i * FAKE for i in range(1, 6))
    rope = dict(pos=None, lens=FAKE, cu=FAKE)
    for name in rope:
        a = {**rope, name: odd}
        assert L.cp_qk_norm_rope(ctypes.byref(desc), ctypes.byref(prep), q, 0, k, 0, None, None, FAKE, a["pos"], a["lens"],
                                 a["cu"], 4, 8, qo, ko, None) == INVALID
    full = dict(pos=FAKE, cu=FAKE, lens=FAKE, table=FAKE, status=FAKE)
    for name in full:
        a = {**full, name: odd}
        assert L.cp_qk_norm_rope_append(ctypes.byref(paged), ctypes.byref(prep), q, 0, k, 0, v, 0, None, None, FAKE, a["pos"],
                                        a["cu"], 4, 8, qo, FAKE, FAKE, a["lens"], a["table"], 128, a["status"],
                                        None) == INVALID
        if name == "pos":
            continue
        d, c, rows = ctypes.byref(paged), ctypes.byref(cache), (a["cu"], 4, 8)
        ws = (FAKE, 1 << 40, 1, a["status"], None)
        assert L.cp_kv_append_q4(d, k, v, *rows, c, a["lens"], a["table"], 128, a["status"], None) == INVALID
        assert L.cp_kv_read_q4(d, c, a["lens"], a["table"], *rows, 128, k, v, a["status"], None) == INVALID
        assert L.cp_chunk_attn_q4(d, q, c, a["lens"], a["table"], *rows, 128, qo, *ws) == INVALID
        assert L.cp_mixed_step_q4(d, q, k, v, c, a["table"], a["cu"], a["lens"], 4, 8, 128, qo, *ws) == INVALID


def test_binding_takes_what_fits_and_nothing_else():
    """Each check of a tensor by itself, on a device (-1, the CPU's) that all of them share."""
    bf16, i32 = torch.bfloat16, torch.int32
    x = torch.zeros(8, 8, 128, dtype=bf16)
    assert cp._arg("call", x, bf16, x.numel(), -1) == x.data_ptr()
    assert cp._arg("call", x, bf16, 5, -1) == x.data_ptr()  # room to spare
    assert cp._arg("call", None, bf16, 5, -1) is None and cp._arg("call", FAKE, bf16, 5, -1) == FAKE
    for bad, dtype, n, dev in ((x, i32, 8, -1), (x, bf16, x.numel() + 1, -1), (x, bf16, 8, 0), (x[:, :4], bf16, 8, -1),
                               (x.transpose(0, 1), bf16, 8, -1), (x.half(), bf16, 8, -1)):
        with pytest.raises(cp.CPError) as e:
            cp._arg("call", bad, dtype, n, dev)
        assert e.value.status == INVALID

    desc = _desc()
    rows = lambda t, n=8, heads=8, dev=-1: cp._rows_arg("call", t, desc, heads, n, dev)  # noqa: E731
    fused = torch.zeros(8, 10 * 128, dtype=bf16)
    q, k = (y.unflatten(1, (-1, 128)) for y in fused.split([8 * 128, 2 * 128], 1))
    assert rows(x) == (x.data_ptr(), 0) and rows(q) == (fused.data_ptr(), 1280)
    assert rows(k, heads=2) == (fused.data_ptr() + 2 * 1024, 1280)
    assert rows(q.unflatten(0, (2, 4))) == (fused.data_ptr(), 1280) and rows(q[:1], 1) == (fused.data_ptr(), 0)
    assert rows(q[::2], 4) == (fused.data_ptr(), 2560) and rows(q[:0], 0)[1] == 0
    assert rows(torch.zeros(8, 1, 256, dtype=bf16)[..., :128], heads=1)[1] == 256
    one = torch.zeros(1, 8, 128, dtype=bf16)
    for bad, n, heads, dev in ((x.half(), 8, 8, -1), (x, 8, 8, 0), (x, 7, 8, -1), (x, 8, 4, -1), (x.flatten(1), 8, 8, -1),
                               (x.transpose(0, 1), 8, 8, -1), (x.flatten(), 8, 8, -1), (one.expand(8, 8, 128), 8, 8, -1),
                               (torch.zeros(8, 8, 256, dtype=bf16)[..., ::2], 8, 8, -1),
                               (torch.zeros(8, 8, 256, dtype=bf16)[..., :128], 8, 8, -1),
                               (torch.zeros(3, 8, 8, 128, dtype=bf16)[:, :4][::2], 8, 8, -1)):
        with pytest.raises(cp.CPError) as e:
            rows(bad, n, heads, dev)
        assert e.value.status == INVALID

    codes, params = torch.zeros(1, 2, 16, 64, dtype=torch.uint8), torch.zeros(1, 2, 16, 4, 2, dtype=bf16)
    make = lambda kc=codes, vc=codes, kp=params, vp=params: cp.q4_cache(*(On(t, 0) for t in (kc, vc, kp, vp)))  # noqa: E731
    assert make().k_codes == codes.data_ptr()
    for kw in (dict(kc=codes.int()), dict(vp=params.float()), dict(kp=params.half()), dict(kc=codes[..., :32]),
               dict(vc=codes[:, :1]), dict(vp=params[..., :1]), dict(kp=params.transpose(1, 2)), dict(vc=codes.transpose(1, 2)),
               dict(vc=codes[:, :1], vp=params[:, :1])):
        with pytest.raises(cp.CPError) as e:
            make(**kw)
        assert e.value.status == INVALID
    cache = make()
    assert cp._q4_arg("call", _desc(batch=1, capacity=16), cache, 0)
    for desc in (_desc(batch=1, capacity=17), _desc(batch=2, capacity=16), _desc(batch=1, capacity=16, dtype=torch.float16)):
        with pytest.raises(cp.CPError) as e:
            cp._q4_arg("call", desc, cache, 0)
        assert e.value.status == INVALID
    with pytest.raises(cp.CPError):
        cp._workspace("call", torch.zeros(16, 16, dtype=torch.uint8).t()[:3], -1)
    assert cp._workspace("call", params, -1) == (params.data_ptr(), params.numel() * 2)
