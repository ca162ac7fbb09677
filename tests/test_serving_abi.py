"""Refusals of the serving operators on the host, and the binding's argument lists
(CPU only: no kernel runs)."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch

from lut_attention_b200 import axr

INV, UNS, OK = axr.AXR_EINVAL, axr.AXR_EUNSUPPORTED, axr.AXR_OK


def _buf():
    host = np.zeros(8192, np.uint8)
    return host, (host.ctypes.data + 255) // 256 * 256


def _strides(*v):
    return ctypes.addressof((ctypes.c_int64 * 8)(*v))


def test_prompt_refusals(axr_lib):
    f = axr_lib.axr_prompt_attention
    keep, p = _buf()
    st = (ctypes.c_int64 * 8)(1280, 128, 1280, 128, 1280, 128, 1280, 128)
    s = ctypes.addressof(st)

    def call(q=p, K=p, V=p, dt=2, tq=10, tk=10, cq=p, ck=p, batch=1, heads=1, group=1, d=128, strides=s, out=p, lse=p):
        return f(q, K, V, dt, tq, tk, cq, ck, batch, heads, group, d, strides, out, lse, None)

    assert call(dt=4) == INV and call(d=96) == UNS and call(d=16) == UNS and call(d=1024) == UNS
    assert call(heads=0) == INV and call(group=0) == INV and call(group=9) == UNS
    assert call(tq=-1) == INV and call(tk=-1) == INV and call(batch=-1) == INV
    assert call(tq=1 << 31) == UNS and call(heads=10000, group=8) == UNS
    assert call(tq=0, q=None) == OK and call(batch=0, q=None) == OK
    assert call(strides=None) == INV and call(q=None) == INV and call(q=p + 8) == INV
    for bad in ((1280, 64), (1281, 128), (1280, 129), (-1280, 128)):
        for at in range(4):
            v = [1280, 128] * 4
            v[2 * at:2 * at + 2] = bad
            st2 = (ctypes.c_int64 * 8)(*v)
            assert call(strides=ctypes.addressof(st2)) == INV, (bad, at)
    assert call() == INV and b"device" in axr_lib.axr_last_error()           # host memory
    del keep


def test_prompt_refuses_overlapping_rows_of_out(axr_lib):
    """out by heads, or by rows with the heads inside; anything else would be written twice."""
    f = axr_lib.axr_prompt_attention
    keep, p = _buf()

    def call(o_head, o_row, tq=10, heads=2, group=2):
        st = (ctypes.c_int64 * 8)(1280, 128, 1280, 128, 1280, 128, o_head, o_row)
        rc = f(p, p, p, 2, tq, 10, p, p, 1, heads, group, 128, ctypes.addressof(st), p, p, None)
        return rc, axr_lib.axr_last_error()

    for bad in ((0, 128), (128, 128), (128, 384), (1272, 128), (64, 512), (1 << 62, 1 << 62)):
        rc, why = call(*bad)
        assert rc == INV and b"overlap" in why, bad
    for good in ((1280, 128), (128, 512), (136, 3 * 136 + 128), (9 * 200 + 128, 200)):
        rc, why = call(*good)
        assert rc == INV and b"device" in why, good            # as far as the host memory
    assert b"device" in call(0, 128, heads=1, group=1)[1] and b"device" in call(128, 128, tq=1)[1]
    del keep


def test_prompt_refuses_more_tiles_than_a_grid(axr_lib):
    f = axr_lib.axr_prompt_attention
    keep, p = _buf()
    st = (ctypes.c_int64 * 8)(*([128, 128] * 4))
    call = lambda tq, batch, heads: f(p, p, p, 2, tq, 10, p, p, batch, heads, 1, 128, ctypes.addressof(st), p, p, None)
    most = (1 << 31) - 1
    assert call(most, most, 2) == UNS and call(most, 1, 33) == UNS and call(1 << 20, 1 << 20, 2048) == UNS
    assert call(most, most, 1) == INV and b"device" in axr_lib.axr_last_error()
    del keep


def test_shared_refusals(axr_lib):
    f, ws = axr_lib.axr_attention_shared, axr_lib.axr_attention_shared_workspace_bytes
    keep, p = _buf()
    need = ctypes.c_int64(0)
    assert ws(2, 1, 1, 128, ctypes.byref(need)) == OK and need.value > 0
    assert ws(0, 1, 1, 128, ctypes.byref(need)) == OK and need.value == 0
    assert ws(2, 1, 1, 128, None) == INV and ws(-1, 1, 1, 128, ctypes.byref(need)) == INV
    assert ws(2, 0, 1, 128, ctypes.byref(need)) == INV and ws(2, 1, 9, 128, ctypes.byref(need)) == UNS
    assert ws(2, 1, 1, 16, ctypes.byref(need)) == UNS and ws(1 << 20, 1 << 9, 8, 128, ctypes.byref(need)) == UNS

    def call(q=p, qd=2, n=10, cap=10, vd=2, batch=1, heads=1, group=1, d=128, b=4, work=p, size=1 << 40, lens=p):
        return f(q, qd, p, p, p, n, p, p, p, cap, lens, vd, batch, heads, group, d, b, p, work, size, p, p, None)

    assert call(qd=3) == INV and call(vd=-1) == INV and call(n=-1) == INV and call(cap=-1) == INV
    assert call(n=1 << 31) == UNS and call(cap=(1 << 31) - 128) == UNS
    assert call(d=100) == UNS and call(d=16) == UNS and call(b=0) == UNS and call(b=5) == UNS
    assert call(heads=0) == INV and call(group=9) == UNS and call(batch=-1) == INV
    assert call(size=8) == INV and call(q=None) == INV and call(q=p + 4) == INV
    assert call(batch=0, q=None) == OK
    assert call() == INV and b"device" in axr_lib.axr_last_error()
    del keep


def test_weights_refusals(axr_lib):
    f = axr_lib.axr_accumulate_weights
    keep, p = _buf()
    assert f(p, -1, 1, 1, None, p, 10, None) == INV and f(p, 11, 1, 1, None, p, 10, None) == INV
    assert f(p, 10, 0, 1, None, p, 10, None) == INV and f(p, 10, 1, 9, None, p, 10, None) == UNS
    assert f(p, 10, 1, 1, None, p, 1 << 31, None) == UNS
    assert f(None, 0, 1, 1, None, None, 10, None) == OK
    assert f(None, 10, 1, 1, None, p, 10, None) == INV and f(p + 2, 10, 1, 1, None, p, 10, None) == INV
    assert f(p, 10, 1, 1, None, p, 10, None) == INV and b"device" in axr_lib.axr_last_error()
    del keep


def test_evict_refusals(axr_lib):
    f = axr_lib.axr_evict
    keep_alive, p = _buf()

    def call(idx=p, vd=2, cap=100, keep=10, recent=2, heads=1, d=128, b=4, cap_out=10):
        return f(idx, p, p, vd, p, p, cap, keep, recent, heads, d, b, p, p, p, p, cap_out, p, p, None)

    assert call(vd=5) == INV and call(d=12) == UNS and call(b=0) == UNS and call(heads=0) == INV
    assert call(heads=65536) == UNS and call(cap=-1) == INV and call(cap=1 << 31) == UNS
    assert call(keep=0) == INV and call(recent=-1) == INV and call(recent=11) == INV and call(cap_out=9) == INV
    assert call(idx=None) == INV and call() == INV
    del keep_alive


class _FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            return axr.AXR_OK
        return fn


@pytest.fixture
def fake(monkeypatch):
    lib = _FakeLib()

    @contextlib.contextmanager
    def device(d):
        yield

    class _Stream:
        cuda_stream = 12345

    monkeypatch.setattr(axr, "library", lambda: lib)
    monkeypatch.setattr(axr, "_require_cuda", lambda t, name: None)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: _Stream())
    real = axr._require_rows

    def rows(t, name):
        class _Cuda:
            is_cuda = True
            shape = t.shape

            def dim(self):
                return t.dim()

            def stride(self, i):
                return t.stride(i)
        real(_Cuda(), name)

    monkeypatch.setattr(axr, "_require_rows", rows)
    return lib


def _last(lib, name, expect):
    got, args = lib.calls[-1]
    assert got == name and len(args) == len(axr.SIGNATURES[name][1]) and args[-1] == 12345
    for pos, val in expect.items():
        assert args[pos] == val, (name, pos, args[pos], val)
    return args


def test_binding_prompt(fake):
    q = torch.zeros((30, 8, 64), dtype=torch.float16).transpose(0, 1)
    K = torch.zeros((2, 50, 64), dtype=torch.float16)
    cu_q, cu_k = torch.tensor([0, 30], dtype=torch.int32), torch.tensor([0, 50], dtype=torch.int32)
    out, lse = axr.axr_prompt_attention(q, K, K, cu_q, cu_k)
    assert out.shape == q.shape and out.stride() == q.stride() and lse.shape == (8, 30)
    args = _last(fake, "axr_prompt_attention", {3: axr.AXR_F16, 4: 30, 5: 50, 8: 1, 9: 2, 10: 4, 11: 64})
    assert isinstance(args[12], int)
    with pytest.raises(ValueError):
        axr.axr_prompt_attention(q.float(), K, K, cu_q, cu_k)
    with pytest.raises(ValueError):
        axr.axr_prompt_attention(q, K, K[:, :-1], cu_q, cu_k)
    with pytest.raises(ValueError):
        axr.axr_prompt_attention(q, K, K, cu_q.long(), cu_k)
    with pytest.raises(ValueError):
        axr.axr_prompt_attention(q, K, K, cu_q, cu_k[:1])
    with pytest.raises(ValueError):
        axr.axr_prompt_attention(q[:7], K, K, cu_q, cu_k)
    with pytest.raises(ValueError):
        axr.axr_prompt_attention(q.transpose(1, 2).contiguous().transpose(1, 2), K, K, cu_q, cu_k)


def test_row_strides():
    assert axr._row_strides(torch.zeros((4, 9, 32))) == (288, 32)
    assert axr._row_strides(torch.zeros((9, 4, 32)).transpose(0, 1)) == (32, 128)
    assert axr._row_strides(torch.zeros((1, 9, 32))[:, ::3]) == (288, 96)
    assert axr._row_strides(torch.zeros((4, 1, 32))) == (32, 32)
    assert axr._row_strides(torch.zeros((4, 9, 32))[:, :1]) == (288, 32)


def _shared_args(batch=3, heads=2, group=4, n=50, cap=20, d=64, b=2):
    P = d * b // 8
    return dict(q=torch.zeros((batch * heads * group, d), dtype=torch.float16),
                prefix_idx=torch.zeros((heads, n, P), dtype=torch.uint8), prefix_norms=torch.zeros((heads, n)),
                prefix_V=torch.zeros((heads, n, d), dtype=torch.float16),
                idx=torch.zeros((batch * heads, cap, P), dtype=torch.uint8),
                norms=torch.zeros((batch * heads, cap)), V=torch.zeros((batch * heads, cap, d), dtype=torch.float16),
                lengths=torch.zeros(batch, dtype=torch.int32), group=group, b=b, signs=torch.ones(d, dtype=torch.int8))


def test_binding_shared(fake):
    a = _shared_args()
    out, lse = axr.axr_attention_shared(**a)
    assert out.dtype == torch.float16 and out.shape == a["q"].shape and lse.shape == (24,)
    _last(fake, "axr_attention_shared", {1: axr.AXR_F16, 5: 50, 9: 20, 11: axr.AXR_F16, 12: 3, 13: 2, 14: 4, 15: 64,
                                         16: 2})
    n = len(fake.calls)
    bad = dict(q=a["q"][:-1], prefix_norms=a["prefix_norms"].half(), prefix_V=a["prefix_V"].float(),
               idx=a["idx"][:, :, :-1], norms=a["norms"][:-1], V=a["V"][:, :-1], lengths=a["lengths"].long(),
               signs=a["signs"][:-1])
    for k, v in bad.items():
        with pytest.raises(ValueError):
            axr.axr_attention_shared(**{**a, k: v})
    with pytest.raises(ValueError):
        axr.axr_attention_shared(**a, out=torch.zeros(a["q"].shape))
    assert all(name.endswith("workspace_bytes") for name, _ in fake.calls[n:])


def test_binding_weights_and_evict(fake):
    scores, w = torch.zeros((8, 30)), torch.zeros((2, 40))
    assert axr.axr_accumulate_weights(scores, w, 4) is w
    _last(fake, "axr_accumulate_weights", {1: 30, 2: 2, 3: 4, 4: None, 6: 40})
    for bad in ((scores, w[:, :20], 4), (scores, w, 2), (scores.half(), w, 4)):
        with pytest.raises(ValueError):
            axr.axr_accumulate_weights(*bad)
    with pytest.raises(ValueError):
        axr.axr_accumulate_weights(scores, w, 4, lengths=torch.zeros(3, dtype=torch.int32))
    idx, V = torch.zeros((2, 40, 24), dtype=torch.uint8), torch.zeros((2, 40, 64), dtype=torch.bfloat16)
    lens = torch.zeros(2, dtype=torch.int32)
    got = axr.axr_evict(idx, w, V, w, lens, 10, 3)
    assert [tuple(t.shape) for t in got] == [(2, 10, 24), (2, 10), (2, 10, 64), (2, 10), (2, 10), (2,)]
    _last(fake, "axr_evict", {3: axr.AXR_BF16, 6: 40, 7: 10, 8: 3, 9: 2, 10: 64, 11: 3, 16: 10})
    n = len(fake.calls)
    for kw in (dict(keep=0, recent=0), dict(keep=5, recent=6), dict(keep=5, recent=-1)):
        with pytest.raises(ValueError):
            axr.axr_evict(idx, w, V, w, lens, **kw)
    for args in ((idx[:, :, :23], w, V, w, lens), (idx, w[:1], V, w, lens), (idx, w, V, w, lens[:1]),
                 (idx, w, V.to(torch.int16), w, lens)):
        with pytest.raises(ValueError):
            axr.axr_evict(*args, 10, 3)
    with pytest.raises(ValueError):
        axr.axr_evict(idx, w, V, w, lens, 11, 3, out=got)
    assert len(fake.calls) == n


def test_binding_refuses_cpu_tensors():
    q = torch.zeros((2, 4, 64))
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        axr.axr_prompt_attention(q, q, q, cu)
    with pytest.raises(ValueError, match="CUDA"):
        axr.axr_attention_shared(**_shared_args())
    with pytest.raises(ValueError, match="CUDA"):
        axr.axr_accumulate_weights(torch.zeros((1, 4)), torch.zeros((1, 4)), 1)
