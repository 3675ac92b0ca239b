"""The routed-expert entry points refuse bad calls on the host, before anything is enqueued."""
import ctypes

import pytest
import torch

from sparse_mla_decode_front_b200 import _lib, experts

P = [ctypes.c_void_p(0x1000 + 256 * i) for i in range(8)]
ODD = ctypes.c_void_p(0x1008)
SKEW = ctypes.c_void_p(0x1002)
WS = ctypes.c_void_p(0x100000)


def test_sort_workspace():
    l = _lib.lib()
    assert l.mla_moe_sort_workspace_bytes(128, 8, 256) == 0            # one launch, no workspace
    assert l.mla_moe_sort_workspace_bytes(512, 8, 256) == 0
    assert l.mla_moe_sort_workspace_bytes(513, 8, 256) == 4 * 2 * 257
    # at most 256 chunks, whatever the length
    assert l.mla_moe_sort_workspace_bytes((1 << 30) // 8, 8, 32) <= 4 * 256 * 33
    for bad in [(-1, 8, 256), (4, 0, 256), (4, 33, 256), (4, 8, 0), (4, 8, 1025), (1 << 28, 8, 256)]:
        assert l.mla_moe_sort_workspace_bytes(*bad) == 0, bad


def test_sort_rejections():
    def call(idx=P[0], aff=None, T=4, K=2, total=0, first=0, E=8, norm=0, scale=1.0, off=P[1], row=P[2], src=P[3],
             w=None, ws=None, nws=0):
        return _lib.lib().mla_moe_sort(idx, aff, T, K, total, first, E, norm, ctypes.c_float(scale), off, row, src, w,
                                       ws, nws, None)
    assert call(T=-1) == call(K=0) == call(E=0) == call(first=-1) == call(aff=P[4], w=P[5], total=0) \
        == _lib.MLA_ERR_BAD_DIMS
    assert call(K=33) == call(E=1025) == call(T=1 << 29, K=8) == _lib.MLA_ERR_UNSUPPORTED_DIMS
    assert call(scale=float("nan")) == call(scale=float("inf")) == call(norm=2) == _lib.MLA_ERR_BAD_ARGUMENT
    for k in ("idx", "off", "row", "src"):
        assert call(**{k: None}) == _lib.MLA_ERR_NULL_POINTER, k
        assert call(**{k: SKEW}) == _lib.MLA_ERR_MISALIGNED, k
    assert call(aff=P[4], total=8) == call(w=P[4]) == _lib.MLA_ERR_NULL_POINTER
    assert call(aff=ODD, w=P[4], total=8) == call(aff=P[4], w=SKEW, total=8) == _lib.MLA_ERR_MISALIGNED
    assert call(T=4096) == _lib.MLA_ERR_NULL_POINTER                   # the chunked form needs a workspace
    assert call(T=4096, ws=P[6], nws=16) == _lib.MLA_ERR_WORKSPACE_TOO_SMALL
    assert call(T=4096, ws=ODD, nws=1 << 20) == _lib.MLA_ERR_MISALIGNED


def test_row_mover_rejections():
    l = _lib.lib()

    def gather(x=P[0], dtype=0, row=P[1], T=4, K=2, H=64, R=8, rows=P[2], sc=None):
        return l.mla_moe_gather(x, dtype, row, T, K, H, R, rows, sc, None)

    def combine(rows=P[0], dtype=0, row=P[1], w=P[2], T=4, K=2, H=64, R=8, out=P[3]):
        return l.mla_moe_combine(rows, dtype, row, w, T, K, H, R, out, None)

    def back(g=P[0], rows=P[1], dtype=0, row=P[2], w=P[3], T=4, K=2, H=64, R=8, gr=P[4], gw=P[5]):
        return l.mla_moe_combine_backward(g, rows, dtype, row, w, T, K, H, R, gr, gw, None)

    for f in (gather, combine, back):
        assert f(T=-1) == f(K=0) == f(H=0) == f(R=-1) == _lib.MLA_ERR_BAD_DIMS
        assert f(dtype=3) == f(dtype=-1) == _lib.MLA_ERR_BAD_ARGUMENT
        assert f(K=33) == f(H=24) == _lib.MLA_ERR_UNSUPPORTED_DIMS
        assert f(T=1 << 26, H=1 << 20) == _lib.MLA_ERR_UNSUPPORTED_DIMS
        assert f(T=0) == _lib.MLA_OK
        assert f(row=None) == _lib.MLA_ERR_NULL_POINTER and f(row=SKEW) == _lib.MLA_ERR_MISALIGNED
        assert f(rows=None) == _lib.MLA_ERR_NULL_POINTER and f(rows=ODD) == _lib.MLA_ERR_MISALIGNED
    assert gather(x=None) == combine(out=None) == back(g=None) == back(gr=None, gw=None) == _lib.MLA_ERR_NULL_POINTER
    assert gather(x=ODD) == gather(sc=SKEW) == combine(out=ODD) == combine(w=SKEW) == back(g=ODD) == back(gr=ODD) \
        == back(gw=SKEW) == back(w=SKEW) == _lib.MLA_ERR_MISALIGNED
    assert gather(R=0) == _lib.MLA_OK


def test_quantize_rejections():
    def call(x=P[0], dtype=0, R=4, C=64, gated=0, valid=None, q=P[1], sc=P[2]):
        return _lib.lib().mla_fp8_quantize(x, dtype, R, C, gated, valid, q, sc, None)
    assert call(R=-1) == call(C=0) == _lib.MLA_ERR_BAD_DIMS
    assert call(dtype=5) == call(gated=2) == _lib.MLA_ERR_BAD_ARGUMENT
    assert call(C=24) == call(C=1 << 30) == _lib.MLA_ERR_UNSUPPORTED_DIMS
    assert call(R=0) == _lib.MLA_OK
    assert call(x=None) == call(q=None) == call(sc=None) == _lib.MLA_ERR_NULL_POINTER
    assert call(x=ODD) == call(q=ODD) == call(sc=SKEW) == call(valid=SKEW) == _lib.MLA_ERR_MISALIGNED


@pytest.mark.parametrize("grouped", [False, True])
def test_product_rejections(grouped):
    def call(x=P[0], xs=P[1], w=P[2], ws=P[3], off=P[4], M=4, E=2, N=64, K=64, out=P[5], dtype=0, st=None):
        l = _lib.lib()
        if grouped:
            return l.mla_fp8_grouped_matmul(x, xs, w, ws, off, M, E, N, K, out, dtype, st, None)
        return l.mla_fp8_matmul(x, xs, w, ws, M, N, K, out, dtype, st, None)
    assert call(M=-1) == call(N=0) == call(K=0) == _lib.MLA_ERR_BAD_DIMS
    assert call(dtype=3) == _lib.MLA_ERR_BAD_ARGUMENT
    assert call(N=24) == call(K=24) == call(M=(1 << 31) - 1, N=(1 << 31) - 16) == _lib.MLA_ERR_UNSUPPORTED_DIMS
    assert call(M=0) == _lib.MLA_OK
    for k in ("x", "w", "out"):
        assert call(**{k: None}) == _lib.MLA_ERR_NULL_POINTER, k
        assert call(**{k: ODD}) == _lib.MLA_ERR_MISALIGNED, k
    for k in ("xs", "ws"):
        assert call(**{k: None}) == _lib.MLA_ERR_NULL_POINTER, k
        assert call(**{k: SKEW}) == _lib.MLA_ERR_MISALIGNED, k
    assert call(st=SKEW) == _lib.MLA_ERR_MISALIGNED
    if grouped:
        assert call(E=0) == _lib.MLA_ERR_BAD_DIMS
        assert call(E=1025) == call(E=1024, N=1 << 22) == _lib.MLA_ERR_UNSUPPORTED_DIMS
        assert call(off=None) == _lib.MLA_ERR_NULL_POINTER and call(off=SKEW) == _lib.MLA_ERR_MISALIGNED


def test_binding_refuses_host_tensors_and_missing_arguments():
    t = torch.zeros(2, 16)
    for call in (lambda: experts.mla_moe_sort(t, t, t, t), lambda: experts.mla_moe_gather(t, t, t),
                 lambda: experts.mla_moe_combine(t, t, None, t), lambda: experts.mla_fp8_quantize(t, t, t),
                 lambda: experts.mla_moe_combine_backward(t, t, t, None, t, None),
                 lambda: experts.mla_fp8_matmul(t, t, t, t, t)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="None"):
        experts.mla_moe_gather(None, t, t)
    with pytest.raises(ValueError, match="list"):
        experts.mla_moe_combine([1.0], t, None, t)
    with pytest.raises(ValueError, match="2 dimensions"):
        experts.mla_fp8_matmul(t[0], t, t, t, t)


def test_missing_native_binding_fails_loudly(monkeypatch):
    """Without the built library or the native checks every call raises; there is no other path."""
    import sys
    monkeypatch.setattr(experts, "_bound", None)
    monkeypatch.setitem(sys.modules, "sparse_mla_decode_front_b200._bind", None)
    import sparse_mla_decode_front_b200 as pkg
    monkeypatch.delattr(pkg, "_bind", raising=False)
    t = torch.zeros(2, 16)
    with pytest.raises(ImportError, match="_bind"):
        experts.mla_moe_gather(t, t, t)
