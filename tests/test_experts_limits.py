"""The size limits that include/moe_experts.h documents: refused just past them, taken at them (with no rows,
so that nothing is launched)."""
import ctypes

from sparse_mla_decode_front_b200 import _lib

P = [ctypes.c_void_p(0x1000 + 256 * i) for i in range(6)]


def quantize(R, C):
    return _lib.lib().mla_fp8_quantize(P[0], 0, R, C, 0, None, P[1], P[2], None)


def gather(T, H):
    return _lib.lib().mla_moe_gather(P[0], 0, P[1], T, 1, H, 8, P[2], None, None)


def product(M, N, K=64, E=None):
    l = _lib.lib()
    if E is None:
        return l.mla_fp8_matmul(*P[:4], M, N, K, P[5], 0, None, None)
    return l.mla_fp8_grouped_matmul(*P[:5], M, E, N, K, P[5], 0, None, None)


def test_row_movers():
    assert quantize(0, 1 << 29) == gather(0, 1 << 30) == _lib.MLA_OK
    assert quantize(0, (1 << 29) + 16) == gather(0, (1 << 30) + 16) == _lib.MLA_ERR_UNSUPPORTED_DIMS
    # rows x width past 2^42 - 2048, the width counted up to a multiple of 512
    assert quantize(1 << 20, 1 << 22) == quantize(1 << 20, (1 << 22) - 496) == _lib.MLA_ERR_UNSUPPORTED_DIMS
    assert gather(1 << 20, 1 << 22) == gather(1 << 20, (1 << 22) - 496) == _lib.MLA_ERR_UNSUPPORTED_DIMS


def test_products():
    assert product(0, 1 << 30) == product(0, 64, 1 << 30) == product(0, (1 << 21) - 16, E=1024) == _lib.MLA_OK
    assert product(0, (1 << 30) + 16) == product(0, 64, (1 << 30) + 16) == product((1 << 30) + 1, 64) \
        == product(0, 1 << 21, E=1024) == _lib.MLA_ERR_UNSUPPORTED_DIMS
    # (rows / 16 + experts) * ceil(n / 128) reaches 2^30
    assert product(1 << 30, 2048) == product((1 << 24) - 16 * 512, 1 << 17, E=512) == _lib.MLA_ERR_UNSUPPORTED_DIMS


def test_gradient_of_no_rows():
    # an empty tensor has no address: with no rows there is no grad_rows to write, given or not
    def back(R, grad_rows, grad_weights=None):
        return _lib.lib().mla_moe_combine_backward(P[0], None, 0, P[1], P[2], 4, 2, 64, R, grad_rows, grad_weights,
                                                   None)
    assert back(0, P[3]) == back(0, None) == _lib.MLA_OK
    assert back(8, None) == _lib.MLA_ERR_NULL_POINTER
