"""How the operators around the layer refuse and fail, as far as it needs no GPU."""
import ctypes

import decode_moe_layer_b200 as moe

P = ctypes.c_void_p
INV, UNS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED_SHAPE


def test_norm_selftest_refusals():
    def call(x=0x1000000, w=0x3000000, h=0x4000000, M=592, H=512):
        n = lambda v: P(v) if v else None  # noqa: E731
        return moe.load().moe_selftest_norm_timeout(n(x), None, None, n(w), None, n(h), None, None, M, H, None)

    assert call(M=0) == INV and call(M=-1) == INV and call(H=0) == INV
    assert call(M=591) == UNS and call(M=148, H=8192) == UNS and call(H=516) == UNS
    assert call(x=0) == INV and call(w=0) == INV and call(h=0) == INV and call(h=0x1000010) == INV


def test_product_selftest_refusals():
    n = lambda v: P(v) if v else None  # noqa: E731

    def call(int8=0, x=0x1000000, off=0x5000000, y=0x4000000, st=0x6000000, M=64, N=512, K=1024, E=4):
        return moe.load().moe_selftest_product_timeout(int8, n(x), n(0x7000000), n(0x10000000), n(0x8000000), n(off), None,
                                                       n(y), 0, 0, M, N, K, E, 1, n(st), None)

    for int8 in (0, 1):
        assert call(int8, M=0) == INV and call(int8, st=0) == INV and call(int8, x=0) == INV and call(int8, y=0) == INV
        assert call(int8, st=0x4000000) == INV and call(int8, K=1020) == UNS
        assert call(int8, M=4, E=64) == UNS            # by rows: nothing is waited for
    assert call(0, off=0) == INV and call(0, M=64, E=96) == UNS
