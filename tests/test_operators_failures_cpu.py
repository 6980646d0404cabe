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
