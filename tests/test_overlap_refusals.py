"""Buffers that must not overlap: refused on the host, before anything is launched.  No GPU is needed."""
import pytest

MB = 1 << 20


@pytest.fixture(scope="module")
def B():
    from sigmoid_top_routing_warp_b200 import build
    build.build()
    from sigmoid_top_routing_warp_b200 import binding
    return binding


def refused(B, status, *words):
    return status == B.MOE_ERR_INVALID_ARG and all(w in B.get_last_error() for w in ("overlap",) + words)


def test_mx(B):
    """x is 64 KB, q 16 KB, scale 1 KB."""
    L, rows, cols = B.lib(), 64, 512
    x, q, s = 1 * MB, 2 * MB, 3 * MB
    for call in (lambda x, q, s: L.moe_quantize_mx(x, rows, cols, q, s, None),
                 lambda x, q, s: L.moe_dequantize_mx(q, s, rows, cols, x, None)):
        assert refused(B, call(x, x, s), "x", "q")
        assert refused(B, call(x, x + 65536 - 16, s), "x", "q")
        assert refused(B, call(x, x - 16384 + 16, s), "x", "q")
        assert refused(B, call(x, q, x + 65535), "x", "scale")
        assert refused(B, call(x, q, q + 16383), "q", "scale")
        assert refused(B, call(x, q, q - 1023), "q", "scale")
