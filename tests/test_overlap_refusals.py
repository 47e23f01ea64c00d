"""Buffers that must not overlap: refused on the host, before anything is launched.  No GPU is needed."""
import ctypes

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


@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_few(B, dtype):
    """Every output over the first and the last bytes of every other buffer."""
    T, H, E, k, I = 4, 512, 64, 4, 256
    c = B.MoeConfig(T=T, H=H, E=E, k=k, I=I, n_shared=1, dtype=dtype)
    per = {0: 2.0, 1: 1.0, 2: 0.5}[dtype]
    block = {0: 0.0, 1: 4.0 / 128 ** 2, 2: 1.0 / 32}[dtype]
    size = {"x": T * H * 2, "w_router": E * H * 2, "bias": E * 4}
    for name, n in (("w13", E * 2 * I * H), ("w2", E * H * I), ("w13s", 2 * I * H), ("w2s", H * I)):
        size[name], size["s" + name] = int(n * per), int(n * block)
    size.update(out=T * H * 2, idx=T * k * 4, w=T * k * 4, ws=B.few_workspace_size(c))
    order = ["x", "w_router", "bias", "w13", "sw13", "w2", "sw2", "w13s", "sw13s", "w2s", "sw2s", "out", "idx",
             "w", "ws"]
    base, at = {}, 1 << 30
    for name in order:
        base[name] = at if size[name] else None
        at += (size[name] + 2 * MB) // MB * MB
    cc = c.c()

    def call(**over):
        a = {**base, **over}
        return B.lib().moe_forward_few(ctypes.byref(cc), *[a[n] for n in order], size["ws"], None)

    words = {"out": "out", "idx": "topk_idx", "w": "topk_w", "ws": "workspace"}
    for o in words:
        align = {"out": 16, "idx": 4, "w": 4, "ws": 256}[o]
        for other in order:
            if other == o or not size[other]:
                continue
            spots = {base[other], (base[other] + size[other] - 1) // align * align}
            spots.add(base[other] - (size[o] - 1) // align * align)
            if o == "out" and other == "x":
                spots.discard(base["x"])            # out may be x
            for p in spots:
                s = call(**{o: p})
                assert refused(B, s) and any(w in B.get_last_error() for w in (words[o], words.get(other, "?"))), \
                    (o, other, p - base[other], B.get_last_error())
