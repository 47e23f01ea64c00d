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


def every_overlap(B, call, base, size, aligns, may):
    """Each output (aligns: its alignment) over the ends of each other buffer, but for where it may start."""
    for o, align in aligns.items():
        for other in base:
            if other == o or base[other] is None or base[o] is None:
                continue
            spots = {base[other], (base[other] + size[other] - 1) // align * align,
                     base[other] - (size[o] - 1) // align * align}
            if may.get(o) == other:
                spots.discard(base[other])
            for p in spots:
                assert refused(B, call(**{o: p})), (o, other, p - base[other], B.get_last_error())


def place(size):
    base, at = {}, 1 << 30
    for name, n in size.items():
        base[name] = at if n else None
        at += (n + 2 * MB) // MB * MB
    return base


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("pre", [True, False])
def test_norms(B, mode, pre):
    T, H = 6, 512
    n, row, fp = T * H * 2, H * 2, H * 4
    c = B.MoeConfig(T=T, H=H, E=32, k=1, I=128)
    cc = c.c()
    gate = {0: 0, 1: row, 2: n}[mode]
    rstd = T * (8 if pre else 4)
    size = dict(h=n, y=n, gamma_post=row, gate=gate, gamma_pre=row * pre, h_out=n, u=n * pre, rstd=rstd)
    base = place(size)

    def forward(**over):
        a = {**base, **over}
        return B.lib().moe_norm_residual(ctypes.byref(cc), a["h"], a["y"], a["gamma_post"], a["gate"], mode, 1.0,
                                         1e-6, a["gamma_pre"], a["h_out"], a["u"], a["rstd"], None)

    every_overlap(B, forward, base, size, {"h_out": 16, "u": 16, "rstd": 4}, {"h_out": "h", "u": "y"})
    size = dict(h=n, y=n, gamma_post=row, gate=gate, gamma_pre=row * pre, rstd=rstd, dh_out=n, du=n * pre, dh=n,
                dy=n, dgate={0: 0, 1: fp, 2: n}[mode], dgamma_post=fp, dgamma_pre=fp * pre,
                ws=B.norm_residual_workspace_size(c))
    base2 = place(size)

    def backward(**over):
        a = {**base2, **over}
        return B.lib().moe_norm_residual_backward(
            ctypes.byref(cc), a["h"], a["y"], a["gamma_post"], a["gate"], mode, 1.0, a["gamma_pre"], a["rstd"],
            a["dh_out"], a["du"], a["dh"], a["dy"], a["dgate"], a["dgamma_post"], a["dgamma_pre"], a["ws"],
            size["ws"], None)

    may = {"dh": "dh_out", "dy": "du"}
    if mode == 2:
        may["dgate"] = "gate"
    every_overlap(B, backward, base2, size, {"dh": 16, "dy": 16, "dgate": 16, "dgamma_post": 16, "dgamma_pre": 16,
                                             "ws": 256}, may)
