"""Host side of the few-token layer, MXFP4 and the norms around a block: what
their calls refuse (before anything is launched), and the 64-bit references
against plain cases and differences.  No GPU is needed."""
import ctypes
import math

import pytest
import torch

from oracle import few as F

EPS = 1e-6
WS = 1 << 20     # aligned, never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def B():
    from sigmoid_top_routing_warp_b200 import build
    build.build()
    from sigmoid_top_routing_warp_b200 import binding
    return binding


def cfg(B, **kw):
    base = dict(T=4, H=512, E=64, k=4, I=256, n_shared=1)
    base.update(kw)
    return B.MoeConfig(**base)


# ---------------------------------------------------------------- few-token layer
def few(B, c, ws_bytes=None, **kw):
    """Status of moe_forward_few with plausible fake pointers, some replaced."""
    a = dict(x=16, w_router=16, bias=16, w13=16, s13=None, w2=16, s2=None, w13s=16, s13s=None, w2s=16,
             s2s=None, out=16, idx=None, w=None, ws=WS)
    a.update(kw)
    cc = c.c()
    n = B.few_workspace_size(c) if ws_bytes is None else ws_bytes
    return B.lib().moe_forward_few(ctypes.byref(cc), *list(a.values())[:14], a["ws"], n, None)


def test_few_workspace(B):
    n = B.few_workspace_size(cfg(B))
    assert n > 256 and B.few_workspace_size(cfg(B, T=16)) > n
    for dt in (B.MOE_DTYPE_BF16, B.MOE_DTYPE_FP8_E4M3_BLOCK128, B.MOE_DTYPE_MXFP4_BLOCK32):
        assert B.few_workspace_size(cfg(B, dtype=dt)) == n


@pytest.mark.parametrize("kw", [dict(T=17), dict(T=-1), dict(H=100), dict(E=33), dict(I=100), dict(k=0),
                                dict(k=33), dict(dtype=3), dict(n_group=3), dict(n_shared=-1),
                                dict(flags=0x80)])
def test_few_refuses_configurations(B, kw):
    c = cfg(B, **kw)
    with pytest.raises(B.MoeError):
        B.few_workspace_size(c)
    assert few(B, c, ws_bytes=1 << 30) != B.MOE_OK and B.get_last_error() != ""


@pytest.mark.parametrize("name", ["x", "w_router", "bias", "w13", "w2", "w13s", "w2s", "out", "ws"])
def test_few_refuses_pointers(B, name):
    c = cfg(B)
    word = "workspace" if name == "ws" else name
    assert few(B, c, **{name: None}) == B.MOE_ERR_INVALID_ARG and word in B.get_last_error()
    if name != "ws":
        odd = 18 if name != "bias" else 17
        assert few(B, c, **{name: odd}) == B.MOE_ERR_INVALID_ARG and "aligned" in B.get_last_error()
    else:
        assert few(B, c, ws=WS + 16) == B.MOE_ERR_INVALID_ARG and "aligned" in B.get_last_error()


def test_few_refuses_scales_and_small_workspaces(B):
    c = cfg(B)
    assert few(B, c, s13=16) == B.MOE_ERR_INVALID_ARG and "scale" in B.get_last_error()
    assert few(B, c, ws_bytes=B.few_workspace_size(c) - 1) == B.MOE_ERR_WORKSPACE
    for dt in (B.MOE_DTYPE_FP8_E4M3_BLOCK128, B.MOE_DTYPE_MXFP4_BLOCK32):
        q = cfg(B, dtype=dt)
        scales = dict(s13=16, s2=16, s13s=16, s2s=16)
        for name in scales:
            bad = dict(scales)
            bad[name] = None
            assert few(B, q, **bad) == B.MOE_ERR_INVALID_ARG and "scale" in B.get_last_error()
            bad[name] = 18
            assert few(B, q, **bad) == B.MOE_ERR_INVALID_ARG and "aligned" in B.get_last_error()
    # out over x is allowed, over a part of it refused
    assert few(B, c, x=4096, out=4096 + 16) == B.MOE_ERR_INVALID_ARG and "overlap" in B.get_last_error()
    assert few(B, c, x=4096 + 32, out=4096) == B.MOE_ERR_INVALID_ARG and "overlap" in B.get_last_error()
    # no tokens: nothing to do, nothing is looked at
    assert few(B, cfg(B, T=0), ws_bytes=0, x=None, out=None, ws=None) == B.MOE_OK


def test_other_calls_refuse_mxfp4(B):
    c = cfg(B, dtype=B.MOE_DTYPE_MXFP4_BLOCK32)
    with pytest.raises(B.MoeError):
        B.workspace_size(c)
    with pytest.raises(B.MoeError):
        B.backward_workspace_size(c)


def test_binding_looks_its_tensors_over(B):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    q = torch.zeros((4, 32), dtype=torch.uint8)
    s = torch.zeros((4, 2), dtype=torch.uint8)
    with pytest.raises(TypeError, match="x must be"):
        B.moe_quantize_mx(x.float(), q, s)
    with pytest.raises(ValueError, match="dense"):
        B.moe_quantize_mx(torch.zeros((64, 4), dtype=torch.bfloat16).t(), q, s)
    with pytest.raises(ValueError, match="elements"):
        B.moe_norm_residual(cfg(B, T=4, H=128), x, x, x[0], x, EPS)
    with pytest.raises(ValueError, match="current CUDA device"):
        B.moe_quantize_mx(x, q, s)


# ---------------------------------------------------------------- MXFP4
def test_mx_refusals(B):
    L = B.lib()
    for f in (lambda x, r, c, q, s: L.moe_quantize_mx(x, r, c, q, s, None),
              lambda x, r, c, q, s: L.moe_dequantize_mx(q, s, r, c, x, None)):
        assert f(16, -1, 32, 16, 16) == B.MOE_ERR_INVALID_ARG
        assert f(16, 1, 33, 16, 16) == B.MOE_ERR_INVALID_ARG
        assert f(16, 1, -32, 16, 16) == B.MOE_ERR_INVALID_ARG
        for bad in ((None, 16, 16), (16, None, 16), (16, 16, None), (8, 16, 16), (16, 8, 16)):
            assert f(bad[0], 1, 32, bad[1], bad[2]) == B.MOE_ERR_INVALID_ARG
            assert B.get_last_error() != ""
        assert f(None, 0, 32, None, None) == B.MOE_OK and f(None, 7, 0, None, None) == B.MOE_OK


def test_mx_reference():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    x[0, :8] = torch.tensor([6.0, -6.0, 7.0, 0.3, -0.25, 2.6, 4.9, 1.0])
    x[1, 32] = 2.0 ** -130
    x[1, 0] = math.inf
    q, s = F.mx_quantize(x)
    v = F.mx_values(q, s)
    assert s.tolist() == [[127, 127], [255, 0]]
    assert v[0, :8].tolist() == [6.0, -6.0, 6.0, 0.5, -0.0, 3.0, 4.0, 1.0]
    assert bool(v[1, :32].isnan().all()) and float(v[1, 32]) == 0.0


# ---------------------------------------------------------------- norms around a block
def norm(B, c, mode=0, a=1.0, eps=EPS, **kw):
    p = dict(h=4096, y=8192, gamma_post=16, gate=None, gamma_pre=16, h_out=4096, u=1 << 16, rstd=None)
    p.update(kw)
    cc = c.c()
    return B.lib().moe_norm_residual(ctypes.byref(cc), p["h"], p["y"], p["gamma_post"], p["gate"], mode, a,
                                     eps, p["gamma_pre"], p["h_out"], p["u"], p["rstd"], None)


def norm_bwd(B, c, mode=0, a=1.0, ws_bytes=None, **kw):
    p = dict(h=16, y=16, gamma_post=16, gate=None, gamma_pre=16, rstd=16, dh_out=4096, du=8192,
             dh=1 << 16, dy=1 << 17, dgate=None, dgamma_post=16, dgamma_pre=16, ws=WS)
    p.update(kw)
    cc = c.c()
    n = B.norm_residual_workspace_size(c) if ws_bytes is None else ws_bytes
    return B.lib().moe_norm_residual_backward(
        ctypes.byref(cc), p["h"], p["y"], p["gamma_post"], p["gate"], mode, a, p["gamma_pre"], p["rstd"],
        p["dh_out"], p["du"], p["dh"], p["dy"], p["dgate"], p["dgamma_post"], p["dgamma_pre"], p["ws"], n,
        None)


def test_norm_refusals(B):
    c = cfg(B, H=64)
    bad = B.MOE_ERR_INVALID_ARG
    for name in ("h", "y", "gamma_post", "h_out"):
        assert norm(B, c, **{name: None}) == bad and name in B.get_last_error()
        assert norm(B, c, **{name: 8}) == bad and "aligned" in B.get_last_error()
    assert norm(B, c, gamma_pre=None) == bad and norm(B, c, u=None) == bad
    assert norm(B, c, u=4096) == bad                              # u over h
    assert norm(B, c, u=4096 + 64) == bad                         # u inside h
    assert norm(B, c, h_out=4096 + 128) == bad                    # h_out shifted against h
    assert norm(B, c, h_out=8192) == bad                          # h_out over y
    assert norm(B, c, u=8192 + 16) == bad                         # u shifted against y
    assert norm(B, c, mode=3) == bad and norm(B, c, mode=-1) == bad
    assert norm(B, c, gate=16) == bad and norm(B, c, mode=1) == bad and norm(B, c, mode=2) == bad
    for v in (math.nan, math.inf):
        assert norm(B, c, a=v) == bad
    for v in (math.nan, math.inf, -1.0):
        assert norm(B, c, eps=v) == bad
    for h in (0, 4, 16392):
        assert norm(B, cfg(B, H=h)) == B.MOE_ERR_UNSUPPORTED
    assert norm(B, cfg(B, T=-1)) == bad
    assert norm(B, cfg(B, T=0, H=64), h=None, y=None, h_out=None, u=None) == B.MOE_OK


def test_norm_backward_refusals(B):
    c = cfg(B, H=64)
    bad = B.MOE_ERR_INVALID_ARG
    for name in ("h", "y", "gamma_post", "rstd", "dh_out", "du", "dh", "dy", "gamma_pre", "dgamma_post",
                 "dgamma_pre", "ws"):
        assert norm_bwd(B, c, **{name: None}) == bad and B.get_last_error() != ""
        assert norm_bwd(B, c, **{name: 18}) == bad or name == "rstd"
    assert norm_bwd(B, c, rstd=18) == bad and "aligned" in B.get_last_error()
    assert norm_bwd(B, c, dgate=16) == bad
    assert norm_bwd(B, c, mode=1, gate=16) == bad and "dgate" in B.get_last_error()
    assert norm_bwd(B, c, dh=16) == bad                           # dh over h
    assert norm_bwd(B, c, dh=4096 + 64) == bad                    # shifted against dh_out
    assert norm_bwd(B, c, dy=4096) == bad                         # dy over dh_out
    assert norm_bwd(B, c, dy=(1 << 16) + 32) == bad               # dy inside dh
    assert norm_bwd(B, c, ws_bytes=B.norm_residual_workspace_size(c) - 1) == B.MOE_ERR_WORKSPACE
    for h in (0, 4, 16392):
        with pytest.raises(B.MoeError):
            B.norm_residual_workspace_size(cfg(B, H=h))


def test_reference_gradients_match_differences():
    """The reference's gradients against central differences of the reference's forward pass."""
    torch.manual_seed(0)
    T, H, a = 3, 24, 0.8
    h, y, do, du = (torch.randn(T, H, dtype=torch.float64) for _ in range(4))
    gp, gq = (1 + 0.1 * torch.randn(H, dtype=torch.float64) for _ in range(2))
    gate = torch.rand(1, H, dtype=torch.float64)

    def loss():
        o = F.norm_residual(h, y, gp, gate, a, EPS, gq)
        return float((o["h_out"] * do).sum() + (o["u"] * du).sum())

    o = F.norm_residual(h, y, gp, gate, a, EPS, gq)
    g = F.norm_residual_backward(h, y, gp, gate, a, gq, o["rp"], o["rq"], do, du)
    grads = {"dh": h, "dy": y, "dgamma_post": gp, "dgamma_pre": gq, "dgate": gate}
    for name, var in grads.items():
        ref = g[name][0].sum(0, keepdim=True) if name == "dgate" else g[name][0]
        flat, rf = var.view(-1), ref.reshape(-1)
        for i in range(0, flat.numel(), 5):
            v0, step = float(flat[i]), 1e-5
            flat[i] = v0 + step
            up = loss()
            flat[i] = v0 - step
            down = loss()
            flat[i] = v0
            assert abs((up - down) / (2 * step) - float(rf[i])) <= 1e-6 * (1 + abs(float(rf[i])))
