"""The norms around a block with gate and residual scale, and their gradients,
against the 64-bit reference with its derived bounds."""
import math

import pytest
import torch

from oracle import few as F

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def B():
    from sigmoid_top_routing_warp_b200 import binding
    return binding


MODES = ("none", "channel", "token")


def mode_of(B, gate):
    return {"none": B.MOE_GATE_NONE, "channel": B.MOE_GATE_CHANNEL, "token": B.MOE_GATE_TOKEN}[gate]


def make(T, H, gate, pre, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * T + H)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    d = {"h": r(T, H) * 2.0, "y": r(T, H) * 0.5, "gamma_post": 1.0 + 0.1 * r(H),
         "gate": None if gate == "none" else torch.sigmoid(r(H) if gate == "channel" else r(T, H)),
         "gamma_pre": 1.0 + 0.1 * r(H) if pre else None, "dh_out": r(T, H),
         "du": r(T, H) if pre else None}
    return {n: None if v is None else v.to(torch.bfloat16) for n, v in d.items()}


def f64(d):
    return {n: None if v is None else v.cpu().double() for n, v in d.items()}


def cfg_of(B, T, H):
    return B.MoeConfig(T=T, H=H, E=32, k=1, I=128)


def forward(B, d, T, H, gate, a, h_out=None, u=None, stream=None, eps=EPS):
    h_out = torch.empty_like(d["h"]) if h_out is None else h_out
    pre = d["gamma_pre"] is not None
    u = (torch.empty_like(d["h"]) if u is None else u) if pre else None
    rstd = torch.full((2, T), math.nan, device="cuda")
    B.moe_norm_residual(cfg_of(B, T, H), d["h"], d["y"], d["gamma_post"], h_out, eps, gate=d["gate"],
                        gate_mode=mode_of(B, gate), res_scale=a, gamma_pre=d["gamma_pre"], u=u,
                        rstd=rstd, stream=stream)
    return h_out, u, rstd


def backward(B, d, T, H, gate, a, rstd, dh=None, dy=None, stream=None, ws=None):
    cfg = cfg_of(B, T, H)
    pre = d["gamma_pre"] is not None
    o = {"dh": torch.empty_like(d["h"]) if dh is None else dh,
         "dy": torch.empty_like(d["h"]) if dy is None else dy,
         "dgamma_post": torch.full((H,), math.nan, device="cuda"),
         "dgamma_pre": torch.full((H,), math.nan, device="cuda") if pre else None,
         "dgate": None if gate == "none" else torch.full((H,), math.nan, device="cuda")
         if gate == "channel" else torch.empty_like(d["h"])}
    B.moe_norm_residual_backward(cfg, d["h"], d["y"], d["gamma_post"], rstd, d["dh_out"], o["dh"], o["dy"],
                                 o["dgamma_post"], B.alloc_norm_residual_workspace(cfg) if ws is None else ws,
                                 gate=d["gate"], gate_mode=mode_of(B, gate), res_scale=a,
                                 gamma_pre=d["gamma_pre"], du=d["du"], dgamma_pre=o["dgamma_pre"],
                                 dgate=o["dgate"], stream=stream)
    return o


def gate64(d, H):
    return torch.ones((1, H), dtype=torch.float64) if d["gate"] is None else d["gate"]


def near(got, ref, tol, what):
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), "%s: %.3g of its bound" % (what, float((err / tol).max()))


def check_forward(d, T, H, a, h_out, u, rstd, eps=EPS):
    r = f64(d)
    ref = F.norm_residual(r["h"], r["y"], r["gamma_post"], gate64(r, H), a, eps, r["gamma_pre"])
    near(h_out, ref["h_out"], ref["h_tol"], "h_out")
    rel = (H + 16) * F.U32
    near(rstd[0], ref["rp"], rel * ref["rp"], "rp")
    if u is not None:
        near(u, ref["u"], ref["u_tol"], "u")
        # rq also carries the errors of h' (of the magnitudes that cancel in it)
        mag = (a * r["h"]).abs() + (ref["h_out"] - a * r["h"]).abs()
        slack = rel * (1.0 + (ref["rq"][:, None] ** 2 * mag * ref["h_out"].abs()).mean(1))
        near(rstd[1], ref["rq"], slack * ref["rq"], "rq")
    return ref


SHAPES = [(1, 8), (1, 5120), (3, 264), (5, 8192), (7, 1032), (150, 512), (301, 72), (2, 16384), (4, 9000)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("gate", MODES)
@pytest.mark.parametrize("pre", [True, False])
def test_forward(B, T, H, gate, pre):
    d = make(T, H, gate, pre)
    a = 0.75 if T % 2 else 1.0
    h_out, u, rstd = forward(B, d, T, H, gate, a)
    torch.cuda.synchronize()
    check_forward(d, T, H, a, h_out, u, rstd)
    if not pre:
        assert bool(rstd[1].isnan().all())     # left alone


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("gate", MODES)
@pytest.mark.parametrize("pre", [True, False])
def test_backward(B, T, H, gate, pre):
    d = make(T, H, gate, pre, seed=1)
    a = 1.0 if T % 2 else -0.5
    _, _, rstd = forward(B, d, T, H, gate, a)
    got = backward(B, d, T, H, gate, a, rstd)
    torch.cuda.synchronize()
    check_backward(d, T, H, gate, a, rstd, got)


def check_backward(d, T, H, gate, a, rstd, got):
    r = f64(d)
    rs = rstd.cpu().double()
    ref = F.norm_residual_backward(r["h"], r["y"], r["gamma_post"], gate64(r, H), a, r["gamma_pre"],
                                   rs[0], rs[1], r["dh_out"], r["du"])
    for name, (v, e) in ref.items():
        if name == "dgate":
            if gate == "none":
                continue
            if gate == "channel":
                v, e = v.sum(0), e.sum(0) + T * F.U32 * v.abs().sum(0)
        if got[name].dtype is torch.bfloat16:
            e = e + F.HALF_BF16 * (v.abs() + e)
        else:
            e = e + 2.0 ** -24 * v.abs()
        near(got[name], v, e + 1e-38, name)


def test_gradients_of_the_kernel_match_differences(B):
    """Directional differences of the 64-bit forward pass along the kernel's own gradients."""
    T, H, a = 4, 512, 1.0
    d = make(T, H, "channel", True, seed=5)
    _, _, rstd = forward(B, d, T, H, "channel", a)
    got = backward(B, d, T, H, "channel", a, rstd)
    torch.cuda.synchronize()
    r = f64(d)

    def loss(**over):
        v = {**r, **over}
        o = F.norm_residual(v["h"], v["y"], v["gamma_post"], v["gate"][None], a, EPS, v["gamma_pre"])
        return float((o["h_out"] * r["dh_out"]).sum() + (o["u"] * r["du"]).sum())

    gen = torch.Generator().manual_seed(2)
    for name, grad in (("h", "dh"), ("y", "dy"), ("gamma_post", "dgamma_post"),
                       ("gamma_pre", "dgamma_pre"), ("gate", "dgate")):
        dirn = torch.randn(r[name].shape, generator=gen, dtype=torch.float64)
        step = 1e-4
        diff = (loss(**{name: r[name] + step * dirn}) - loss(**{name: r[name] - step * dirn})) / (2 * step)
        dot = got[grad].cpu().double() * dirn
        # each stored gradient is off by half a bf16 step at most (fp32 ones far less)
        assert abs(float(dot.sum()) - diff) <= 2 * F.HALF_BF16 * float(dot.abs().sum()) + 1e-4


def test_zero_rows_and_large_rows(B):
    """Rows of zeros (the norm is 1/sqrt(eps)), and rows near bf16's ends."""
    T, H = 4, 512
    d = make(T, H, "channel", True, seed=9)
    d["y"][0] = 0
    d["h"][0] = 0
    d["y"][1] *= 2.0 ** 40
    d["h"][1] *= 2.0 ** -30
    d["y"][2] *= 2.0 ** -60
    h_out, u, rstd = forward(B, d, T, H, "channel", 1.0)
    torch.cuda.synchronize()
    check_forward(d, T, H, 1.0, h_out, u, rstd)
    assert torch.equal(u[0], torch.zeros_like(u[0]))
    got = backward(B, d, T, H, "channel", 1.0, rstd)
    torch.cuda.synchronize()
    assert all(bool(v.isfinite().all()) for v in got.values())


def test_nan_row_stays_in_its_row(B):
    T, H = 3, 256
    d = make(T, H, "token", True)
    clean, uc, _ = forward(B, d, T, H, "token", 1.0)
    d["y"][1, 7] = math.nan
    h_out, u, _ = forward(B, d, T, H, "token", 1.0)
    torch.cuda.synchronize()
    for t in (0, 2):
        assert torch.equal(h_out[t], clean[t]) and torch.equal(u[t], uc[t])
    assert bool(h_out[1].isnan().all()) and bool(u[1].isnan().all())


@pytest.mark.parametrize("gate", MODES)
def test_in_place(B, gate):
    """h_out over h, u over y; dh over dh_out, dy over du: the same bits as apart."""
    T, H, a = 200, 1024, 0.5
    d = make(T, H, gate, True, seed=3)
    h_out, u, rstd = forward(B, d, T, H, gate, a)
    ref = backward(B, d, T, H, gate, a, rstd)
    e = {n: None if v is None else v.clone() for n, v in d.items()}
    got = backward(B, e, T, H, gate, a, rstd, dh=e["dh_out"], dy=e["du"])
    assert all(ref[n] is None or torch.equal(ref[n], got[n]) for n in ref)
    h2, u2, r2 = forward(B, e, T, H, gate, a, h_out=e["h"], u=e["y"])
    assert torch.equal(h2, h_out) and torch.equal(u2, u) and torch.equal(r2, rstd)


def test_no_tokens(B):
    H = 256
    d = make(0, H, "channel", True)
    forward(B, d, 0, H, "channel", 1.0)
    got = backward(B, d, 0, H, "channel", 1.0, torch.empty((2, 0), device="cuda"))
    torch.cuda.synchronize()
    for n in ("dgamma_post", "dgamma_pre", "dgate"):
        assert torch.equal(got[n], torch.zeros(H, device="cuda"))


def test_same_bits_from_graph_and_stream(B):
    T, H = 333, 640
    d = make(T, H, "channel", True, seed=4)
    _, _, rstd = forward(B, d, T, H, "channel", 1.0)
    ref = backward(B, d, T, H, "channel", 1.0, rstd)
    ws = B.alloc_norm_residual_workspace(cfg_of(B, T, H))
    ws.fill_(0xff)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = backward(B, d, T, H, "channel", 1.0, rstd, ws=ws)
    side.synchronize()
    assert all(torch.equal(ref[n], got[n]) for n in ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h_out, u, r2 = forward(B, d, T, H, "channel", 1.0)
        got = backward(B, d, T, H, "channel", 1.0, r2, ws=ws)
    d["y"].copy_(torch.randn((T, H), device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    check_forward(d, T, H, 1.0, h_out, u, r2)
    check_backward(d, T, H, "channel", 1.0, r2, got)
    del g


def test_offsets_beyond_32_bits(B):
    """2^31 elements and more in a tensor: the last rows are right, and the column sums."""
    T, H, last = 262200, 8192, 5
    cfg = cfg_of(B, T, H)
    h, y = (torch.zeros((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    d = make(last, H, "token", True, seed=6)
    h[-last:], y[-last:] = d["h"], d["y"]
    gate = torch.zeros_like(h)
    gate[-last:] = d["gate"]
    h_out, u = torch.empty_like(h), torch.empty_like(h)
    rstd = torch.empty((2, T), device="cuda")
    B.moe_norm_residual(cfg, h, y, d["gamma_post"], h_out, EPS, gate=gate, gate_mode=B.MOE_GATE_TOKEN,
                        res_scale=0.5, gamma_pre=d["gamma_pre"], u=u, rstd=rstd)
    torch.cuda.synchronize()
    r2 = rstd[:, -last:].contiguous()
    check_forward(d, last, H, 0.5, h_out[-last:], u[-last:], r2)
    assert not bool(h_out[:-last].any()) and not bool(u[:-last].any())
    # the other rows' gradients are zero, so the sums are the last rows'
    dh_out, du = h_out.zero_(), u.zero_()
    dh_out[-last:], du[-last:] = d["dh_out"], d["du"]
    o = {"dh": torch.empty_like(h), "dy": torch.empty_like(h), "dgate": torch.empty_like(h),
         "dgamma_post": torch.empty(H, device="cuda"), "dgamma_pre": torch.empty(H, device="cuda")}
    B.moe_norm_residual_backward(cfg, h, y, d["gamma_post"], rstd, dh_out, o["dh"], o["dy"], o["dgamma_post"],
                                 B.alloc_norm_residual_workspace(cfg), gate=gate, gate_mode=B.MOE_GATE_TOKEN,
                                 res_scale=0.5, gamma_pre=d["gamma_pre"], du=du, dgamma_pre=o["dgamma_pre"],
                                 dgate=o["dgate"])
    torch.cuda.synchronize()
    assert not any(bool(o[n][:-last].any()) for n in ("dh", "dy", "dgate"))
    check_backward(d, last, H, "token", 0.5, r2, {n: v[-last:] if v.dim() == 2 else v for n, v in o.items()})


@pytest.mark.parametrize("T,H", [(2400, 64), (1500, 264), (1201, 2560), (310, 5136), (320, 6144), (305, 6152),
                                 (300, 8200), (299, 12000)])
@pytest.mark.parametrize("gate", MODES)
def test_many_rows(B, T, H, gate):
    """More rows than blocks at every number of blocks an SM and every row length class."""
    d = make(T, H, gate, gate != "channel", seed=7)
    h_out, u, rstd = forward(B, d, T, H, gate, 0.75)
    got = backward(B, d, T, H, gate, 0.75, rstd)
    torch.cuda.synchronize()
    check_forward(d, T, H, 0.75, h_out, u, rstd)
    check_backward(d, T, H, gate, 0.75, rstd, got)
