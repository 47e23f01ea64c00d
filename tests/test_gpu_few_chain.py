"""The operators together, as a model uses them: a decode step of two MoE
blocks on MXFP4 weights, captured and replayed, and a training step of a block
with norms, gate and residual scale around it."""
import math

import pytest
import torch

from oracle import few as F
from test_gpu_backward import assert_close_grad
from test_gpu_few import make as make_layer
from test_gpu_norm_residual import check_backward, check_forward, near

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def B():
    from sigmoid_top_routing_warp_b200 import binding
    return binding


@pytest.mark.parametrize("kind,T", [("mxfp4", 1), ("mxfp4", 4), ("fp8", 6), ("bf16", 16)])
def test_decode_step_of_two_blocks(B, kind, T):
    """norm -> layer -> residual and next norm, twice, in one graph; each result
    against the 64-bit formula of what the call before it left."""
    H, gates = 512, ("token", "none")
    layers = [make_layer(B, kind, T, H, 64, 4, 256, seed=41 + i) for i in range(2)]
    cfg = layers[0]["cfg"]
    g = torch.Generator(device="cuda").manual_seed(43 + T)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    bf = lambda v: v.to(torch.bfloat16)  # noqa: E731
    h0 = bf(r(T, H))
    gamma = [bf(1.0 + 0.1 * r(H)) for _ in range(5)]
    gate = bf(torch.sigmoid(r(T, H)))
    u = [torch.empty_like(h0) for _ in range(3)]
    h = [torch.empty_like(h0) for _ in range(2)]
    rstd = [torch.empty((2, T), device="cuda") for _ in range(2)]

    def step():
        B.moe_rmsnorm(cfg, h0, gamma[0], EPS, u[0])
        for i, p in enumerate(layers):
            B.moe_forward_few(cfg, u[i], p["w_router"], p["bias"], p["w13"][0], p["w2"][0], p["w13s"][0],
                              p["w2s"][0], p["out"], p["ws"], topk_idx=p["idx"], topk_w=p["w"],
                              w13_scale=p["w13"][1], w2_scale=p["w2"][1], w13s_scale=p["w13s"][1],
                              w2s_scale=p["w2s"][1])
            B.moe_norm_residual(cfg, h[i - 1] if i else h0, p["out"], gamma[1 + 2 * i], h[i], EPS,
                                gate=gate if gates[i] == "token" else None,
                                gate_mode=B.MOE_GATE_TOKEN if gates[i] == "token" else B.MOE_GATE_NONE,
                                res_scale=0.5, gamma_pre=gamma[2 + 2 * i], u=u[i + 1], rstd=rstd[i])

    def check():
        torch.cuda.synchronize()
        for i, p in enumerate(layers):
            B.moe_check_device_status(p["ws"])
            out, tol, idx, _ = F.layer(u[i].cpu().double(), p["w_router"].cpu().double(), p["bias"].cpu(),
                                       p["w13"][2], p["w2"][2], p["w13s"][2], p["w2s"][2], cfg.k)
            assert torch.equal(p["idx"].cpu(), idx)
            near(p["out"], out, tol, "layer %d" % i)
            check_forward({"h": h[i - 1] if i else h0, "y": p["out"], "gamma_post": gamma[1 + 2 * i],
                           "gate": gate if gates[i] == "token" else None, "gamma_pre": gamma[2 + 2 * i]},
                          T, H, 0.5, h[i], u[i + 1], rstd[i])

    step()
    check()
    first = u[2].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    u[2].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(u[2], first)
    h0.copy_(bf(r(T, H)))
    for _ in range(3):
        graph.replay()
    check()
    del graph


def test_training_step_of_a_block(B):
    """norm -> moe_forward -> norm, gate and residual; the gradient of the block's
    output goes back through moe_norm_residual_backward into moe_backward."""
    T, H, E, k, I = 96, 512, 32, 4, 128
    cfg = B.MoeConfig(T=T, H=H, E=E, k=k, I=I, n_shared=1)
    g = torch.Generator(device="cuda").manual_seed(53)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    bf = lambda v: v.to(torch.bfloat16)  # noqa: E731
    d = {"h": bf(r(T, H)), "gamma_post": bf(1.0 + 0.1 * r(H)), "gate": bf(torch.sigmoid(r(H))),
         "gamma_pre": bf(1.0 + 0.1 * r(H)), "dh_out": bf(r(T, H)), "du": bf(r(T, H))}
    w = {"w_router": bf(r(E, H) * 0.05), "w13": bf(r(E, 2 * I, H) * 0.05), "w2": bf(r(E, H, I) * 0.05),
         "w13s": bf(r(2 * I, H) * 0.05), "w2s": bf(r(H, I) * 0.05)}
    bias = r(E) * 0.05
    x, y = torch.empty_like(d["h"]), torch.empty_like(d["h"])
    ws = B.alloc_workspace(cfg)
    B.moe_rmsnorm(cfg, d["h"], d["gamma_pre"], EPS, x)
    B.moe_forward(cfg, x, w["w_router"], bias, w["w13"], w["w2"], w["w13s"], w["w2s"], y, ws)
    d["y"] = y
    h_out, u, rstd = torch.empty_like(y), torch.empty_like(y), torch.empty((2, T), device="cuda")
    B.moe_norm_residual(cfg, d["h"], y, d["gamma_post"], h_out, EPS, gate=d["gate"],
                        gate_mode=B.MOE_GATE_CHANNEL, res_scale=0.5, gamma_pre=d["gamma_pre"], u=u, rstd=rstd)
    o = {"dh": torch.empty_like(y), "dy": torch.empty_like(y)}
    for n in ("dgamma_post", "dgamma_pre", "dgate"):
        o[n] = torch.full((H,), math.nan, device="cuda")
    B.moe_norm_residual_backward(cfg, d["h"], y, d["gamma_post"], rstd, d["dh_out"], o["dh"], o["dy"],
                                 o["dgamma_post"], B.alloc_norm_residual_workspace(cfg), gate=d["gate"],
                                 gate_mode=B.MOE_GATE_CHANNEL, res_scale=0.5, gamma_pre=d["gamma_pre"],
                                 du=d["du"], dgamma_pre=o["dgamma_pre"], dgate=o["dgate"])
    logits, idx, tw = (B.ws_view(ws, cfg, n) for n in ("logits", "topk_idx", "topk_w"))
    dx = torch.empty_like(x)
    grads = {n: torch.empty(v.shape, dtype=torch.float32, device="cuda") for n, v in w.items()}
    B.moe_backward(cfg, x, w["w_router"], logits, idx, tw, w["w13"], w["w2"], w["w13s"], w["w2s"], o["dy"],
                   dx, grads["w_router"], grads["w13"], grads["w2"], grads["w13s"], grads["w2s"],
                   B.alloc_backward_workspace(cfg))
    torch.cuda.synchronize()
    check_forward(d, T, H, 0.5, h_out, u, rstd)
    check_backward(d, T, H, "channel", 0.5, rstd, o)
    # the shared expert's down projection, whose gradient is dy^T (SiLU(g) u), to
    # moe_backward's own bar; dx is finite (its parity is tested with moe_backward)
    gg, uu = (x.cpu().double() @ w["w13s"].cpu().double().T).split(I, 1)
    want = o["dy"].cpu().double().T @ (gg / (1.0 + torch.exp(-gg)) * uu)
    assert_close_grad(grads["w2s"].cpu().double().numpy(), want.numpy(), "dw2s")
    assert bool(dx.isfinite().all())
