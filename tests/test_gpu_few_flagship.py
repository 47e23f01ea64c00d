"""The few-token layer at the decode layer's width (5120 x 1536) against its 64-bit reference, for every
weight type."""
import functools
import math

import pytest
import torch

from oracle import few as F
from test_gpu_few import KINDS, check

pytestmark = pytest.mark.gpu
H, I, E = 5120, 1536, 32


@pytest.fixture(scope="module")
def B():
    from sigmoid_top_routing_warp_b200 import binding
    return binding


class Values:
    """float64 CPU values of the experts that are asked for."""

    def __init__(self, kind, stored, scale):
        self.kind, self.stored, self.scale = kind, stored, scale

    @functools.lru_cache(maxsize=None)
    def __getitem__(self, e):
        w = self.stored[e].cpu()
        if self.kind == "bf16":
            return w.double()
        return (F.fp8_values if self.kind == "fp8" else F.mx_values)(w, self.scale[e].cpu())


def weights(B, kind, g, n, rows, cols):
    from sigmoid_top_routing_warp_b200 import workloads as W
    w = (torch.randn((n, rows, cols), generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    if kind == "bf16":
        return w, None, Values(kind, w, None)
    if kind == "fp8":
        q, s = (torch.stack(v) for v in zip(*(W.quantize_weight_e4m3(m.float()) for m in w)))
    else:
        q = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device="cuda")
        s = torch.empty((n, rows, cols // 32), dtype=torch.uint8, device="cuda")
        B.moe_quantize_mx(w.view(n * rows, cols), q, s)
    return q, s, Values(kind, q, s)


@pytest.mark.parametrize("kind", KINDS)
def test_against_64_bits(B, kind):
    """Batches of every tile shape on the same weights, on one workspace."""
    k = 3
    g = torch.Generator(device="cuda").manual_seed(101)
    p = {"w13": weights(B, kind, g, E, 2 * I, H), "w2": weights(B, kind, g, E, H, I)}
    shared = {"w13s": weights(B, kind, g, 1, 2 * I, H), "w2s": weights(B, kind, g, 1, H, I)}
    for name, (q, s, v) in shared.items():
        p[name] = (q[0], None if s is None else s[0], v[0])
    p["w_router"] = (torch.randn((E, H), generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    p["bias"] = torch.rand((E,), generator=g, device="cuda") * 0.2 - 0.1
    ws = None
    for T in (16, 1, 4, 7):
        p["cfg"] = B.MoeConfig(T=T, H=H, E=E, k=k, I=I, n_shared=1,
                               dtype={"bf16": B.MOE_DTYPE_BF16, "fp8": B.MOE_DTYPE_FP8_E4M3_BLOCK128,
                                      "mxfp4": B.MOE_DTYPE_MXFP4_BLOCK32}[kind])
        p["x"] = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
        p["ws"] = ws = B.alloc_few_workspace(p["cfg"]) if ws is None else ws
        p["out"] = torch.full((T, H), math.nan, dtype=torch.bfloat16, device="cuda")
        p["idx"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        p["w"] = torch.empty((T, k), device="cuda")
        B.moe_forward_few(p["cfg"], p["x"], p["w_router"], p["bias"], p["w13"][0], p["w2"][0], p["w13s"][0],
                          p["w2s"][0], p["out"], p["ws"], topk_idx=p["idx"], topk_w=p["w"],
                          w13_scale=p["w13"][1], w2_scale=p["w2"][1], w13s_scale=p["w13s"][1],
                          w2s_scale=p["w2s"][1])
        check(B, p)
