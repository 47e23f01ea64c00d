"""MXFP4 quantisation and its read-back against the value-by-value reference: exact."""
import math

import pytest
import torch

from oracle import few as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from sigmoid_top_routing_warp_b200 import binding
    return binding


def roundtrip(B, x):
    R, C = x.shape
    q = torch.full((R, C // 2), 0xaa, dtype=torch.uint8, device="cuda")
    s = torch.full((R, C // 32), 0xaa, dtype=torch.uint8, device="cuda")
    back = torch.full((R, C), math.nan, dtype=torch.bfloat16, device="cuda")
    B.moe_quantize_mx(x.cuda(), q, s)
    B.moe_dequantize_mx(q, s, back)
    torch.cuda.synchronize()
    return q.cpu(), s.cpu(), back.cpu()


@pytest.mark.parametrize("R,C", [(1, 32), (3, 32), (5, 96), (7, 544), (64, 128), (33, 1056)])
def test_random(B, R, C):
    g = torch.Generator().manual_seed(R * C)
    x = torch.randn((R, C), generator=g) * torch.exp2(torch.randint(-20, 20, (R, 1), generator=g).float())
    x = x.to(torch.bfloat16)
    q, s, back = roundtrip(B, x)
    rq, rs = F.mx_quantize(x)
    assert torch.equal(s, rs) and torch.equal(q, rq)
    assert torch.equal(back.double(), F.mx_values(rq, rs))


def test_every_bf16_value(B):
    """All 65536 bit patterns, each at the head of its own block of zeros, and beside a block maximum
    that fixes the scale at 1."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16)
    x = torch.zeros((65536, 32), dtype=torch.bfloat16)
    x[:, 0] = v
    q, s, back = roundtrip(B, x)
    bad = ~v.double().isfinite()
    assert bool((s[:, 0][bad] == 255).all()) and bool((q[bad] == 0).all())
    assert bool(back[bad].isnan().all())
    ok = ~bad
    amax = v.double().abs()
    e = torch.frexp(torch.where(ok & (amax > 0), amax, torch.ones_like(amax))).exponent.long() + 124
    e = torch.where(amax == 0, torch.full_like(e, 127), e.clamp(min=0))
    assert torch.equal(s[:, 0][ok].long(), e[ok])
    assert torch.equal(back.double()[ok], F.mx_values(q, s)[ok])
    # the head is rounded to nearest of its block's grid
    grid = torch.tensor(F.E2M1, dtype=torch.float64)
    m = amax * torch.exp2(127.0 - e.double())
    near = (grid[None] - m[:, None]).abs().amin(1)
    got = (back[:, 0].double().abs() * torch.exp2(127.0 - e.double()) - m).abs()
    assert torch.equal(got[ok], near[ok])
    # ties go to the even code: halfway points at scale 1
    x = torch.zeros((1, 32), dtype=torch.bfloat16)
    x[0, :9] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.0])
    q, s, back = roundtrip(B, x)
    assert int(s[0, 0]) == 127
    assert back[0, :9].tolist() == [4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -0.0]
    assert int(q[0, 4]) & 8 == 8


def test_every_code_and_scale_reads_back(B):
    s = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(256, 1)
    q = torch.arange(16, dtype=torch.uint8)
    q = (q | ((15 - q) << 4)).repeat(256, 1)
    out = torch.empty((256, 32), dtype=torch.bfloat16, device="cuda")
    B.moe_dequantize_mx(q.cuda(), s.cuda(), out)
    ref = F.mx_values(q, s).float().to(torch.bfloat16)
    got = out.cpu()
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got[~got.isnan()], ref[~ref.isnan()])


def test_graph_and_stream(B):
    x = torch.randn((9, 160), device="cuda").to(torch.bfloat16)
    q = torch.empty((9, 80), dtype=torch.uint8, device="cuda")
    s = torch.empty((9, 5), dtype=torch.uint8, device="cuda")
    back = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.moe_quantize_mx(x, q, s)
        B.moe_dequantize_mx(q, s, back)
    x.copy_(torch.randn((9, 160), device="cuda") * 3.0)
    g.replay()
    torch.cuda.synchronize()
    rq, rs = F.mx_quantize(x.cpu())
    assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu(), rs)
    side = torch.cuda.Stream()
    q.zero_()
    side.wait_stream(torch.cuda.current_stream())
    B.moe_quantize_mx(x, q, s, stream=side)
    side.synchronize()
    assert torch.equal(q.cpu(), rq)


def test_offsets_beyond_32_bits(B):
    """2^31 elements and more: the last rows are right."""
    R, C, last = 262200, 8192, 3
    x = torch.zeros((R, C), dtype=torch.bfloat16, device="cuda")
    x[-last:] = torch.randn((last, C), device="cuda").to(torch.bfloat16)
    q = torch.empty((R, C // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((R, C // 32), dtype=torch.uint8, device="cuda")
    B.moe_quantize_mx(x, q, s)
    rq, rs = F.mx_quantize(x[-last:].cpu())
    assert torch.equal(q[-last:].cpu(), rq) and torch.equal(s[-last:].cpu(), rs)
    assert not bool(q[:-last].any()) and bool((s[:-last] == 127).all())
    x.fill_(1.0)
    B.moe_dequantize_mx(q, s, x)
    torch.cuda.synchronize()
    assert torch.equal(x[-last:].cpu().double(), F.mx_values(rq, rs)) and not bool(x[:-last].any())
