"""The few-token layer (moe_forward_few) against its 64-bit reference."""
import math

import pytest
import torch

from oracle import few as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from sigmoid_top_routing_warp_b200 import binding
    return binding


KINDS = ("bf16", "fp8", "mxfp4")


def matrix(B, kind, g, n, rows, cols, std):
    """n matrices: (stored, scale, float64 CPU values)."""
    from sigmoid_top_routing_warp_b200 import workloads as W
    w = torch.randn((n, rows, cols), generator=g, device="cuda") * std
    if kind == "bf16":
        w = w.to(torch.bfloat16)
        return w, None, w.cpu().double()
    if kind == "fp8":
        q, s = zip(*(W.quantize_weight_e4m3(m) for m in w))
        q, s = torch.stack(q), torch.stack(s)
        return q, s, F.fp8_values(q.cpu(), s.cpu())
    w = w.to(torch.bfloat16)
    q = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((n, rows, cols // 32), dtype=torch.uint8, device="cuda")
    B.moe_quantize_mx(w.view(n * rows, cols), q, s)
    return q, s, F.mx_values(q.cpu(), s.cpu())


def make(B, kind, T, H, E, k, I, n_shared=1, seed=0, x=None, bias=None, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    p = {"kind": kind}
    p["x"] = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16) if x is None else x
    p["w_router"] = (torch.randn((E, H), generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    p["bias"] = torch.rand((E,), generator=g, device="cuda") * 0.2 - 0.1 if bias is None else bias
    p["w13"] = matrix(B, kind, g, E, 2 * I, H, 0.05)
    p["w2"] = matrix(B, kind, g, E, H, I, 0.05)
    p["w13s"] = p["w2s"] = (None, None, None)
    if n_shared:
        for name, r, c in (("w13s", 2 * n_shared * I, H), ("w2s", H, n_shared * I)):
            p[name] = tuple(None if v is None else v[0] for v in matrix(B, kind, g, 1, r, c, 0.05))
    p["cfg"] = B.MoeConfig(T=T, H=H, E=E, k=k, I=I, n_shared=n_shared,
                           dtype={"bf16": B.MOE_DTYPE_BF16, "fp8": B.MOE_DTYPE_FP8_E4M3_BLOCK128,
                                  "mxfp4": B.MOE_DTYPE_MXFP4_BLOCK32}[kind], **kw)
    p["ws"] = B.alloc_few_workspace(p["cfg"])
    p["out"] = torch.full((T, H), math.nan, dtype=torch.bfloat16, device="cuda")
    p["idx"] = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    p["w"] = torch.full((T, k), math.nan, device="cuda")
    return p


def call(B, p, stream=None, ws=None, out=None, idx="idx", w="w"):
    B.moe_forward_few(p["cfg"], p["x"], p["w_router"], p["bias"], p["w13"][0], p["w2"][0],
                      p["w13s"][0], p["w2s"][0], p["out"] if out is None else out,
                      p["ws"] if ws is None else ws, topk_idx=p.get(idx), topk_w=p.get(w),
                      stream=stream, w13_scale=p["w13"][1], w2_scale=p["w2"][1],
                      w13s_scale=p["w13s"][1], w2s_scale=p["w2s"][1])


def reference(p):
    c = p["cfg"]
    return F.layer(p["x"].cpu().double(), p["w_router"].cpu().double(), p["bias"].cpu(),
                   p["w13"][2], p["w2"][2], p["w13s"][2], p["w2s"][2], c.k, n_group=c.n_group,
                   topk_group=c.topk_group, group_topn=c.group_topn, norm=c.norm_topk_prob,
                   rsf=c.routed_scaling_factor)


def check(B, p):
    torch.cuda.synchronize()
    B.moe_check_device_status(p["ws"])
    out, tol, idx, w = reference(p)
    assert torch.equal(p["idx"].cpu(), idx)
    # binary64 weights rounded once; a logit is off by a few 2^-25 of its partial sums
    assert torch.allclose(p["w"].cpu().double(), w, rtol=2.0 ** -20, atol=0)
    err = (p["out"].cpu().double() - out).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,H,E,k,I,n_shared", [
    (1, 128, 32, 1, 128, 0), (1, 512, 32, 4, 128, 1), (2, 256, 64, 8, 384, 1),
    (3, 640, 96, 6, 256, 2), (7, 1024, 32, 2, 128, 0), (8, 384, 160, 5, 128, 3),
    (9, 128, 32, 32, 128, 1), (13, 768, 64, 3, 640, 1), (16, 1152, 128, 8, 256, 2),
    (16, 128, 32, 31, 128, 1)])
def test_layer(B, kind, T, H, E, k, I, n_shared):
    p = make(B, kind, T, H, E, k, I, n_shared, seed=T)
    call(B, p)
    check(B, p)


@pytest.mark.parametrize("kw", [
    dict(n_group=4, topk_group=2), dict(n_group=8, topk_group=1, group_topn=1, norm_topk_prob=False),
    dict(n_group=32, topk_group=7, group_topn=3), dict(n_group=2, topk_group=2, group_topn=16),
    dict(routed_scaling_factor=2.5)])
def test_group_choice(B, kw):
    p = make(B, "bf16", 5, 256, 96 if kw.get("n_group") == 32 else 128, 6 if kw.get("n_group") != 32 else 4,
             128, seed=3, **kw)
    call(B, p)
    check(B, p)


@pytest.mark.parametrize("E", [512, 768, 1024])
def test_many_experts(B, E):
    p = make(B, "mxfp4", 16, 128, E, 32, 128, seed=E)
    call(B, p)
    check(B, p)


def test_ties_go_to_the_lower_expert(B):
    """Zero tokens give equal scores; the bias alone decides, and ties by index."""
    bias = torch.zeros(64, device="cuda")
    bias[40] = 0.25
    p = make(B, "bf16", 4, 256, 64, 4, 128, x=torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda"),
             bias=bias)
    call(B, p)
    torch.cuda.synchronize()
    assert p["idx"].cpu().tolist() == [[40, 0, 1, 2]] * 4
    assert torch.equal(p["out"], torch.zeros_like(p["out"]))


def test_all_tokens_on_the_same_experts(B):
    bias = torch.zeros(32, device="cuda")
    bias[[3, 17, 30]] = 5.0
    p = make(B, "fp8", 16, 256, 32, 3, 256, bias=bias, seed=5)
    call(B, p)
    check(B, p)
    assert sorted(set(p["idx"].cpu().flatten().tolist())) == [3, 17, 30]


def test_nan_and_infinite_tokens_stay_in_their_rows(B):
    p = make(B, "mxfp4", 6, 256, 32, 4, 128, seed=7)
    clean = torch.empty_like(p["out"])
    call(B, p, out=clean)
    p["x"][2, 5] = math.nan
    p["x"][4, 9] = math.inf
    call(B, p)
    torch.cuda.synchronize()
    for t in (0, 1, 3, 5):
        assert torch.equal(p["out"][t], clean[t])
    assert bool(p["out"][2].isnan().all())
    assert not bool(p["out"][4].isfinite().all())
    # every key of a NaN token ranks equal: the lowest experts
    assert p["idx"][2].cpu().tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("kind", KINDS)
def test_nan_weights_are_seen(B, kind):
    """A NaN weight, code (e4m3 0x7f) or scale (e8m0 255) of a down projection row makes that output
    NaN for the tokens of its expert, and no other."""
    p = make(B, kind, 3, 256, 32, 2, 128, seed=11)
    clean = torch.empty_like(p["out"])
    call(B, p, out=clean)
    torch.cuda.synchronize()
    e = int(p["idx"][1, 0])
    if kind == "fp8":
        p["w2"][0][e, 77, 33] = 0xff
    elif kind == "bf16":
        p["w2"][0][e, 77, 33] = math.nan
    else:
        p["w2"][1][e, 77, 1] = 255
    call(B, p)
    torch.cuda.synchronize()
    hit = (p["idx"] == e).any(1)
    bad = p["out"].isnan()
    assert torch.equal(bad[:, 77], hit) and int(bad.sum()) == int(hit.sum())
    bad[:, 77] = True
    assert torch.equal(p["out"][~bad], clean[~bad])


@pytest.mark.parametrize("kind", KINDS)
def test_wide_range_of_magnitudes(B, kind):
    """Tokens at 2^-40 and 2^20 of the usual size (the reference's bound scales with them)."""
    p = make(B, kind, 4, 512, 32, 2, 128, seed=13)
    p["x"][1] *= 2.0 ** -40
    p["x"][2] *= 2.0 ** 20
    p["w_router"].zero_()          # keep the choice with the biases
    call(B, p)
    check(B, p)


def test_repeat_streams_graph_and_workspace(B):
    """The same bits from a second call, another stream, a captured and replayed graph with new
    inputs; two workspaces at once on two streams."""
    p = make(B, "bf16", 5, 512, 64, 4, 256, seed=17)
    call(B, p)
    first = p["out"].clone()
    call(B, p)
    assert torch.equal(p["out"], first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p["out"].zero_()
    s.wait_stream(torch.cuda.current_stream())
    call(B, p, stream=s)
    s.synchronize()
    assert torch.equal(p["out"], first)
    ws2, out2 = B.alloc_few_workspace(p["cfg"]), torch.empty_like(first)
    torch.cuda.synchronize()
    for _ in range(20):
        call(B, p, stream=s)
        call(B, p, ws=ws2, out=out2, idx="none", w="none")
    torch.cuda.synchronize()
    assert torch.equal(p["out"], first) and torch.equal(out2, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(B, p)
    p["out"].zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(p["out"], first)
    p["x"].copy_(torch.randn_like(p["x"].float()).to(torch.bfloat16))
    g.replay()
    check(B, p)
    del g


def test_optional_outputs_and_dirty_workspace_contents(B):
    """The choice need not be returned, and only the status block of the workspace has to be zero."""
    p = make(B, "bf16", 2, 256, 32, 2, 128, seed=19)
    call(B, p)
    first = p["out"].clone()
    p["ws"][256:] = 0xff
    p["out"].zero_()
    call(B, p, idx="none", w="none")
    torch.cuda.synchronize()
    assert torch.equal(p["out"], first)


@pytest.mark.parametrize("kind,T", [("bf16", 3), ("bf16", 12), ("fp8", 2), ("mxfp4", 7)])
def test_out_over_x(B, kind, T):
    """The same bits when out is x itself."""
    p = make(B, kind, T, 512, 64, 4, 256, seed=29)
    call(B, p)
    apart = p["out"].clone()
    call(B, p, out=p["x"])
    torch.cuda.synchronize()
    assert torch.equal(p["x"], apart)


@pytest.mark.parametrize("kind", ("fp8", "mxfp4"))
def test_one_value_far_above_the_others(B, kind):
    """A token whose largest value is 2^20 times the others keeps the others' bits: the lift is for the
    whole token, and what it drops is below 2^-39 of the largest, 2^-19 of the others.  Columns where the
    large value meets a zero weight show it."""
    p = make(B, kind, 2, 256, 32, 2, 128, n_shared=0, seed=31)
    p["w_router"].zero_()
    big = 8
    p["x"][0, big] = 2.0 ** 20
    pack = 2 if kind == "mxfp4" else 1
    p["w13"][0][:, :, big // pack] = 0         # (its neighbour's codes too, for MXFP4)
    vals = p["w13"][2]
    vals[:, :, big] = 0
    if pack == 2:
        vals[:, :, big + 1] = 0
    call(B, p)
    torch.cuda.synchronize()
    out, tol, idx, _ = reference(p)
    assert torch.equal(p["idx"].cpu(), idx)
    # the token's values are off by half a binary16 step below 2^-14 of the lift, 2^-39 of the
    # largest: less than 2^-9 (half a bf16 step) of a value of 2^-10 or more; the sums of 256
    # terms by 2^-39 * 2^20 * sum |w|, which the SwiGLU and the down projection carry on
    e = 2.0 ** -19
    for t in range(2):
        extra = torch.zeros_like(out[t])
        for j in range(2):
            w13, w2 = vals[int(idx[t, j])], p["w2"][2][int(idx[t, j])]
            g, u = (p["x"][t].cpu().double() @ w13.T).split(128)
            dg, du = (e * w13.abs().sum(1)).split(128)
            extra += (w2.abs() @ (1.1 * dg * (u.abs() + du) + g.abs() * du))
        err = (p["out"][t].cpu().double() - out[t]).abs()
        assert bool((err <= tol[t] + 2 * extra).all()), float((err / (tol[t] + 2 * extra)).max())


def test_stalled_block_times_out_and_the_next_call_is_clean(B):
    p = make(B, "bf16", 1, 256, 32, 2, 128, seed=23)
    call(B, p)
    first = p["out"].clone()
    p["cfg"].flags = B.MOE_FLAG_TEST_STALL
    call(B, p)
    with pytest.raises(B.MoeError) as err:
        B.moe_check_device_status(p["ws"])
    assert err.value.status == B.MOE_ERR_TIMEOUT
    p["cfg"].flags = 0
    call(B, p)
    B.moe_check_device_status(p["ws"])
    assert torch.equal(p["out"], first)


def test_flagship_shape_agrees_with_moe_forward(B):
    """The decode layer's sizes: moe_forward's own tolerance against this layer, same choice."""
    from sigmoid_top_routing_warp_b200 import workloads as W
    import dataclasses
    wl = dataclasses.replace(W.WORKLOADS["decode"], T=3)
    inp = W.make_inputs(wl, device="cuda")
    cfg = B.MoeConfig(T=wl.T, H=wl.H, E=wl.E, k=wl.k, I=wl.I, n_shared=wl.n_shared)
    ws, out = B.alloc_workspace(cfg), torch.empty((wl.T, wl.H), dtype=torch.bfloat16, device="cuda")
    args = [inp[n] for n in ("x", "w_router", "bias", "w13", "w2", "w13s", "w2s")]
    B.moe_forward(cfg, *args, out, ws)
    few = torch.empty_like(out)
    idx = torch.empty((wl.T, wl.k), dtype=torch.int32, device="cuda")
    B.moe_forward_few(cfg, *args, few, B.alloc_few_workspace(cfg), topk_idx=idx)
    torch.cuda.synchronize()
    assert torch.equal(idx, B.ws_view(ws, cfg, "topk_idx"))
    a, b = few.double(), out.double()
    assert float((a - b).norm() / a.norm()) <= 1e-2


def test_one_workspace_for_every_batch_size(B):
    """A decode loop's workspace, of the largest batch, serves the smaller ones and other weight types."""
    big = make(B, "bf16", 16, 256, 64, 4, 256, seed=37)
    for kind, T in (("bf16", 16), ("mxfp4", 1), ("fp8", 9), ("bf16", 3), ("mxfp4", 16), ("bf16", 16)):
        p = make(B, kind, T, 256, 64, 4, 256, seed=38 + T)
        p["ws"] = big["ws"]
        call(B, p)
        check(B, p)
