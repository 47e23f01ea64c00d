"""The few-token layer (moe_forward_few) where its inputs or its shape reach an edge:
stages of several widths in one slot of its ring, a call that
gives up, SwiGLU outputs at the end of their range, logits that cancel, tie
or leave no score."""
import math

import pytest
import torch

from test_gpu_few import KINDS, call, check, make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from sigmoid_top_routing_warp_b200 import binding
    return binding


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [4, 9, 16])
def test_wide_and_narrow_stages_share_slots(B, kind, T):
    """Two experts with every token between experts with a few: the activations of a narrow stage lie
    where a full stage's weights land next.  The same bits from every call, and right ones."""
    bias = torch.zeros(32, device="cuda")
    bias[[11, 30]] = 3.0
    p = make(B, kind, T, 2304, 32, 6, 256, bias=bias, seed=61)
    call(B, p)
    check(B, p)
    first = p["out"].clone()
    for _ in range(50):
        call(B, p)
        assert torch.equal(p["out"], first)


@pytest.mark.parametrize("kind", KINDS)
def test_a_stalled_call_leaves_nothing_behind(B, kind):
    """A call that gives up waits for its own copies first: with shared and routed experts, a call of another
    size that follows at once gives its bits."""
    p = make(B, kind, 3, 1024, 32, 4, 256, n_shared=2, seed=67)
    q = make(B, kind, 8, 640, 32, 4, 128, seed=71)
    call(B, p)
    call(B, q)
    first, other = p["out"].clone(), q["out"].clone()
    p["cfg"].flags = B.MOE_FLAG_TEST_STALL
    call(B, p)
    q["out"].zero_()
    call(B, q)
    with pytest.raises(B.MoeError) as err:
        B.moe_check_device_status(p["ws"])
    assert err.value.status == B.MOE_ERR_TIMEOUT
    B.moe_check_device_status(q["ws"])
    assert torch.equal(q["out"], other)
    p["cfg"].flags = 0
    call(B, p)
    check(B, p)
    assert torch.equal(p["out"], first)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 3, 6, 12])
@pytest.mark.parametrize("n_shared", [0, 1])
@pytest.mark.parametrize("end", ["finite", "infinite"])
def test_swiglu_outputs_at_the_end_of_their_range(B, kind, T, n_shared, end):
    """One feature of token 0's SwiGLU output is just below 2^128, above bf16's largest value with bf16
    weights, or infinite: the outputs are the formula's, an infinity times a weight its sign's infinity."""
    H, I, f, col, e = 256, 128, 5, 6, 7
    bias = torch.zeros(32, device="cuda")
    bias[e] = 5.0
    p = make(B, kind, T, H, 32, 1, I, n_shared=n_shared, bias=bias, seed=73)
    p["w_router"].zero_()
    stored, scale, vals = p["w13"]
    pack = 2 if kind == "mxfp4" else 1
    stored[:, :, col // pack] = 0                    # (its neighbour's codes too, for MXFP4)
    vals[:, :, col:col + pack] = 0
    if n_shared:
        p["w13s"][0][:, col // pack] = 0
        p["w13s"][2][:, col:col + pack] = 0
    if kind == "bf16":
        for row, v in ((f, 181.0 / 128.0), (I + f, 181.0 / 256.0)):      # 181^2 / 2^14 is above 2 - 2^-8
            stored[:, row, col] = v
            vals[:, row, col] = v
    elif kind == "fp8":
        stored[:, (f, I + f), col] = 0x38            # 1.0
        vals[:, (f, I + f), col] = scale[:, (0, 1), 0].cpu().double()
    else:
        stored[:, (f, I + f), col // 2] = 0x02       # 1.0 in the lower half
        vals[:, (f, I + f), col] = torch.exp2(scale[:, (f, I + f), col // 32].cpu().double() - 127.0)
    unit = float(vals[e, f, col] * vals[e, I + f, col])
    p["x"][0] = 0
    n = math.ceil((128.0 - math.log2(unit)) / 2.0) - 1       # the largest with unit * 4^n below 2^128
    p["x"][0, col] = 2.0 ** (n if end == "finite" else n + 1)
    a = unit * float(p["x"][0, col]) ** 2
    assert (2.0 ** 126 <= a < 2.0 ** 128) if end == "finite" else a >= 2.0 ** 128
    if kind == "bf16" and end == "finite":
        assert a > float(torch.finfo(torch.bfloat16).max)
    call(B, p)
    torch.cuda.synchronize()
    B.moe_check_device_status(p["ws"])
    assert p["idx"].cpu().tolist() == [[e]] * T
    out, tol, _, _ = reference(p)
    got = p["out"].cpu().double()
    if end == "infinite":
        # 0 times infinity is a NaN; the shared expert's part is zero
        w2 = p["w2"][2][e, :, f]
        want = torch.where(w2 == 0, torch.full_like(w2, math.nan), torch.sign(w2) * math.inf)
        assert torch.equal(got[0].isnan(), want.isnan())
        assert torch.equal(got[0][~want.isnan()], want[~want.isnan()])
        got, out, tol = got[1:], out[1:], tol[1:]
    err = (got - out).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("T", [1, 3, 9])
@pytest.mark.parametrize("H", [384, 5120])
def test_weights_of_cancelling_channels(B, T, H):
    """Two channels of +-4096 cancel in every logit: the choice and its weights are binary64's, rounded
    once (a binary64 sum of H products is off by H * 2^-53 of their magnitudes, about 2^-30 here)."""
    p = make(B, "bf16", T, H, 32, 4, 128, seed=79 + T)
    for a, b in ((8, 9), (40, 300), (H - 1, H - 7)):
        p["x"][:, a] = 4096.0
        p["x"][:, b] = -4096.0
        p["w_router"][:, b] = p["w_router"][:, a]
    call(B, p)
    torch.cuda.synchronize()
    x, wr = p["x"].cpu().double(), p["w_router"].cpu().double()
    slack = float(H * 2.0 ** -53 * (x.abs() @ wr.abs().T).max())
    assert slack < 2.0 ** -28
    _, _, idx, w = reference(p)
    assert torch.equal(p["idx"].cpu(), idx)
    # d(score)/score is at most d(logit), once more in the sum
    err = (p["w"].cpu().double() - w).abs()
    assert bool((err <= (2.0 ** -24 + 2 * slack + 2.0 ** -48) * w).all()), float((err / w).max())


@pytest.mark.parametrize("H", [256, 5120])
def test_permuted_router_rows_tie(B, H):
    """Experts whose products are the same in another order have equal keys: the lower ones are chosen."""
    p = make(B, "bf16", 2, H, 32, 5, 128, bias=torch.zeros(32, device="cuda"), seed=83)
    g = torch.Generator(device="cuda").manual_seed(89)
    row = p["w_router"][0].clone()
    for e in range(32):
        p["w_router"][e] = row[torch.randperm(H, generator=g, device="cuda")]
    p["x"][0] = 171.0 / 128.0
    p["x"][1] = -201.0 / 128.0
    call(B, p)
    torch.cuda.synchronize()
    assert p["idx"].cpu().tolist() == [[0, 1, 2, 3, 4]] * 2
    assert bool((p["w"] == p["w"][0, 0]).all())


@pytest.mark.parametrize("norm", [True, False])
def test_a_token_whose_scores_all_vanish(B, norm):
    """Every logit below -709, where a score underflows to zero in binary64: equal weights with
    norm_topk_prob, as moe_forward has them, zero without; the other tokens as ever."""
    p = make(B, "bf16", 3, 256, 32, 4, 128, bias=torch.zeros(32, device="cuda"), seed=97, n_shared=0,
             norm_topk_prob=norm)
    p["w_router"][:, 0] = -1.0
    p["x"][1] = 0
    p["x"][1, 0] = 1024.0
    call(B, p)
    torch.cuda.synchronize()
    assert p["idx"][1].cpu().tolist() == [0, 1, 2, 3]
    assert p["w"][1].cpu().tolist() == ([0.25] * 4 if norm else [0.0] * 4)
    c = p["cfg"]
    ws, out = B.alloc_workspace(c), torch.empty_like(p["out"])
    B.moe_forward(c, p["x"], p["w_router"], p["bias"], p["w13"][0], p["w2"][0], None, None, out, ws)
    torch.cuda.synchronize()
    assert torch.equal(B.ws_view(ws, c, "topk_idx"), p["idx"])
    a, b = p["out"].double(), out.double()
    assert bool(a.isfinite().all()) and float((a - b).norm() / b.norm()) <= 1e-2


@pytest.mark.parametrize("kind", ["fp8", "mxfp4"])
def test_weights_in_torchs_own_types(B, kind):
    """e4m3 weights, e2m1 codes and e8m0 scales as tensors of those types, and addresses: the same bits."""
    p = make(B, kind, 2, 256, 32, 2, 128, seed=103)
    call(B, p)
    first = p["out"].clone()
    p["out"].zero_()
    code = torch.float8_e4m3fn if kind == "fp8" else torch.float4_e2m1fn_x2
    for n in ("w13", "w2", "w13s", "w2s"):
        q, s, v = p[n]
        p[n] = (q.view(code), s if kind == "fp8" else s.view(torch.float8_e8m0fnu), v)
    bias, p["bias"] = p["bias"], p["bias"].data_ptr()
    call(B, p)
    torch.cuda.synchronize()
    assert torch.equal(p["out"], first)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [2, 7])
def test_outputs_near_the_small_end(B, kind, T):
    """Tokens so small that the outputs come near 2^-110: as exact as ever (and a binary32 sum of n terms
    loses up to n halves of its smallest step, 2^-149, which is 2^-133 where the sums are held 2^-16
    lower)."""
    H, I = 512, 128
    p = make(B, kind, T, H, 32, 2, I, seed=107)
    p["w_router"].zero_()
    p["x"][0] *= 2.0 ** -54
    call(B, p)
    torch.cuda.synchronize()
    B.moe_check_device_status(p["ws"])
    out, tol, idx, _ = reference(p)
    assert torch.equal(p["idx"].cpu(), idx)
    assert 2.0 ** -116 < float(out[0].abs().max()) < 2.0 ** -100
    err = (p["out"].cpu().double() - out).abs()
    tol = tol + 3 * I * 2.0 ** -133 if kind != "bf16" else tol + 3 * I * 2.0 ** -149
    assert bool((err <= tol).all()), float((err / tol).max())
