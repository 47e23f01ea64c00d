"""Cases of the few-token MoE layer, the MXFP4 weight format it can read, and the norms around the
block with their gate and residual scale: inputs, plain forms and 64-bit results.

A case names its operator in ``op``:

  few        the whole MoE layer for a few tokens (weights bf16, e4m3 with 128 x 128 block scales, or MXFP4)
  mxfp4      weights to MXFP4 (blocks of 32 along a row) and back to bf16
  norm       residual update with the block output's norm, gate and residual scale, then the next pre-norm
  norm_bwd   its gradients
"""
import math

import numpy as np
import torch

own = False

FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # e2m1 magnitudes, code bit 3 is the sign
EPS = 1e-6                                       # the norm epsilon of the workloads


# ---------------------------------------------------------------------------------------------- cases
def _few(name, T, weights="bf16", H=5120, E=256, k=8, I=1536, n_shared=1, n_group=1, topk_group=1,
         norm=True, rsf=1.0):
    return {"name": name, "op": "few", "T": T, "H": H, "E": E, "k": k, "I": I, "n_shared": n_shared,
            "n_group": n_group, "topk_group": topk_group, "norm": norm, "rsf": rsf,
            "weights": weights}


def listed():
    return [
        # the test layer's size, one token: nothing but latency
        _few("few_tiny_t1", 1, H=512, E=32, k=4, I=128),
        # one user decoding on the flagship layer: nine experts' weights
        _few("few_decode_t1", 1),
        # a small batch of users on the same layer, the largest the operator takes
        _few("few_decode_t16", 16),
        # the group-limited layer with two shared experts, an odd batch
        _few("few_grouped_t5", 5, H=4096, E=128, k=6, I=1408, n_shared=2, n_group=8, topk_group=4,
             rsf=2.5),
        # one user on the FP8 checkpoint
        _few("few_fp8_t1", 1, weights="fp8"),
        # a few users on 4-bit weights
        _few("few_mxfp4_t4", 4, weights="mxfp4"),
        # a checkpoint load: the down projections of 32 experts
        {"name": "mxfp4_w2_32_experts", "op": "mxfp4", "rows": 32 * 5120, "cols": 1536},
        # one small matrix with an odd number of rows
        {"name": "mxfp4_small", "op": "mxfp4", "rows": 333, "cols": 512},
        # the block boundary of a decode step
        {"name": "norm_decode_t4", "op": "norm", "T": 4, "H": 5120, "gate": "channel", "res": 1.0},
        # the same of an 8192-token prefill, with a gate for each token
        {"name": "norm_prefill", "op": "norm", "T": 8192, "H": 5120, "gate": "token", "res": 1.0},
        # training on the same batch, a learned gate for each channel
        {"name": "norm_bwd_train", "op": "norm_bwd", "T": 8192, "H": 5120, "gate": "channel",
         "res": 1.0},
        # a ragged batch of the second layer, token gates, a scaled residual
        {"name": "norm_bwd_ragged", "op": "norm_bwd", "T": 777, "H": 4096, "gate": "token",
         "res": 0.75},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("few", "few", "few", "mxfp4", "norm", "norm_bwd"))
    if op == "few":
        E = rng.choice((32, 64, 96, 128, 160, 192, 256))
        n_group = rng.choice((1, 1, 4, 8))
        topk_group = 1 if n_group == 1 else rng.randint(2, n_group)
        k = min(_log(rng, 1, 8), topk_group * (E // n_group))
        return {"op": "few", "T": _log(rng, 1, 16), "H": 128 * _log(rng, 1, 40), "E": E, "k": k,
                "I": 128 * _log(rng, 1, 12), "n_shared": rng.randint(0, 2), "n_group": n_group,
                "topk_group": topk_group, "norm": rng.random() < 0.8,
                "rsf": rng.choice((1.0, 2.5)), "weights": rng.choice(("bf16", "fp8", "mxfp4"))}
    if op == "mxfp4":
        return {"op": "mxfp4", "rows": _log(rng, 1, 160000), "cols": 32 * _log(rng, 1, 48)}
    return {"op": op, "T": _log(rng, 1, 8192), "H": 8 * _log(rng, 8, 640),
            "gate": rng.choice(("none", "channel", "token")), "res": rng.choice((1.0, 0.75, 0.5))}


# ---------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std


def _bf16(g, *shape, std=1.0):
    return _randn(g, *shape, std=std).to(torch.bfloat16)


def _to_fp8(w):
    """e4m3 codes and one fp32 scale for each 128 x 128 block (sizes are multiples of 128)."""
    R, C = w.shape
    b = w.view(R // 128, 128, C // 128, 128)
    amax = b.abs().amax(dim=(1, 3))
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    q = (b / scale[:, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(R, C).view(torch.uint8), scale


def _to_mxfp4(w):
    """e2m1 codes (two to a byte, the lower column in the low half) and e8m0 scales of 32 columns."""
    R, C = w.shape
    b = w.float().view(R, C // 32, 32)
    amax = b.abs().amax(dim=2)
    e = torch.frexp(amax).exponent - 1                       # floor(log2 amax)
    code = torch.where(amax > 0, e - 2 + 127, torch.full_like(e, 127)).clamp(0, 254)
    v = (b.double() * torch.exp2(127.0 - code.double())[:, :, None]).view(R, C)
    a = v.abs()
    # round to nearest, ties to the even code: borders between neighbouring magnitudes
    m = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) +
         (a >= 3.5) + (a > 5.0))
    c = m.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    return c[:, 0::2] | (c[:, 1::2] << 4), code.to(torch.uint8)


def _matrix(case, g, n, rows, cols):
    """n weight matrices [rows, cols] ~ N(0, 0.02^2) in the case's format: (stored, scales or None)."""
    kind = case["weights"]
    if kind == "bf16":
        w = torch.empty((n, rows, cols), dtype=torch.bfloat16, device="cuda")
        for i in range(n):
            w[i] = _randn(g, rows, cols, std=0.02)
        return w, None
    if kind == "fp8":
        w = torch.empty((n, rows, cols), dtype=torch.uint8, device="cuda")
        s = torch.empty((n, rows // 128, cols // 128), device="cuda")
        pack = _to_fp8
    else:
        w = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device="cuda")
        s = torch.empty((n, rows, cols // 32), dtype=torch.uint8, device="cuda")
        pack = _to_mxfp4
    for i in range(n):
        w[i], s[i] = pack(_randn(g, rows, cols, std=0.02))
    return w, s


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "few":
        T, H, E, I, ns = case["T"], case["H"], case["E"], case["I"], case["n_shared"]
        d = {"x": _bf16(g, T, H), "w_router": _bf16(g, E, H, std=0.02),
             "bias": torch.rand((E,), generator=g, device="cuda") * 0.2 - 0.1}
        d["w13"], d["w13_scale"] = _matrix(case, g, E, 2 * I, H)
        d["w2"], d["w2_scale"] = _matrix(case, g, E, H, I)
        d["w13s"] = d["w13s_scale"] = d["w2s"] = d["w2s_scale"] = None
        if ns:
            for name, rows, cols in (("w13s", 2 * ns * I, H), ("w2s", H, ns * I)):
                w, s = _matrix(case, g, 1, rows, cols)
                d[name], d[name + "_scale"] = w[0], None if s is None else s[0]
        return d
    if op == "mxfp4":
        return {"w": _bf16(g, case["rows"], case["cols"], std=0.02)}
    T, H = case["T"], case["H"]
    d = {"h": _bf16(g, T, H, std=2.0), "y": _bf16(g, T, H, std=0.5),
         "gamma_post": (1.0 + _randn(g, H, std=0.1)).to(torch.bfloat16),
         "gamma_pre": (1.0 + _randn(g, H, std=0.1)).to(torch.bfloat16), "gate": None}
    if case["gate"] != "none":
        shape = (H,) if case["gate"] == "channel" else (T, H)
        d["gate"] = torch.sigmoid(_randn(g, *shape)).to(torch.bfloat16)
    if op == "norm_bwd":
        d["dh_out"], d["du"] = _bf16(g, T, H), _bf16(g, T, H)
        # the reciprocal norms that the forward pass has left
        h, y = d["h"].double(), d["y"].double()
        r_post = (y.square().mean(1) + EPS).rsqrt()
        n = y * r_post[:, None] * d["gamma_post"].double()
        h2 = case["res"] * h + (n if d["gate"] is None else n * d["gate"].double())
        d["rstd"] = torch.stack((r_post, (h2.square().mean(1) + EPS).rsqrt())).float()
    return d


def prepare(case, seed):
    st = {"case": case, **_inputs(case, seed)}
    if not own:
        return st
    from sigmoid_top_routing_warp_b200 import binding as B
    st["B"] = B
    op = case["op"]
    if op == "few":
        T, k = case["T"], case["k"]
        dtype = {"bf16": B.MOE_DTYPE_BF16, "fp8": B.MOE_DTYPE_FP8_E4M3_BLOCK128,
                 "mxfp4": B.MOE_DTYPE_MXFP4_BLOCK32}[case["weights"]]
        cfg = B.MoeConfig(T=T, H=case["H"], E=case["E"], k=k, I=case["I"],
                          n_shared=case["n_shared"], n_group=case["n_group"],
                          topk_group=case["topk_group"], norm_topk_prob=case["norm"],
                          routed_scaling_factor=case["rsf"], dtype=dtype)
        st["ws"] = B.alloc_few_workspace(cfg)
        st["out"] = torch.empty((T, case["H"]), dtype=torch.bfloat16, device="cuda")
        st["idx"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        st["w"] = torch.empty((T, k), device="cuda")
    elif op == "mxfp4":
        R, C = case["rows"], case["cols"]
        cfg = None
        st["q"] = torch.empty((R, C // 2), dtype=torch.uint8, device="cuda")
        st["s"] = torch.empty((R, C // 32), dtype=torch.uint8, device="cuda")
        st["back"] = torch.empty((R, C), dtype=torch.bfloat16, device="cuda")
    else:
        T, H = case["T"], case["H"]
        cfg = B.MoeConfig(T=T, H=H, E=32, k=1, I=128)
        st["mode"] = {"none": B.MOE_GATE_NONE, "channel": B.MOE_GATE_CHANNEL,
                      "token": B.MOE_GATE_TOKEN}[case["gate"]]
        if op == "norm":
            st["h_out"], st["u"] = torch.empty_like(st["h"]), torch.empty_like(st["h"])
            st["rstd"] = torch.empty((2, T), device="cuda")
        else:
            st["ws"] = B.alloc_norm_residual_workspace(cfg)
            st["dh"], st["dy"] = torch.empty_like(st["h"]), torch.empty_like(st["h"])
            st["dgate"] = None
            if case["gate"] == "channel":
                st["dgate"] = torch.empty((H,), device="cuda")
            elif case["gate"] == "token":
                st["dgate"] = torch.empty_like(st["gate"])
            st["dgamma_post"] = torch.empty((H,), device="cuda")
            st["dgamma_pre"] = torch.empty((H,), device="cuda")
    st["cfg"] = cfg
    return st


# ---------------------------------------------------------------------------------------------- plain forms
def _unpack(w, s, kind):
    """Stored matrix [rows, ...] -> the fp32 values it stands for."""
    if kind == "bf16":
        return w.float()
    if kind == "fp8":
        return w.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, 0).repeat_interleave(
            128, 1)
    table = torch.tensor(FP4 + tuple(-v for v in FP4), device=w.device)
    v = torch.stack((table[(w & 15).int()], table[(w >> 4).int()]), 2).view(w.shape[0], -1)
    return v * torch.exp2(s.float() - 127.0).repeat_interleave(32, 1)


def _route(case, x, w_router, bias):
    """(idx, w): the choice in 64 bits, ties to the lower expert."""
    T, E, k, G = case["T"], case["E"], case["k"], case["n_group"]
    s = 1.0 / (1.0 + torch.exp(-(x.double() @ w_router.double().T)))
    key = s + bias.double()
    if G > 1:
        best = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values[:, :, :2].sum(2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices
        keep = torch.zeros((T, G), dtype=torch.bool, device=x.device)
        keep.scatter_(1, order[:, :case["topk_group"]], True)
        key = torch.where(keep.repeat_interleave(E // G, 1), key, torch.full_like(key, -math.inf))
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, idx)
    if case["norm"]:
        w = w / w.sum(1, keepdim=True)
    return idx, (w * case["rsf"]).float()


def _swiglu(x, w13, w2):
    g, u = (x @ w13.T).chunk(2, dim=1)
    return (g / (1.0 + torch.exp(-g)) * u) @ w2.T


def _plain_few(st):
    case, kind = st["case"], st["case"]["weights"]
    idx, w = _route(case, st["x"], st["w_router"], st["bias"])
    x = st["x"].float()
    out = torch.zeros_like(x)
    if case["n_shared"]:
        out = _swiglu(x, _unpack(st["w13s"], st["w13s_scale"], kind),
                      _unpack(st["w2s"], st["w2s_scale"], kind))

    def expert(name, e):
        s = st[name + "_scale"]
        return _unpack(st[name].index_select(0, e)[0],
                       None if s is None else s.index_select(0, e)[0], kind)

    for t in range(case["T"]):
        for j in range(case["k"]):
            e = idx[t, j:j + 1]
            out[t:t + 1] += w[t, j] * _swiglu(x[t:t + 1], expert("w13", e), expert("w2", e))
    return out.to(torch.bfloat16), idx.int(), w


def _plain_mxfp4(st):
    q, s = _to_mxfp4(st["w"])
    return _unpack(q, s, "mxfp4").to(torch.bfloat16), s


def _plain_norm(st):
    case = st["case"]
    h, y = st["h"].float(), st["y"].float()
    r_post = 1.0 / torch.sqrt(y.square().mean(1) + EPS)
    n = y * r_post[:, None] * st["gamma_post"].float()
    h2 = case["res"] * h + (n if st["gate"] is None else st["gate"].float() * n)
    r_pre = 1.0 / torch.sqrt(h2.square().mean(1) + EPS)
    u = h2 * r_pre[:, None] * st["gamma_pre"].float()
    return h2.to(torch.bfloat16), u.to(torch.bfloat16), torch.stack((r_post, r_pre))


def _plain_norm_bwd(st):
    case = st["case"]
    h, y, du = st["h"].float(), st["y"].float(), st["du"].float()
    gp, gq = st["gamma_post"].float(), st["gamma_pre"].float()
    gate = torch.ones_like(gp) if st["gate"] is None else st["gate"].float()
    rp, rq = st["rstd"][0][:, None], st["rstd"][1][:, None]
    yn = y * rp
    hn = (case["res"] * h + gate * (yn * gp)) * rq
    q = du * gq
    D = st["dh_out"].float() + rq * (q - hn * (q * hn).mean(1, keepdim=True))
    p = D * gate * gp
    dy = rp * (p - yn * (p * yn).mean(1, keepdim=True))
    out = [(case["res"] * D).to(torch.bfloat16), dy.to(torch.bfloat16),
           (D * gate * yn).double().sum(0).float(), (du * hn).double().sum(0).float()]
    if case["gate"] == "channel":
        out.append((D * gp * yn).double().sum(0).float())
    elif case["gate"] == "token":
        out.append((D * gp * yn).to(torch.bfloat16))
    return out


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"few": _plain_few, "mxfp4": _plain_mxfp4, "norm": _plain_norm,
                "norm_bwd": _plain_norm_bwd}[op](st)
    B, cfg = st["B"], st["cfg"]
    if op == "few":
        B.moe_forward_few(cfg, st["x"], st["w_router"], st["bias"], st["w13"], st["w2"],
                          st["w13s"], st["w2s"], st["out"], st["ws"], topk_idx=st["idx"],
                          topk_w=st["w"], w13_scale=st["w13_scale"], w2_scale=st["w2_scale"],
                          w13s_scale=st["w13s_scale"], w2s_scale=st["w2s_scale"])
        return st["out"], st["idx"], st["w"]
    if op == "mxfp4":
        B.moe_quantize_mx(st["w"], st["q"], st["s"])
        B.moe_dequantize_mx(st["q"], st["s"], st["back"])
        return st["back"], st["s"]
    if op == "norm":
        B.moe_norm_residual(cfg, st["h"], st["y"], st["gamma_post"], st["h_out"], EPS,
                            gate=st["gate"], gate_mode=st["mode"], res_scale=st["case"]["res"],
                            gamma_pre=st["gamma_pre"], u=st["u"], rstd=st["rstd"])
        return st["h_out"], st["u"], st["rstd"]
    B.moe_norm_residual_backward(cfg, st["h"], st["y"], st["gamma_post"], st["rstd"], st["dh_out"],
                                 st["dh"], st["dy"], st["dgamma_post"], st["ws"], gate=st["gate"],
                                 gate_mode=st["mode"], res_scale=st["case"]["res"],
                                 gamma_pre=st["gamma_pre"], du=st["du"],
                                 dgamma_pre=st["dgamma_pre"], dgate=st["dgate"])
    out = [st["dh"], st["dy"], st["dgamma_post"], st["dgamma_pre"]]
    return out if st["dgate"] is None else out + [st["dgate"]]


# ---------------------------------------------------------------------------------------------- work
def _touched(case):
    """Experts that a batch of this case touches, on average: a seeded simulation of the inputs'
    distribution (logits of variance 0.02^2 H, biases uniform in +-0.1)."""
    T, E, k, G = case["T"], case["E"], case["k"], case["n_group"]
    rng = np.random.default_rng(0)
    counts = []
    for _ in range(16):
        s = 1.0 / (1.0 + np.exp(-rng.standard_normal((T, E)) * 0.02 * math.sqrt(case["H"])))
        key = s + rng.uniform(-0.1, 0.1, E)
        if G > 1:
            top2 = np.sort(key.reshape(T, G, E // G), axis=2)[:, :, -2:].sum(2)
            drop = np.argsort(top2, axis=1)[:, :G - case["topk_group"]]
            for t in range(T):
                key.reshape(T, G, E // G)[t, drop[t]] = -math.inf
        counts.append(len(np.unique(np.argsort(key, axis=1)[:, E - k:])))
    return sum(counts) / len(counts)


def work(case):
    op = case["op"]
    if op == "few":
        T, H, E, k, I, ns = (case[n] for n in ("T", "H", "E", "k", "I", "n_shared"))
        per = {"bf16": 2.0, "fp8": 1.0 + 4.0 / 128 ** 2, "mxfp4": 0.5 + 1.0 / 32}[case["weights"]]
        experts = _touched(case) + ns
        return {"bytes": experts * 3 * H * I * per + E * H * 2 + E * 4 + T * H * 4 + T * k * 8,
                "flops": 2.0 * T * ((k + ns) * 3 * H * I + E * H)}
    if op == "mxfp4":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 + 2 + 2 * (0.5 + 1.0 / 32)), "flops": 6.0 * n}
    n, H = case["T"] * case["H"], case["H"]
    gate = {"none": 0, "channel": 0, "token": n}[case["gate"]]
    vec = H if case["gate"] == "channel" else 0
    if op == "norm":
        return {"bytes": 2 * (4 * n + gate + vec + 2 * H) + 8 * case["T"], "flops": 12.0 * n}
    return {"bytes": 2 * (6 * n + 2 * gate + vec + 2 * H) + 8 * case["T"] + 4 * (2 * H + vec),
            "flops": 30.0 * n}


# ---------------------------------------------------------------------------------------------- 64 bits
def _exact_matrix(w, s, kind):
    if kind == "bf16":
        return w.double()
    if kind == "fp8":
        R, C = w.shape
        v = w.view(torch.float8_e4m3fn).double().view(R // 128, 128, C // 128, 128)
        return (v * s.double().view(R // 128, 1, C // 128, 1)).view(R, C)
    nib = torch.stack((w.bitwise_and(15), w.bitwise_right_shift(4)), dim=-1).flatten(1).long()
    mag = nib % 8
    # e2m1 by its fields: 2^(e-1) (1 + m/2), or m/2 for e = 0
    e, m = (mag // 2).double(), (mag % 2).double()
    v = torch.where(e > 0, torch.exp2(e - 1.0) * (1.0 + 0.5 * m), 0.5 * m)
    v = torch.where(nib >= 8, -v, v).view(w.shape[0], -1, 32)
    return (v * torch.exp2(s.double() - 127.0)[:, :, None]).view(w.shape[0], -1)


def _exact_few(case, d):
    T, E, k, G, kind = case["T"], case["E"], case["k"], case["n_group"], case["weights"]
    logits = (d["x"].double() @ d["w_router"].double().T).cpu().numpy()
    score = 1.0 / (1.0 + np.exp(-logits))
    key = score + d["bias"].cpu().numpy().astype(np.float64)
    idx, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        allowed = range(E)
        if G > 1:
            n = E // G
            total = [sum(sorted(key[t, a * n:(a + 1) * n])[-2:]) for a in range(G)]
            best = sorted(range(G), key=lambda a: (-total[a], a))[:case["topk_group"]]
            allowed = [e for a in best for e in range(a * n, (a + 1) * n)]
        chosen = sorted(allowed, key=lambda e: (-key[t, e], e))[:k]
        idx[t], w[t] = chosen, score[t, chosen]
        if case["norm"]:
            w[t] /= w[t].sum()
        w[t] *= case["rsf"]
    x = d["x"].double()
    out = torch.zeros_like(x)

    def add(tokens, coef, w13, w2):
        rows = x[tokens]
        half = w13.shape[0] // 2
        gate, up = rows @ w13[:half].T, rows @ w13[half:].T
        out[tokens] += coef[:, None] * ((gate * torch.sigmoid(gate) * up) @ w2.T)

    def values(name, e=None):
        s = d[name + "_scale"]
        return _exact_matrix(d[name] if e is None else d[name][e],
                             s if e is None or s is None else s[e], kind)

    if case["n_shared"]:
        every = torch.arange(T, device="cuda")
        add(every, torch.ones(T, device="cuda", dtype=torch.float64), values("w13s"), values("w2s"))
    for e in sorted(set(idx.ravel().tolist())):
        ts, js = np.nonzero(idx == e)
        add(torch.as_tensor(ts, device="cuda"), torch.as_tensor(w[ts, js], device="cuda"),
            values("w13", e), values("w2", e))
    return out, torch.as_tensor(idx, device="cuda"), torch.as_tensor(w, device="cuda")


def _exact_mxfp4(d):
    x = d["w"].double()
    R, C = x.shape
    b = x.view(R, C // 32, 32)
    top = b.abs().amax(2, keepdim=True)
    code = torch.where(top > 0, torch.floor(torch.log2(top)) + 125.0, torch.full_like(top, 127.0))
    # log2 next to a power of two may round across it
    code = torch.where((top > 0) & (torch.exp2(code - 125.0) > top), code - 1.0, code)
    code = torch.where((top > 0) & (torch.exp2(code - 124.0) <= top), code + 1.0, code)
    code = code.clamp(0.0, 254.0)
    scale = torch.exp2(code - 127.0)
    a = (b / scale).abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).double()
    v = (torch.round(a / step) * step).clamp(max=6.0)          # torch.round: ties to even
    return (torch.copysign(v, b) * scale).view(R, C), code.view(R, C // 32).to(torch.uint8)


def _exact_norm(case, d):
    h, y = d["h"].double(), d["y"].double()
    inv = lambda v: torch.rsqrt(torch.mean(v * v, dim=1, keepdim=True) + EPS)  # noqa: E731
    gate = 1.0 if d["gate"] is None else d["gate"].double()
    r1 = inv(y)
    h2 = h * case["res"] + gate * d["gamma_post"].double() * y * r1
    r2 = inv(h2)
    return h2, d["gamma_pre"].double() * h2 * r2, torch.cat((r1, r2), 1).T.contiguous()


def _exact_norm_bwd(case, d):
    """By the quotient rule, with the squared norms written out."""
    H = case["H"]
    h, y = d["h"].double(), d["y"].double()
    gp, gq = d["gamma_post"].double(), d["gamma_pre"].double()
    gate = torch.ones_like(h) if d["gate"] is None else d["gate"].double().expand_as(h)
    r1, r2 = d["rstd"].double()[0][:, None], d["rstd"].double()[1][:, None]
    h2 = h * case["res"] + gate * gp * y * r1
    du = d["du"].double()
    g2 = gq * du
    D = d["dh_out"].double() + g2 * r2 - h2 * (r2 ** 3 / H) * (g2 * h2).sum(1, keepdim=True)
    g1 = gate * gp * D
    dy = g1 * r1 - y * (r1 ** 3 / H) * (g1 * y).sum(1, keepdim=True)
    out = [D * case["res"], dy, (D * gate * y * r1).sum(0), (du * h2 * r2).sum(0)]
    if case["gate"] != "none":
        dgate = D * gp * y * r1
        out.append(dgate.sum(0) if case["gate"] == "channel" else dgate)
    return out


def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"] == "few":
        return _exact_few(case, d)
    if case["op"] == "mxfp4":
        return _exact_mxfp4(d)
    return _exact_norm(case, d) if case["op"] == "norm" else _exact_norm_bwd(case, d)
