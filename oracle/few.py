"""64-bit references of the few-token layer, of MXFP4 and of the norms around
a block, with the error bounds their tests use.

Plain torch in float64 on the CPU, straight from the formulas in
include/moe.h.  A bound next to a result is derived from the operations that
the definition allows to round: every binary32 sum of n terms is off by at
most n * 2^-23 of the sum of its terms' magnitudes (an adder may truncate),
and what is stored is off by half a step of its type, torch.finfo(t).eps / 2.
"""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -23
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- MXFP4
def mx_quantize(x: torch.Tensor):
    """x [R, C] -> (codes uint8 [R, C/2], scale uint8 [R, C/32]), value by value."""
    R, C = x.shape
    q = torch.zeros((R, C), dtype=torch.uint8)
    s = torch.zeros((R, C // 32), dtype=torch.uint8)
    for r in range(R):
        for b in range(C // 32):
            v = [float(a) for a in x[r, 32 * b:32 * b + 32]]
            if any(math.isnan(a) or math.isinf(a) for a in v):
                s[r, b] = 255
                continue
            amax = max(abs(a) for a in v)
            e = 127 if amax == 0.0 else max(math.frexp(amax)[1] - 1 - 2 + 127, 0)
            s[r, b] = e
            for i, a in enumerate(v):
                m = abs(a) * 2.0 ** (127 - e)
                best = min(range(8), key=lambda c: (abs(E2M1[c] - m), c & 1))
                q[r, 32 * b + i] = best | (8 if math.copysign(1.0, a) < 0 else 0)
    return q[:, 0::2] | (q[:, 1::2] << 4), s


def mx_values(q: torch.Tensor, s: torch.Tensor) -> torch.Tensor:
    """The float64 values of MXFP4 codes [..., C/2] and scales [..., C/32]."""
    tab = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64)
    v = torch.stack((tab[(q & 15).long()], tab[(q >> 4).long()]), -1).flatten(-2)
    f = torch.where(s == 255, torch.full(s.shape, math.nan, dtype=torch.float64),
                    torch.exp2(s.double() - 127.0))
    return v * f.repeat_interleave(32, -1)


def fp8_values(q: torch.Tensor, s: torch.Tensor) -> torch.Tensor:
    """The float64 values of e4m3 codes [..., R, C] and 128 x 128 block scales."""
    return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(
        128, -1).repeat_interleave(128, -2)


# ---------------------------------------------------------------- few-token layer
def choose(logits, bias, k, n_group=1, topk_group=1, group_topn=2, norm=True, rsf=1.0):
    """(idx, w) of float64 logits [T, E]: keys sigmoid + bias, NaN below numbers,
    ties to the lower index."""
    T, E = logits.shape
    score = 1.0 / (1.0 + torch.exp(-logits))
    key = score + bias.double()
    key = torch.where(torch.isnan(key), torch.full_like(key, -math.inf), key)
    idx = torch.zeros((T, k), dtype=torch.int32)
    w = torch.zeros((T, k), dtype=torch.float64)
    n = E // n_group
    for t in range(T):
        allowed = list(range(E))
        if n_group > 1:
            total = []
            for g in range(n_group):
                best = sorted((float(v) for v in key[t, g * n:(g + 1) * n]), reverse=True)
                total.append(sum(best[:group_topn]))
            keep = sorted(range(n_group), key=lambda g: (-total[g], g))[:topk_group]
            allowed = [e for g in sorted(keep) for e in range(g * n, (g + 1) * n)]
        order = sorted(allowed, key=lambda e: (-float(key[t, e]), e))[:k]
        idx[t] = torch.tensor(order, dtype=torch.int32)
        s = score[t, order]
        w[t] = (s / s.sum() if norm else s) * rsf
    return idx, w


def _swiglu(x, w13, w2):
    """(values, error bound before the last rounding) of W2 (SiLU(g) u)."""
    I = w2.shape[1]
    ax = x.abs()
    g, u = (x @ w13.T).split(I, 1)
    eg, eu = (U32 * x.shape[1] * (ax @ w13.abs().T)).split(I, 1)
    silu = g / (1.0 + torch.exp(-g))
    a = silu * u
    # |SiLU'| < 1.1; a few binary32 operations; the activations' 16 bits
    ea = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + a.abs() * (8 * U32 + 2.0 ** -16)
    return a @ w2.T, (ea + U32 * I * a.abs()) @ w2.abs().T


def layer(x, w_router, bias, w13, w2, w13s, w2s, k, **route):
    """The layer for x [T, H] (all float64; w13[e] and w2[e] index experts).
    Returns (out, bound, idx, w)."""
    idx, w = choose(x @ w_router.T, bias, k, **route)
    out, err = torch.zeros_like(x), torch.zeros_like(x)
    if w13s is not None:
        out, err = _swiglu(x, w13s, w2s)
    mag = out.abs().clone()
    for t in range(x.shape[0]):
        for j in range(k):
            e = int(idx[t, j])
            v, d = _swiglu(x[t:t + 1], w13[e], w2[e])
            out[t] += w[t, j] * v[0]
            err[t] += w[t, j].abs() * (d[0] + 2.0 ** -22 * v[0].abs())
            mag[t] += w[t, j].abs() * v[0].abs()
    return out, err + U32 * 64 * mag + HALF_BF16 * (out.abs() + err), idx, w


# ---------------------------------------------------------------- norms around a block
def norm_residual(h, y, gamma_post, gate, a, eps, gamma_pre):
    """(h', u, rp, rq, and the bounds of h' and u), float64; u None without gamma_pre."""
    H = h.shape[1]
    rp = 1.0 / torch.sqrt((y * y).mean(1, keepdim=True) + eps)
    n = gate * gamma_post * y * rp
    h2 = a * h + n
    rel = H * U32                          # of a norm's sum of squares, all terms positive
    e2 = 8 * U32 * ((a * h).abs() + n.abs()) + rel * n.abs()
    rq = 1.0 / torch.sqrt((h2 * h2).mean(1, keepdim=True) + eps)
    out = {"h_out": h2, "rp": rp[:, 0], "rq": rq[:, 0],
           "h_tol": e2 + HALF_BF16 * (h2.abs() + e2)}
    if gamma_pre is not None:
        u = gamma_pre * h2 * rq
        # rq's relative error: half of the mean square's, whose terms carry 2 |h'| e2
        er = rq * rq * (h2.abs() * e2).mean(1, keepdim=True) + rel
        eu = gamma_pre.abs() * rq * (e2 + h2.abs() * (er + 8 * U32))
        out.update(u=u, u_tol=eu + HALF_BF16 * (u.abs() + eu))
    return out


def norm_residual_backward(h, y, gamma_post, gate, a, gamma_pre, rp, rq, dh_out, du):
    """Gradients in float64 and their bounds; gate broadcasts over rows or not.
    dgate is left per token."""
    H = h.shape[1]
    yn = y * rp[:, None]
    w = gate * gamma_post * yn
    mean = lambda v: v.mean(1, keepdim=True)  # noqa: E731
    rel = H * U32
    if gamma_pre is not None:
        hn = (a * h + w) * rq[:, None]
        ehn = 8 * U32 * ((a * h).abs() + w.abs()) * rq[:, None]
        q = du * gamma_pre
        c1 = mean(q * hn)
        ec1 = rel * mean((q * hn).abs()) + mean(q.abs() * ehn)
        D = dh_out + rq[:, None] * (q - hn * c1)
        eD = (8 * U32 * (dh_out.abs() + rq[:, None] * (q.abs() + (hn * c1).abs())) +
              rq[:, None] * (ehn * c1.abs() + hn.abs() * ec1))
        # the three-sum form of mean(p yn) adds up these magnitudes
        mag = mean((w * (dh_out.abs() + rq[:, None] * q.abs())).abs()) + \
            rq[:, None] * (c1.abs() + ec1) * mean((w * hn).abs()) + \
            rq[:, None] * (ec1 / rel + c1.abs()) * mean(w.abs() * hn.abs())
    else:
        hn = ehn = torch.zeros_like(h)
        D, eD = dh_out, torch.zeros_like(h)
        mag = mean((w * dh_out).abs())
    p = D * gate * gamma_post
    c2 = mean(p * yn)
    ec2 = (rel + 16 * U32) * mag + mean((gate * gamma_post * yn).abs() * eD)
    dy = rp[:, None] * (p - yn * c2)
    edy = rp[:, None] * ((gate * gamma_post).abs() * eD + 8 * U32 * (p.abs() + (yn * c2).abs()) +
                         yn.abs() * ec2)
    res = {"dh": (a * D, abs(a) * eD + 4 * U32 * (a * D).abs()), "dy": (dy, edy),
           "dgate": (D * gamma_post * yn, (gamma_post * yn).abs() * (eD + 8 * U32 * D.abs()))}
    T = h.shape[0]
    term = D * gate * yn
    eterm = (gate * yn).abs() * (eD + 8 * U32 * D.abs())
    res["dgamma_post"] = (term.sum(0), eterm.sum(0) + T * U32 * term.abs().sum(0))
    if gamma_pre is not None:
        term = du * hn
        res["dgamma_pre"] = (term.sum(0), (du.abs() * (ehn + 8 * U32 * hn.abs())).sum(0) +
                             T * U32 * term.abs().sum(0))
    return res
