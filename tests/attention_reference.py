"""The attention's definition in 64 bits on the CPU, with a bound on how far
each output of a call in 32 or 16 bits may be off.

Bounds.  u is half a step of the element type (eps / 2), w = 2^-24 that of
fp32.  A score is a sum of d products in fp32, then a multiplication and an
exponential whose argument may be off by as much as the score is:
es = w (d + 16) max_j sum_t |q_t k_t| scale + 8 w (1 + max_j |s|) relative in
every weight, 2 es after division by their sum.  Weights and dS enter their
product rounded to the element type (u relative each; fp16: 2^-31 of the
row's sum absolute in the forward pass, 2^-38 in the backward pass and 2^-24
of the column's largest dS, below which fp16's numbers end).  Sums of N terms in fp32:
w N of the sum of magnitudes (a bound for any order).  Every output is rounded
once more (u)."""
import math

import torch

F8 = torch.float64


def buckets(r, edges, two_sided):
    dist = r.abs() if two_sided else (-r).clamp(min=0)
    c = torch.zeros_like(r)
    for e in edges:
        c += dist >= e
    return c + (r > 0) * (len(edges) + 1) if two_sided else c


def reference(q, k, v, *, scale=None, causal=False, offset=0, offsets=None, q_len=None, kv_len=None,
              key_mask=None, bias=None, edges=None, two_sided=True, d_o=None, d_lse=None):
    """Outputs and bounds: dict of name -> (value, bound), gradients if d_o is given."""
    u = torch.finfo(q.dtype).eps / 2
    w = 2.0 ** -24
    half = q.dtype == torch.float16
    if q.dtype == torch.float32:
        u = w
    B, n, H, d = q.shape
    m, K, dv = k.shape[1], k.shape[2], v.shape[3]
    scale = d ** -0.5 if scale is None else scale
    edges = list(edges) if edges is not None else []
    z = lambda *s: torch.zeros(*s, dtype=F8)
    out = {"o": (z(B, n, H, dv), z(B, n, H, dv)), "lse": (z(B, H, n), z(B, H, n))}
    grad = d_o is not None
    if grad:
        for name, t in (("d_q", q), ("d_k", k), ("d_v", v)):
            out[name] = (z(*t.shape), z(*t.shape))
        if bias is not None:
            out["d_bias"] = (z(*bias.shape), z(*bias.shape))
    for b in range(B):
        off = int(offsets[b]) if offsets is not None else offset
        rows, cols = torch.arange(n), torch.arange(m)
        seen = torch.ones(n, m, dtype=torch.bool)
        if kv_len is not None:
            seen &= (cols < int(kv_len[b]))[None]
        if key_mask is not None:
            seen &= (key_mask[b] != 0)[None]
        if q_len is not None:
            seen &= (rows < int(q_len[b]))[:, None]
        rel = cols[None] - rows[:, None] - off
        if causal:
            seen &= rel <= 0
        used_k, used_q = seen.any(0), seen.any(1)
        bk = buckets(rel, edges, two_sided) if bias is not None else None
        for h in range(H):
            g = h // (H // K)
            zero = lambda t, use: torch.where(use[:, None], t.to(F8), torch.zeros((), dtype=F8))
            Q, Kk, V = zero(q[b, :, h], used_q), zero(k[b, :, g], used_k), zero(v[b, :, g], used_k)
            s = Q @ Kk.t() * scale
            mag = (Q.abs() @ Kk.abs().t()) * scale
            if bias is not None:
                t = bias[:, h].to(F8)
                t = torch.where(t <= -1e30, torch.full_like(t, -math.inf), t)
                s = s + t[bk]
            s = torch.where(seen, s, torch.full_like(s, -math.inf))
            some = torch.isfinite(s).any(1) if m else torch.zeros(n, dtype=torch.bool)
            ss = torch.where(some[:, None], s, torch.zeros_like(s))
            L = torch.logsumexp(ss, 1) if m else torch.zeros(n, dtype=F8)
            P = torch.where(some[:, None], torch.exp(ss - L[:, None]), torch.zeros_like(ss))
            fin = torch.where(torch.isfinite(s), s.abs(), torch.zeros_like(s))
            if m:
                es = w * (d + 16) * mag.amax(1) + 8 * w * (1 + fin.amax(1))
            else:
                es = z(n)
            O = P @ V
            PV = P @ V.abs()
            lost = 2.0 ** -31 * V.abs().sum(0)[None] if half else 0.0
            bo = (u + 2 * es[:, None] + w * m) * PV + u * O.abs() + lost + 1e-30
            if half:
                bo = bo + 2.0 ** -25  # fp16 output below its normal range
            out["o"][0][b, :, h], out["o"][1][b, :, h] = O, bo
            out["lse"][0][b, h] = torch.where(some, L, torch.full_like(L, -math.inf))
            out["lse"][1][b, h] = es + w * m + 4 * w * (1 + L.abs())
            if not grad:
                continue
            dO = zero(d_o[b, :, h], used_q & some)
            gl = z(n) if d_lse is None else torch.where(some, d_lse[b, h].to(F8), z(n))
            dP = dO @ V.t()
            D = (dO * O).sum(1) - gl
            dS = P * (dP - D[:, None])
            # delta is formed from the stored o: its bound and the sum's
            bD = (dO.abs() * bo).sum(1) + w * (dv + 4) * (dO.abs() * O.abs()).sum(1) + 2 * w * gl.abs()
            bdP = w * (dv + 4) * (dO.abs() @ V.abs().t())
            bdS = P * (bdP + bD[:, None]) + (2 * es[:, None] + 6 * w) * dS.abs()
            rS = bdS + u * dS.abs()
            lostk = dS.abs().amax(0)[None] * 2.0 ** -24 if half and n else 0.0
            lostq = dS.abs().amax(1)[:, None] * 2.0 ** -24 if half and m else 0.0
            tiny = 2.0 ** -25 if half else 1e-30
            dQ = scale * (dS @ Kk)
            bQ = scale * ((rS + lostq + w * m * dS.abs()) @ Kk.abs()) + u * dQ.abs() + tiny
            dK = scale * (dS.t() @ Q)
            bK = scale * ((rS + lostk + w * n * H * dS.abs()).t() @ Q.abs()) + tiny
            dV = P.t() @ dO
            bV = ((u + 2 * es[:, None] + w * n * H) * P + (2.0 ** -38 if half else 0.0)).t() @ dO.abs() + tiny
            out["d_q"][0][b, :, h], out["d_q"][1][b, :, h] = dQ, bQ
            out["d_k"][0][b, :, g] += dK
            out["d_k"][1][b, :, g] += bK
            out["d_v"][0][b, :, g] += dV
            out["d_v"][1][b, :, g] += bV
            if bias is not None:
                for i, x in ((0, dS), (1, bdS + w * (m + 64) * dS.abs())):
                    out["d_bias"][i][:, h] += torch.zeros(bias.shape[0], dtype=F8).index_add_(
                        0, bk.reshape(-1), x.reshape(-1))
    if grad:
        for name in ("d_k", "d_v"):
            out[name][1].add_(u * out[name][0].abs())
        if bias is not None:
            out["d_bias"][1].add_(w * out["d_bias"][0].abs() + 1e-30)
    return out


def check(name, got, ref):
    """got within the bound of ref = (value, bound) everywhere."""
    val, bound = ref
    got = got.detach().cpu().to(F8)
    assert got.shape == val.shape, name
    inf = torch.isinf(val)
    assert torch.equal(got[inf], val[inf]), f"{name}: infinities differ"
    err = torch.where(inf, torch.zeros_like(val), (got - val).abs())
    assert torch.isfinite(got[~inf]).all(), f"{name}: not finite"
    if err.numel() == 0:
        return 0.0
    worst = float((err / bound.clamp(min=1e-300)).max())
    assert worst <= 1.0, f"{name}: error is {worst:.2f} of its bound (max {float(err.max()):.3e})"
    return worst


def norm_reference(x, weight, cos, sin, pos, eps, interleaved, g=None):
    """y, and with g (the gradient of y) dx, dw: (value, bound) each.  Bounds:
    the mean of d squares in fp32 is off by w (d + 4) relative, the rest of the
    chain by a few w; sums over N rows by w N of the magnitudes' sum."""
    w = 2.0 ** -24
    u = w if x.dtype == torch.float32 else torch.finfo(x.dtype).eps / 2
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 1e-30
    B, n, H, d = x.shape
    X = x.to(F8)
    W = torch.ones(d, dtype=F8) if weight is None else weight.to(F8)
    inv = 1 / torch.sqrt((X * X).mean(-1, keepdim=True) + eps)
    rot = 0 if cos is None else 2 * cos.shape[1]
    p = torch.arange(rot // 2)
    a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)
    if rot:
        at = pos.clamp(0, cos.shape[0] - 1).long()
        C, S = cos.to(F8)[at][:, :, None], sin.to(F8)[at][:, :, None]

    def turn(z, back=False):
        y = z.clone()
        if rot:
            s = -S if back else S
            y[..., a] = z[..., a] * C - z[..., b] * s
            y[..., b] = z[..., b] * C + z[..., a] * s
        return y

    def spread(z):  # sum of magnitudes that a rotation mixes
        y = z.abs().clone()
        if rot:
            y[..., a] = z[..., a].abs() * C.abs() + z[..., b].abs() * S.abs()
            y[..., b] = z[..., b].abs() * C.abs() + z[..., a].abs() * S.abs()
        return y

    Z = X * inv * W
    y = turn(Z)
    e = w * (d + 16)
    out = {"y": (y, e * spread(Z) + u * y.abs() + tiny)}
    if g is None:
        return out
    G, bG = turn(g.to(F8), True), spread(g.to(F8))
    xw = X * W
    mean = (xw * G).mean(-1, keepdim=True)
    dx = inv * (W * G - X * inv * inv * mean)
    bound = inv * ((W * bG).abs() + (X * inv * inv).abs() * (xw.abs() * bG).mean(-1, keepdim=True))
    out["dx"] = (dx, 2 * e * bound + u * dx.abs() + tiny)
    N = B * n * H
    dw = (X * inv * G).sum((0, 1, 2))
    out["dw"] = (dw, (e + w * (min(N, 4096) + 8)) * (X.abs() * inv * bG).sum((0, 1, 2)) + w * dw.abs())
    return out
