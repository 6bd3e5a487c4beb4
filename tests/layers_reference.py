"""Definitions in 64 bits on the CPU of the operators of include/fs_layers.h, with
a bound on how far each output may be off.

Bounds.  u is half a step of an output's type (eps / 2), w = 2^-24 that of fp32,
tiny what a type's numbers end at (fp16: 2^-25).  A sum of N terms in fp32 is
off by w N of the sum of magnitudes at most (any order); where a row's lanes
add in parallel, N is the length of the longest chain of additions: CHAIN = 64
for the sums over a row (at most 32 elements a lane, or 64 groups of 8 in the
log-sum-exp's, six folds, 16 waves).  The base-2 exponential is off by 2 w."""
import math

import torch

F8, F4 = torch.float64, torch.float32
W = 2.0 ** -24
CHAIN = 64


def half_step(dtype):
    return W if dtype == F4 else torch.finfo(dtype).eps / 2


def tiny_of(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 1e-37


def inside(B, n, lengths):
    """[B, n, 1] truth values: rows that are no padding."""
    if lengths is None:
        return torch.ones(B, n, 1, dtype=torch.bool)
    return (torch.arange(n)[None] < lengths.clamp(0, n)[:, None].long())[..., None]


def norm_values(z, weight, bias, eps, seen):
    """y, mean, rstd in 64 bits from the definition (z of padding: zeros)."""
    mean = z.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((z - mean) ** 2).mean(-1, keepdim=True) + eps)
    return ((z - mean) * rstd * weight + bias) * seen, mean, rstd


def norm_reference(x, weight, bias, eps, residual=None, lengths=None, d_y=None, d_total=None):
    u, tiny = half_step(x.dtype), tiny_of(x.dtype)
    B, n, width = x.shape
    seen = inside(B, n, lengths)
    zero = torch.zeros((), dtype=F8)
    wt = torch.ones(width, dtype=F8) if weight is None else weight.to(F8)
    bs = torch.zeros(width, dtype=F8) if bias is None else bias.to(F8)
    out = {}
    z = x.to(F8)
    if residual is not None:
        # the sum that goes on is of the rows' type
        z = (x.float() + residual.float()).to(x.dtype).to(F8)
        z = torch.where(seen, z, zero)
        out["total"] = (z, torch.zeros_like(z))
    z = torch.where(seen, z, zero)
    y, mean, rstd = norm_values(z, wt, bs, eps, seen)
    far = z - mean
    em = W * (CHAIN + 2) * z.abs().mean(-1, keepdim=True)
    var = (far ** 2).mean(-1, keepdim=True)
    dvar = W * (CHAIN + 4) * var + 2 * em * far.abs().mean(-1, keepdim=True) + em ** 2
    er = dvar / (2 * (var + eps)) + 4 * W
    h = far * rstd
    eh = rstd * (em + W * far.abs()) + h.abs() * (er + 2 * W)
    out["y"] = (y, (wt.abs() * eh + 2 * W * ((wt * h).abs() + bs.abs()) + u * y.abs() + tiny) * seen)
    out["mean"] = ((mean * seen)[..., 0], ((em + W * mean.abs()) * seen)[..., 0] + 1e-37)
    out["rstd"] = ((rstd * seen)[..., 0], (rstd * (er + W) * seen)[..., 0])
    if d_y is None:
        return out
    g = torch.where(seen, d_y.to(F8), zero)
    v = wt * g
    m1, m2 = v.mean(-1, keepdim=True), (v * h).mean(-1, keepdim=True)
    e1 = W * (CHAIN + 4) * v.abs().mean(-1, keepdim=True)
    e2 = (v.abs() * (eh + W * (CHAIN + 6) * h.abs())).mean(-1, keepdim=True)
    d = rstd * (v - m1 - h * m2)
    bd = rstd * (e1 + h.abs() * e2 + eh * m2.abs() + 4 * W * (v.abs() + m1.abs() + (h * m2).abs()))
    bd = bd + d.abs() * (er + 2 * W)
    if d_total is not None:
        d = d + torch.where(seen, d_total.to(F8), zero)
    out["d_x"] = (d * seen, (bd + (W + u) * d.abs() + tiny) * seen)
    rows = B * n
    dw = (g * h).sum((0, 1))
    out["d_weight"] = (dw, (g.abs() * (eh + W * (rows + 8) * h.abs())).sum((0, 1)) + W * dw.abs() + 1e-37)
    db = g.sum((0, 1))
    out["d_bias"] = (db, W * (rows + 8) * g.abs().sum((0, 1)) + W * db.abs() + 1e-37)
    return out


def quantize_reference(x):
    """q and scale, exactly: ties of 127 x / a go to the even whole number.  254 |x|
    and (2 q + 1) a are exact in 64 bits for fp32 values."""
    X = x.to(F8)
    top = X.abs().amax(1) if x.shape[0] else X.new_zeros(0)
    bad = ~torch.isfinite(X).all(1)
    top = torch.where(bad, torch.zeros_like(top), top)[:, None]
    mag = torch.where(bad[:, None], torch.zeros_like(X), X.abs())
    q = torch.floor(mag * 127 / torch.where(top > 0, top, torch.ones_like(top)))
    for _ in range(2):  # the floor of a rounded quotient may be one off
        q = torch.where(127 * mag < q * top, q - 1, q)
        q = torch.where((127 * mag >= (q + 1) * top) & (top > 0), q + 1, q)
    twice, border = 254 * mag, (2 * q + 1) * top
    up = (twice > border) | ((twice == border) & (q % 2 == 1))
    q = torch.where((top > 0) & up, q + 1, q) * torch.sign(torch.where(bad[:, None], mag, X))
    scale = top[:, 0].float() / 127
    scale[bad] = math.nan
    return q.to(torch.int8), scale


def product_reference(q_x, scale_x, q_w, scale_w, dtype, bias=None):
    """The whole numbers' product is exact; it, its two products with the scales and
    the sum with the bias are rounded to fp32 each, y once more."""
    p = (q_x.long() @ q_w.long().t()).to(F8) * scale_x.to(F8)[:, None] * scale_w.to(F8)
    y = p if bias is None else p + bias.to(F8)
    return y, 3 * W * p.abs() + (W + half_step(dtype)) * y.abs() + tiny_of(dtype)


def distill_reference(x, ids, teacher, T, teacher_lse=None, active=None, d_loss=None):
    u, tiny = half_step(x.dtype), tiny_of(x.dtype)
    R, V = x.shape
    k = ids.shape[1]
    out = {"loss": (torch.zeros(R, dtype=F8), torch.zeros(R, dtype=F8)),
           "lse": (torch.zeros(R, dtype=F8), torch.zeros(R, dtype=F8))}
    if d_loss is not None:
        out["d_logits"] = (torch.zeros(R, V, dtype=F8), torch.zeros(R, V, dtype=F8))
    for r in range(R):
        if active is not None and not active[r]:
            continue
        z = x[r].to(F8) / T
        if not torch.isfinite(z).any():
            out["lse"][0][r] = -math.inf
            continue
        lse = torch.logsumexp(z, 0)
        p = torch.exp(z - lse)
        fin = z[torch.isfinite(z)]
        top, low = fin.max(), fin.min()
        e1 = W * (4 * torch.where(torch.isfinite(z), top - z, torch.zeros_like(z)) + 4)
        # a lane's chain, its changes of maximum (their exponents add up to the range)
        chain = V / 2048 * 8 + CHAIN
        el = float((p * e1).sum()) + W * (chain + 4 * (top - low) + 8 * 30)
        el_out = el + W * (4 * abs(top) + 2 * abs(lse))
        out["lse"][0][r], out["lse"][1][r] = lse, el_out
        real = (ids[r] >= 0) & (ids[r] < V) & (teacher[r] != -math.inf)
        if not real.any():
            continue
        at, t = ids[r][real].long(), teacher[r][real].to(F8) / T
        ref = torch.logsumexp(t, 0) if teacher_lse is None else teacher_lse[r].to(F8)
        lt = t - ref
        tau = torch.exp(lt)
        et = W * (8 * (t.abs().max() + abs(ref)) + k + 16)
        mass = tau.sum()
        have = z[at] - lse
        term = torch.where(tau > 0, tau * (lt - have), torch.zeros_like(tau))
        out["loss"][0][r] = T * T * term.sum()
        size = tau * (W * 8 * (t.abs() + abs(ref) + z[at].abs()) + el_out) + et * term.abs()
        out["loss"][1][r] = T * T * (size.sum() + W * (k + 8) * term.abs().sum()) + W * term.sum().abs() * T * T + 1e-37
        if d_loss is None:
            continue
        g = float(d_loss[r].to(F8)) * T
        hit = torch.zeros(V, dtype=F8).index_add_(0, at, tau)
        d = g * (mass * p - hit)
        ep = e1 + W * 8 * (z.nan_to_num(0, 0, 0).abs() + abs(lse)) + el_out + et
        size = abs(g) * (mass * p * (ep + 8 * W) + hit * (et + W * (k + 8)))
        out["d_logits"][0][r] = d
        out["d_logits"][1][r] = size + u * d.abs() + tiny
    return out


def balance_reference(x, k, normalize, lengths=None, d_loss=None, d_gates=None, ids=None):
    """ids: a choice made elsewhere (rows whose first is negative take no part)."""
    u, tiny = half_step(x.dtype), tiny_of(x.dtype)
    B, n, E = x.shape
    seen = inside(B, n, lengths)[..., 0]
    z = lambda *s: torch.zeros(*s, dtype=F8)
    own = ids is None
    if own:
        ids = torch.full((B, n, k), -1, dtype=torch.int32)
    gates, lse = (z(B, n, k), z(B, n, k)), (z(B, n), z(B, n))
    counts = torch.zeros(B, E, dtype=torch.int32)
    loss, dx = (z(B, 2), z(B, 2)), (z(B, n, E), z(B, n, E))
    for b in range(B):
        v = x[b].float()
        # NaN counts as -inf in the choice
        order = torch.where(torch.isnan(v), torch.full_like(v, -math.inf), v)
        on = seen[b] & (order.max(1).values != -math.inf if own else ids[b, :, 0] >= 0)
        rows = on.nonzero()[:, 0]
        N = len(rows)
        if N == 0:
            continue
        X = x[b, rows].to(F8)
        if own:
            ids[b, rows] = torch.sort(order[rows], dim=1, descending=True,
                                      stable=True)[1][:, :k].to(torch.int32)
        pick = ids[b, rows].long()
        L = torch.logsumexp(X, 1, keepdim=True)
        p = torch.exp(X - L)
        top = X.amax(1, keepdim=True)
        far = torch.where(torch.isfinite(X), top - X, torch.zeros_like(X))
        el = (p * W * (4 * far + CHAIN)).sum(1, keepdim=True) + W * (2 * top.abs() + 4 * L.abs() + 4)
        ep = W * (4 * far + 8) + W * 4 * (X.nan_to_num(0, 0, 0).abs() + L.abs()) + el
        chosen, ec = p.gather(1, pick), ep.gather(1, pick)
        S = chosen.sum(1, keepdim=True)
        es = (chosen * ec).sum(1, keepdim=True) / S + W * (k + 8)
        gate = chosen / S if normalize else chosen
        eg = ec + es + 4 * W if normalize else ec + 2 * W
        gates[0][b, rows], gates[1][b, rows] = gate, gate * eg + 1e-37
        lse[0][b, rows], lse[1][b, rows] = L[:, 0], el[:, 0] + W * L[:, 0].abs()
        c = torch.bincount(pick.flatten(), minlength=E)
        counts[b] = c.to(torch.int32)
        f = c.to(F8) / (k * N)
        loss[0][b, 0] = E * (f * p.mean(0)).sum()
        loss[1][b, 0] = E * (f * (p * (ep + W * (N + 8))).mean(0)).sum() + W * loss[0][b, 0]
        loss[0][b, 1] = (L ** 2).mean()
        loss[1][b, 1] = (2 * L.abs() * el + W * (N + 8) * L ** 2).mean() + W * loss[0][b, 1]
        if d_loss is None:
            continue
        g0, g1 = d_loss[b].to(F8)
        even = (g0 * E * f / N).expand(N, E)
        dp, size = even.clone(), 12 * W * even.abs()
        if d_gates is not None:
            dg = d_gates[b, rows].to(F8)
            bg = W * 4 * dg.abs()
            if normalize:
                mid = (dg * gate).sum(1, keepdim=True)
                bm = ((dg * gate).abs() * (eg + W * (k + CHAIN))).sum(1, keepdim=True)
                bg = (bg + bm + (dg - mid).abs() * (es + 8 * W) + 4 * W * mid.abs()) / S
                dg = (dg - mid) / S
            dp = dp.scatter_add(1, pick, dg)
            size = size.scatter_add(1, pick, bg + W * (k + 4) * dg.abs())
        mean = (p * dp).sum(1, keepdim=True)
        bmean = (p * ((ep + W * (CHAIN + 8)) * dp.abs() + size)).sum(1, keepdim=True)
        sq = 2 * g1 * L / N
        d = p * (dp - mean + sq)
        bd = p * (size + bmean + 8 * W * (dp.abs() + mean.abs() + sq.abs()) + (2 * g1 / N).abs() * el)
        dx[0][b, rows] = d
        dx[1][b, rows] = bd + d.abs() * (ep + 4 * W + u) + tiny
    out = {"ids": ids, "counts": counts, "gates": gates, "lse": lse, "loss": loss}
    if d_loss is not None:
        out["d_logits"] = dx
    return out
