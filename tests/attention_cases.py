"""Which form of the attention's kernels a call takes (the library's rules over again,
so that a test can ask whether the cases reach every form), cases that do, and the
bias gradient's definition with a bound that its fp32 sums keep."""
import math

import torch

from attention_reference import F8, buckets

BF, HF, F4 = torch.bfloat16, torch.float16, torch.float32


def cdiv(a, b):
    return -(-a // b)


def forms(dtype, B, n, m, H, K, d, dv, bias, mask):
    """Set of (kernel, type, padded width, bias) a forward and backward call runs,
    and of ("refill", kernel, bytes of a row) where a wave passes over more than
    the 64 mask words that it forms at the start."""
    size = 4 if dtype == F4 else 2
    width = max(d, dv)
    dp = 64 if width <= 64 else 128 if width <= 128 else 256
    row = dp * size
    key = (dtype, dp, bias)
    out = set()
    few = n <= 32 or (d <= 64 and dv <= 64 and B * H * cdiv(n, 128) <= 64)
    waves = 8 if row <= 128 else 4
    turn = waves * 32 if few else 256
    items = B * K * cdiv(H // K * n, 32) if few else B * H * cdiv(n, 128)
    s = cdiv(256, items)
    if few:
        s = 1 if m <= 2 * turn else max(s, cdiv(m, 32 * turn))
    s = max(1, min(s, 64, m // turn))
    keys = cdiv(cdiv(m, s), turn) * turn
    if cdiv(m, keys) > 1:
        out.add(("merge", dtype))
    kernel = "rows" if few else "narrow" if row <= 128 else "wide"
    out.add((kernel,) + key)
    tiles = min(keys, m) // (turn if few else 32 if row > 256 else 64)
    # the wide form starts with the words of 128 tiles
    if mask and tiles > (128 if kernel == "wide" else 64):
        out.add(("refill", kernel, row))
    alone = row <= 256 and B * H * cdiv(n, 128) < 256
    out.add(("q alone" if alone else "q shared",) + key)
    if mask and (m // 128 if alone else m // (32 if row > 256 else 64)) > 64:
        out.add(("refill", "q alone" if alone else "q shared", row))
    most = 256 if row <= 128 or dtype == F4 else 64
    alone = row <= 256 and B * K * cdiv(m, 128) < most
    out.add(("kv alone" if alone else "kv shared",) + key)
    split = max(1, min(256 // (B * K * cdiv(m, 32 if alone else 128)), 16, n // 256))
    if cdiv(n, cdiv(cdiv(n, split), 128) * 128) > 1:
        out.add(("kv merge", dtype))
    return out


def all_forms():
    out = set()
    for dtype in (BF, HF, F4):
        size = 4 if dtype == F4 else 2
        out |= {("merge", dtype), ("kv merge", dtype)}
        for dp in (64, 128) + (() if dtype == F4 else (256,)):
            for bias in (False, True):
                key = (dtype, dp, bias)
                out |= {(x,) + key for x in ("rows", "q shared", "kv shared")}
                out.add(("narrow" if dp * size <= 128 else "wide",) + key)
                if dp * size <= 256:
                    out |= {("q alone",) + key, ("kv alone",) + key}
    for row in (128, 256, 512):
        out |= {("refill", "rows", row), ("refill", "q shared", row),
                ("refill", "narrow" if row == 128 else "wide", row)}
        if row <= 256:
            out.add(("refill", "q alone", row))
    return out


# type, B, n, m, H, K, d, dv, copies of the heads, options
WIDTHS = [(BF, 64, 64), (BF, 128, 96), (BF, 256, 200), (HF, 40, 64), (HF, 96, 128), (HF, 192, 256),
          (F4, 48, 64), (F4, 128, 100)]
FORMS = []
for _i, (_t, _d, _v) in enumerate(WIDTHS):
    for _bias in (None, (16, 40, _i % 2 == 0)):
        _opt = {"mask": True, "ragged": True, "buckets": _bias,
                "causal": bool(_bias) and _i % 2 == 1}
        FORMS += [(_t, 2, 5, 300, 4, 2, _d, _v, 1, _opt),
                  (_t, 2, 150, 170, 4, 2, _d, _v, 1, _opt),
                  (_t, 2, 150, 140, 4, 2, _d, _v, 32, _opt)]
SPLIT = [(t, 1, n, m, 2, 1, d, d, 1, {"mask": True, "buckets": b}) for t, n, m, d, b in (
    (BF, 600, 2100, 128, None), (HF, 1100, 130, 64, (8, 30, True)), (F4, 600, 700, 100, None),
    (HF, 140, 2100, 200, None), (BF, 600, 300, 40, (8, 30, False)))]
# masks of more words than are formed at the start; few of the rows see few keys
LONG = [(BF, 1, 40, 4400, 2, 1, 64, 64, 128, {"mask": True}),
        (HF, 1, 40, 4400, 2, 1, 128, 128, 128, {"mask": True}),
        (F4, 1, 40, 8300, 2, 1, 64, 64, 128, {"mask": True}),
        (BF, 1, 40, 4400, 2, 2, 256, 256, 128, {"mask": True}),
        (BF, 1, 40, 9000, 2, 1, 128, 128, 1, {"mask": True}),
        (HF, 1, 3, 9000, 2, 1, 64, 64, 1, {"mask": True})]
LONG_ROWS = [(BF, 1, 3, 1060000, 2, 1, 64, 64, 1, {"mask": True}),
             (HF, 1, 3, 535000, 2, 1, 128, 128, 1, {"mask": True}),
             (BF, 1, 1, 535000, 2, 1, 256, 256, 1, {"mask": True})]


def case_forms(case):
    t, B, n, m, H, K, d, dv, copies, opt = case
    return forms(t, B, n, m, H * copies, K * copies, d, dv, bool(opt.get("buckets")),
                 bool(opt.get("mask")))


def case_id(case):
    return "-".join(str(x) for x in case[:9]).replace("torch.", "") + \
        ("-bias" if case[9].get("buckets") else "")


def case_inputs(case, seed=0):
    from streaming_sinkhorn_solver_amd import binding

    dtype, B, n, m, H, K, d, dv, copies, opt = case
    g = torch.Generator().manual_seed(seed + 31 * n + m + d)
    rand = lambda *s: torch.randn(*s, generator=g)
    q, k, v = (rand(*s).to(dtype) for s in ((B, n, H, d), (B, m, K, d), (B, m, K, dv)))
    d_o = (rand(B, n, H, dv) * 0.1).to(dtype)
    d_lse = rand(B, H, n) * 0.1
    kw = {"causal": bool(opt.get("causal"))}
    if kw["causal"]:
        kw["offsets"] = torch.randint(-3, max(m - n, 0) + 4, (B,), generator=g, dtype=torch.int32)
    if opt.get("ragged"):
        kw["kv_len"] = torch.tensor([m] + [m - m // 3] * (B - 1), dtype=torch.int32)
        kw["q_len"] = torch.tensor([n] + [n - n // 4] * (B - 1), dtype=torch.int32)
    if opt.get("mask"):
        kw["key_mask"] = (torch.rand(B, m, generator=g) > 0.3).to(torch.uint8)
    if opt.get("buckets"):
        side, far, both = opt["buckets"]
        kw.update(edges=binding.fs_bucket_edges(side, far), two_sided=both,
                  bias=rand(side * (2 if both else 1), H))
    return q, k, v, d_o, d_lse, kw


def bias_gradient(q, k, v, d_o, d_lse, *, bias, edges, two_sided, scale=None, causal=False, offset=0,
                  offsets=None, q_len=None, kv_len=None, key_mask=None, stored_o=False):
    """d_bias and a bound on what a call may be off by.  The sum over a row's keys of
    P dP that enters every dS is an fp32 sum there, whatever the type of o: with
    w = 2^-24, weights off by e = 2 es + 8 w relative (es as in
    attention_reference), dP by w (dv + 4) |d_o|.|v|, and R = |d_o|.|o| + |d_lse|
    (the size of what the sum is refined from), it is off by
      e (sum P |dP| + R) + sum P b_dP + w (m + 4) sum P (|dP| + R) + 4 w (|D| + R).
    stored_o: the gradient of a call that takes the sum from o rounded to q's type
    instead (what the bound has to tell from the right one)."""
    w = 2.0 ** -24
    u = torch.finfo(q.dtype).eps / 2
    B, n, H, d = q.shape
    m, K, dv = k.shape[1], k.shape[2], v.shape[3]
    scale = d ** -0.5 if scale is None else scale
    val, bound = torch.zeros(bias.shape, dtype=F8), torch.zeros(bias.shape, dtype=F8)
    rows, cols = torch.arange(n), torch.arange(m)
    for b in range(B):
        off = int(offsets[b]) if offsets is not None else offset
        rel = cols[None] - rows[:, None] - off
        seen = torch.ones(n, m, dtype=torch.bool)
        if kv_len is not None:
            seen &= (cols < int(kv_len[b]))[None]
        if q_len is not None:
            seen &= (rows < int(q_len[b]))[:, None]
        if key_mask is not None:
            seen &= (key_mask[b] != 0)[None]
        if causal:
            seen &= rel <= 0
        at = buckets(rel, list(edges), two_sided)
        some = seen.any(1)
        for h in range(H):
            g = h // (H // K)
            Q, Kk, V, dO = q[b, :, h].to(F8), k[b, :, g].to(F8), v[b, :, g].to(F8), d_o[b, :, h].to(F8)
            s = torch.where(seen, Q @ Kk.t() * scale + bias[:, h].to(F8)[at], -math.inf)
            s = torch.where(some[:, None], s, 0.0)
            P = torch.where(some[:, None], torch.softmax(s, 1), 0.0)
            fin = torch.where(torch.isfinite(s), s.abs(), 0.0).amax(1)
            es = w * (d + 16) * (Q.abs() @ Kk.abs().t()).amax(1) * scale + 8 * w * (1 + fin)
            e = (2 * es + 8 * w)[:, None]
            gl = torch.where(some, d_lse[b, h].to(F8), 0.0)[:, None]
            O, dP = P @ V, dO @ V.t()
            D = (dO * (O.to(q.dtype).to(F8) if stored_o else O)).sum(1, keepdim=True) - gl
            R = (dO.abs() * O.abs()).sum(1, keepdim=True) * (1 + 2 * u) + gl.abs()
            bP = w * (dv + 4) * (dO.abs() @ V.abs().t())
            size = (P * dP.abs()).sum(1, keepdim=True) + R
            bD = e * size + (P * bP).sum(1, keepdim=True) + w * (m + 4) * size + 4 * w * (D.abs() + R)
            dS = P * (dP - D)
            bS = P * (bP + bD + 2 * w * (dP.abs() + D.abs())) + (e + w * (n + m + 64)) * dS.abs()
            val[:, h].index_add_(0, at.reshape(-1), dS.reshape(-1))
            bound[:, h].index_add_(0, at.reshape(-1), bS.reshape(-1))
    return val, bound + w * val.abs() + 1e-30


def coherent(dtype, n=3, m=40):
    """Inputs whose rounded o shows in delta: every element of a row of o is the
    same number, so all are rounded the same way."""
    g = torch.Generator().manual_seed(5)
    B, H, d = 2, 4, 16
    q, k = ((torch.randn(B, r, H, d, generator=g) * 0.3).to(dtype) for r in (n, m))
    v = (1 + torch.rand(B, m, H, 1, generator=g)).expand(-1, -1, -1, d).to(dtype)
    d_o = torch.full((B, n, H, d), 0.125, dtype=dtype)
    kw = {"bias": torch.randn(6, H, generator=g) * 0.3, "edges": [2, 9], "two_sided": True}
    return q, k, v, d_o, torch.randn(B, H, n, generator=g) * 0.1, kw
