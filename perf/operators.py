"""Timed cases of the attention operators: attention between two sets of
states (forward, backward, single tokens), the learned relative position bias
by buckets inside it, and the per-head norm of queries and keys with the
position rotation.

``run`` computes a case either from elementary torch operations in 32 bits
(``own`` false) or through the library's entry points (``own`` true);
``exact`` gives the same outputs in 64 bits from the definitions.

Definitions (batch b, query row i, key row j, head h; key head h // (H / K)):
  s_ij = scale q_i.k_j + T[c(j - i - off_b), h],
  L_i = log sum_j exp s_ij,  O_i = sum_j exp(s_ij - L_i) v_j  (j visible);
  c(r) = (edges <= |r|) + (E + 1) [r > 0] two-sided, (edges <= max(-r, 0)) else;
  norm and rotation: y = R(position) (w x / sqrt(mean x^2 + eps)).
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_EPS = 1e-6


def _attn(name, op, B, n, m, H, K, d, dtype, dv=0, ragged=False, mask=False, causal=False,
          buckets=0, max_dist=0, two_sided=False):
    return {"name": name, "op": op, "B": B, "n": n, "m": m, "H": H, "K": K, "d": d,
            "dv": dv or d, "dtype": dtype, "ragged": ragged, "mask": mask, "causal": causal,
            "buckets": buckets, "max_dist": max_dist, "two_sided": two_sided}


def _norm(name, op, B, n, H, K, d, dtype, rot=0, interleaved=False):
    return {"name": name, "op": op, "B": B, "n": n, "H": H, "K": K, "d": d, "dtype": dtype,
            "rot": rot or d, "interleaved": interleaved}


def listed():
    return [
        # one token against a short encoded sentence, small model: latency
        _attn("token_short", "attn", 4, 1, 512, 8, 8, 64, "bf16"),
        # one token against a long encoded document, grouped heads: the read of the cache
        _attn("token_long", "attn", 8, 1, 32768, 32, 8, 128, "bf16", ragged=True),
        # a few speculative tokens, an odd head size, scattered padding
        _attn("tokens_few", "attn", 2, 5, 1777, 12, 12, 80, "fp16", mask=True),
        # prompt of a decoder against padded encodings of another length
        _attn("encode_mid", "attn", 8, 512, 1500, 16, 16, 64, "bf16", ragged=True),
        # long prompt against a long document, grouped heads
        _attn("encode_large", "attn", 2, 4096, 8192, 32, 8, 128, "bf16"),
        # a training step of a small model, odd lengths, padding
        _attn("train_mid", "attn_train", 8, 333, 777, 12, 4, 64, "fp16", ragged=True, mask=True),
        # a training step at full size
        _attn("train_large", "attn_train", 2, 2048, 4096, 32, 8, 128, "bf16"),
        # descriptors of two clouds in the solver's own type
        _attn("train_fp32", "attn_train", 2, 500, 700, 8, 8, 48, "fp32"),
        # one token of a decoder with a learned position bias, each sequence at its own length
        _attn("bias_token", "attn", 8, 1, 2049, 16, 16, 64, "bf16", ragged=True, causal=True,
              buckets=32, max_dist=128),
        # a training step of an encoder with a learned position bias
        _attn("bias_train", "attn_train", 4, 2048, 2048, 16, 16, 64, "bf16", buckets=32,
              max_dist=128, two_sided=True),
        # queries and keys of one token of a batch: latency
        _norm("norm_token", "norm", 32, 1, 32, 8, 128, "bf16"),
        # queries and keys of a training step
        _norm("norm_train", "norm_train", 4, 4096, 32, 8, 128, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["token", "attn", "attn", "train", "train", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    K = rng.choice([1, 2, 4, 8])
    H = K * rng.choice([1, 1, 2, 4])
    if kind.startswith("norm"):
        d = rng.choice([32, 64, 80, 96, 128, 256])
        rot = rng.choice([d, d, d // 2])
        return {"op": kind, "B": _log_int(rng, 1, 8), "n": _log_int(rng, 1, 4096), "H": H,
                "K": K, "d": d, "dtype": dtype, "rot": rot,
                "interleaved": rng.random() < 0.4}
    d = rng.choice([32, 40, 64, 64, 72, 96, 128, 128] + ([192, 256] if dtype != "fp32" else []))
    dv = d if rng.random() < 0.8 else rng.choice([32, 64, 128])
    B = _log_int(rng, 1, 8)
    causal, buckets, max_dist, two_sided = False, 0, 0, False
    if kind == "token":
        n, m = rng.choice([1, 1, 1, 2, 4, 7]), _log_int(rng, 100, 32768)
        if dtype == "fp32":
            m = min(m, 8192)
    else:
        n, m = _log_int(rng, 16, 4096), _log_int(rng, 16, 8192)
        if dtype == "fp32":
            n, m = min(n, 1024), min(m, 2048)
    if rng.random() < 0.5:
        buckets = rng.choice([8, 16, 32, 64])
        max_dist = rng.choice([64, 128, 500])
        two_sided = rng.random() < 0.5
        causal = not two_sided
        if causal and kind != "token":
            m = max(n, m)
    # no more pairs than the largest listed case
    while B * H * n * m * (d + dv) * (3 if kind == "train" else 1) > 2 ** 38 and B > 1:
        B -= 1
    while B * H * n * m * (d + dv) * (3 if kind == "train" else 1) > 2 ** 38:
        n = max(1, n // 2)
    return {"op": "attn_train" if kind == "train" else "attn", "B": B, "n": n, "m": m, "H": H,
            "K": K, "d": d, "dv": dv, "dtype": dtype, "ragged": rng.random() < 0.5,
            "mask": rng.random() < 0.3, "causal": causal, "buckets": buckets,
            "max_dist": max_dist, "two_sided": two_sided}


# ---- inputs --------------------------------------------------------------

def _edges(buckets, max_dist, two_sided):
    """Distances at which a new bucket starts: half of a side's buckets one
    distance each, the rest spaced evenly in the logarithm up to max_dist
    (whole-number arithmetic: no rounding at a border)."""
    side = buckets // 2 if two_sided else buckets
    first = side // 2
    rest = side - first
    out = []
    for u in range(1, side):
        if u <= first:
            out.append(u)
            continue
        k = u - first
        bound = first ** (rest - k) * max_dist ** k
        lo, hi = 0, max_dist
        while lo < hi:
            mid = (lo + hi) // 2
            if mid ** rest >= bound:
                hi = mid
            else:
                lo = mid + 1
        out.append(lo)
    return out


def _lengths(case):
    """Key lengths of the sequences, longest first, down to about a half."""
    if not case["ragged"]:
        return [case["m"]] * case["B"]
    return [max(1, case["m"] - (b * case["m"]) // (2 * case["B"])) for b in range(case["B"])]


def _offsets(case, lens):
    """Key position of query row 0: the queries are the last rows."""
    if not case["causal"]:
        return [0] * len(lens)
    return [max(x - case["n"], 0) for x in lens]


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g = _generator(seed)
    t = _TYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=t):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)

    B, n, H, K, d = (case[x] for x in ("B", "n", "H", "K", "d"))
    s = {"case": case}
    if case["op"].startswith("norm"):
        s["q"], s["k"] = normal(B, n, H, d, std=1.7), normal(B, n, K, d, std=1.3)
        s["qw"] = 1 + normal(d, std=0.2, dtype=torch.float32)
        s["kw"] = 1 + normal(d, std=0.2, dtype=torch.float32)
        table = 8192
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        ang = torch.arange(table, device="cuda", dtype=torch.float64)[:, None] * freq[None, :]
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        start = torch.randint(0, table - n + 1, (B, 1), generator=g, device="cuda")
        s["pos"] = (start + torch.arange(n, device="cuda")[None, :]).to(torch.int32)
        if case["op"] == "norm_train":
            s["dqo"], s["dko"] = normal(B, n, H, d, std=0.1), normal(B, n, K, d, std=0.1)
        if own:
            s["out"] = _norm_outputs(s)
        return s
    m, dv = case["m"], case["dv"]
    s["q"], s["k"], s["v"] = normal(B, n, H, d), normal(B, m, K, d), normal(B, m, K, dv)
    lens = _lengths(case)
    order = torch.randperm(B, generator=torch.Generator().manual_seed(seed)).tolist()
    lens = [lens[x] for x in order]
    s["kv_len"] = (torch.tensor(lens, dtype=torch.int32, device="cuda")
                   if case["ragged"] else None)
    s["off"] = (torch.tensor(_offsets(case, lens), dtype=torch.int32, device="cuda")
                if case["causal"] else None)
    s["mask"] = None
    if case["mask"]:
        # scattered padding; the first key stays
        s["mask"] = (torch.rand(B, m, generator=g, device="cuda") > 0.15).to(torch.uint8)
        s["mask"][:, 0] = 1
    s["bias"] = s["edges"] = None
    if case["buckets"]:
        s["edges"] = _edges(case["buckets"], case["max_dist"], case["two_sided"])
        s["bias"] = normal(case["buckets"], H, std=0.7, dtype=torch.float32)
    if case["op"] == "attn_train":
        s["do"] = normal(B, n, H, dv, std=0.05)
    if own:
        s["out"] = _attn_outputs(s)
    return s


def _attn_outputs(s):
    """Output and workspace buffers, as a program keeps them over its steps."""
    from streaming_sinkhorn_solver_amd import binding

    c = s["case"]
    q, v = s["q"], s["v"]
    train = c["op"] == "attn_train"
    out = {"o": q.new_empty(c["B"], c["n"], c["H"], c["dv"]),
           "lse": torch.empty(c["B"], c["H"], c["n"], device="cuda"),
           "ws": torch.empty(binding.fs_attention_workspace_bytes(
               q, s["k"], v, edges=s["edges"], backward=train),
               dtype=torch.uint8, device="cuda")}
    if train:
        out["dq"], out["dk"], out["dv"] = (torch.empty_like(x) for x in (q, s["k"], v))
        out["dbias"] = None if s["bias"] is None else torch.empty_like(s["bias"])
    return out


def _norm_outputs(s):
    from streaming_sinkhorn_solver_amd import binding

    out = {"q": torch.empty_like(s["q"]), "k": torch.empty_like(s["k"])}
    if s["case"]["op"] == "norm_train":
        out["dq"], out["dk"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        out["dqw"], out["dkw"] = torch.empty_like(s["qw"]), torch.empty_like(s["kw"])
        out["ws"] = torch.empty(binding.fs_qk_norm_workspace_bytes(s["q"], s["k"]),
                                dtype=torch.uint8, device="cuda")
    return out


# ---- one pass ------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if op.startswith("norm"):
        return _norm_own(state) if own else _norm_plain(state)
    return _attn_own(state) if own else _attn_plain(state)


def _attn_own(s):
    from streaming_sinkhorn_solver_amd import binding

    c, out = s["case"], s["out"]
    kw = dict(kv_len=s["kv_len"], key_mask=s["mask"], causal=c["causal"], offsets=s["off"],
              bias=s["bias"], edges=s["edges"], two_sided=c["two_sided"], workspace=out["ws"])
    binding.fs_attention_forward(s["q"], s["k"], s["v"], out["o"], out["lse"], **kw)
    if c["op"] == "attn":
        return out["o"], out["lse"]
    binding.fs_attention_backward(s["q"], s["k"], s["v"], out["o"], out["lse"], s["do"],
                                  out["dq"], out["dk"], out["dv"], d_bias=out["dbias"], **kw)
    res = (out["o"], out["lse"], out["dq"], out["dk"], out["dv"])
    return res if s["bias"] is None else res + (out["dbias"],)


def _norm_own(s):
    from streaming_sinkhorn_solver_amd import binding

    c, out = s["case"], s["out"]
    kw = dict(eps=_EPS, cos=s["cos"], sin=s["sin"], positions=s["pos"],
              interleaved=c["interleaved"])
    binding.fs_qk_norm_rotate(s["q"], s["k"], s["qw"], s["kw"], out["q"], out["k"], **kw)
    if c["op"] == "norm":
        return out["q"], out["k"]
    binding.fs_qk_norm_rotate_backward(s["q"], s["k"], s["qw"], s["kw"], s["dqo"], s["dko"],
                                       out["dq"], out["dk"], out["dqw"], out["dkw"],
                                       workspace=out["ws"], **kw)
    return out["q"], out["k"], out["dq"], out["dk"], out["dqw"], out["dkw"]


def _bucket_of(case, edges, r):
    """The bucket of every relative position in r, from the edges."""
    dist = r.abs() if case["two_sided"] else (-r).clamp(min=0)
    at = torch.tensor(edges, device="cuda", dtype=dist.dtype)
    c = torch.bucketize(dist, at, right=True)
    return c + (len(edges) + 1) * (r > 0) if case["two_sided"] else c


def _visible(case, s):
    """[B or 1, 1, n or 1, m] truth values, or None if every key is seen."""
    j = torch.arange(case["m"], device="cuda")
    vis = None
    if s["kv_len"] is not None:
        vis = (j[None, :] < s["kv_len"][:, None])[:, None, None, :]
    if s["mask"] is not None:
        mk = (s["mask"] != 0)[:, None, None, :]
        vis = mk if vis is None else vis & mk
    if case["causal"]:
        i = torch.arange(case["n"], device="cuda")
        cs = (j[None, None, :] <= i[None, :, None] + s["off"][:, None, None])[:, None]
        vis = cs if vis is None else vis & cs
    return vis


def _attn_plain(s):
    c = s["case"]
    B, n, m, H, K, d, dv = (c[x] for x in ("B", "n", "m", "H", "K", "d", "dv"))
    G = H // K
    scale = 1.0 / math.sqrt(d)
    t = s["q"].dtype
    # [B, K, rows, d]: the query heads of a key head as more rows
    q = s["q"].float().view(B, n, K, G, d).permute(0, 2, 3, 1, 4).reshape(B, K, G * n, d)
    k = s["k"].float().permute(0, 2, 1, 3).contiguous()
    v = s["v"].float().permute(0, 2, 1, 3).contiguous()
    x = torch.matmul(q, k.transpose(2, 3).contiguous()).view(B, H, n, m) * scale
    vis = _visible(c, s)
    if s["bias"] is not None:
        r = torch.arange(m, device="cuda")[None, :] - torch.arange(n, device="cuda")[:, None]
        r = r[None] if s["off"] is None else r[None] - s["off"][:, None, None]
        x = x + s["bias"][_bucket_of(c, s["edges"], r)].permute(0, 3, 1, 2)
    if vis is not None:
        x = x.masked_fill(~vis, float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(x - top)
    del x
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    p = p / total.clamp(min=1e-37)
    o = torch.matmul(p.view(B, K, G * n, m), v)

    def rows_back(a, w):
        return a.view(B, K, G, n, w).permute(0, 3, 1, 2, 4).reshape(B, n, H, w)

    o_out = rows_back(o, dv).to(t)
    if c["op"] == "attn":
        return o_out, lse
    do = s["do"].float().view(B, n, K, G, dv).permute(0, 2, 3, 1, 4).reshape(B, K, G * n, dv)
    p = p.view(B, K, G * n, m)
    d_v = torch.matmul(p.transpose(2, 3).contiguous(), do)
    dp = torch.matmul(do, v.transpose(2, 3).contiguous())
    ds = p * (dp - (do * o).sum(-1, keepdim=True))
    del p, dp
    d_q = torch.matmul(ds, k) * scale
    d_k = torch.matmul(ds.transpose(2, 3).contiguous(), q) * scale
    res = (o_out, lse, rows_back(d_q, d).to(t), d_k.permute(0, 2, 1, 3).contiguous().to(t),
           d_v.permute(0, 2, 1, 3).contiguous().to(t))
    if s["bias"] is None:
        return res
    # the gradient of a bucket: the sum over its pairs in 64 bits (long sums),
    # first over the pairs of one relative position: with rows in reverse and
    # m + n wide, reading the same memory m + n - 1 wide puts them in a column
    ds = ds.view(B, H, n, m)
    d_bias = torch.zeros(c["buckets"], H, dtype=torch.float64, device="cuda")
    rel = torch.arange(1 - n, m, device="cuda")
    for b in range(B):
        wide = torch.zeros(H, n, m + n, dtype=torch.float64, device="cuda")
        wide[:, :, :m] = ds[b].flip(1)
        diag = wide.view(H, -1)[:, :n * (m + n - 1)].view(H, n, m + n - 1).sum(1)
        r = rel if s["off"] is None else rel - s["off"][b]
        d_bias.index_add_(0, _bucket_of(c, s["edges"], r), diag.t().contiguous())
    return res + (d_bias.float(),)


def _rotate(x, cos, sin, rot, interleaved, inverse=False):
    """The rotation on the first `rot` elements of the last axis (32 bits)."""
    if inverse:
        sin = -sin
    a = x[..., :rot]
    if interleaved:
        e, o = a[..., 0::2], a[..., 1::2]
        y = torch.stack((e * cos - o * sin, o * cos + e * sin), dim=-1).flatten(-2)
    else:
        e, o = a[..., :rot // 2], a[..., rot // 2:]
        y = torch.cat((e * cos - o * sin, o * cos + e * sin), dim=-1)
    return y if rot == x.shape[-1] else torch.cat((y, x[..., rot:]), dim=-1)


def _norm_plain(s):
    c = s["case"]
    t = s["q"].dtype
    at = s["pos"].long()
    cos, sin = s["cos"][at][:, :, None, :], s["sin"][at][:, :, None, :]
    outs, grads, weights = [], [], []
    for x, w, g in ((s["q"], s["qw"], s.get("dqo")), (s["k"], s["kw"], s.get("dko"))):
        x = x.float()
        inv = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS)
        xn = x * inv
        outs.append(_rotate(xn * w, cos, sin, c["rot"], c["interleaved"]).to(t))
        if g is not None:
            g = _rotate(g.float(), cos, sin, c["rot"], c["interleaved"], inverse=True)
            weights.append((xn * g).double().sum((0, 1, 2)).float())
            gw = g * w
            grads.append((inv * (gw - xn * (xn * gw).mean(-1, keepdim=True))).to(t))
    return tuple(outs + grads + weights)


# ---- 64 bits -------------------------------------------------------------

def exact(case, seed):
    global own
    keep, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    if case["op"].startswith("norm"):
        return _norm_exact(s)
    return _attn_exact(s)


def _attn_exact(s):
    """Sequence by sequence and head by head, the gradients by automatic
    differentiation of the definition."""
    c = s["case"]
    f8 = torch.float64
    B, n, m, H, K = (c[x] for x in ("B", "n", "m", "H", "K"))
    train = c["op"] == "attn_train"
    dev = "cuda"
    o = torch.zeros(B, n, H, c["dv"], dtype=f8, device=dev)
    lse = torch.full((B, H, n), float("-inf"), dtype=f8, device=dev)
    d_q = torch.zeros(B, n, H, c["d"], dtype=f8, device=dev)
    d_k = torch.zeros(B, m, K, c["d"], dtype=f8, device=dev)
    d_v = torch.zeros(B, m, K, c["dv"], dtype=f8, device=dev)
    d_t = None if s["bias"] is None else torch.zeros_like(s["bias"], dtype=f8)
    rows = torch.arange(n, device=dev)
    for b in range(B):
        off = 0 if s["off"] is None else int(s["off"][b])
        size = m if s["kv_len"] is None else int(s["kv_len"][b])
        cols = torch.arange(size, device=dev)
        seen = torch.ones(n, size, dtype=torch.bool, device=dev)
        if s["mask"] is not None:
            seen &= s["mask"][b, :size].bool()[None, :]
        rel = cols[None, :] - rows[:, None] - off
        if c["causal"]:
            seen &= rel <= 0
        if s["bias"] is not None:
            far = rel.abs() if c["two_sided"] else torch.relu(-rel)
            place = torch.zeros_like(rel)
            for e in s["edges"]:
                place += far >= e
            if c["two_sided"]:
                place += (rel > 0) * (len(s["edges"]) + 1)
        for h in range(H):
            q = s["q"][b, :, h].to(f8).requires_grad_(train)
            k = s["k"][b, :size, h // (H // K)].to(f8).requires_grad_(train)
            v = s["v"][b, :size, h // (H // K)].to(f8).requires_grad_(train)
            x = q @ k.t() / math.sqrt(c["d"])
            table = None
            if s["bias"] is not None:
                table = s["bias"][:, h].to(f8).requires_grad_(train)
                x = x + table[place]
            x = torch.where(seen, x, torch.full_like(x, float("-inf")))
            some = seen.any(1)
            x = torch.where(some[:, None], x, torch.zeros_like(x))
            row = torch.logsumexp(x, 1)
            w = torch.exp(x - row[:, None]) * seen
            y = w @ v
            lse[b, h] = torch.where(some, row.detach(), torch.full_like(row.detach(), float("-inf")))
            o[b, :, h] = y.detach()
            if train:
                leaves = [q, k, v] + ([table] if table is not None else [])
                gr = torch.autograd.grad(y, leaves, s["do"][b, :, h].to(f8))
                d_q[b, :, h] = gr[0]
                d_k[b, :size, h // (H // K)] += gr[1]
                d_v[b, :size, h // (H // K)] += gr[2]
                if table is not None:
                    d_t[:, h] += gr[3]
    if not train:
        return o, lse
    res = (o, lse, d_q, d_k, d_v)
    return res if d_t is None else res + (d_t,)


def _norm_exact(s):
    c = s["case"]
    f8 = torch.float64
    rot, d = c["rot"], c["d"]
    half = rot // 2
    p = torch.arange(half, device="cuda")
    first, second = (2 * p, 2 * p + 1) if c["interleaved"] else (p, p + half)
    at = s["pos"].long()
    cos = s["cos"].to(f8)[at][:, :, None, :]
    sin = s["sin"].to(f8)[at][:, :, None, :]
    train = c["op"] == "norm_train"
    outs, grads, weights = [], [], []
    for x, w, g in ((s["q"], s["qw"], s.get("dqo")), (s["k"], s["kw"], s.get("dko"))):
        x = x.to(f8).requires_grad_(train)
        w = w.to(f8).requires_grad_(train)
        z = w * x * torch.rsqrt(x.square().sum(-1, keepdim=True) / d + _EPS)
        y = z.clone()
        y[..., first] = z[..., first] * cos - z[..., second] * sin
        y[..., second] = z[..., second] * cos + z[..., first] * sin
        outs.append(y.detach())
        if train:
            gx, gw = torch.autograd.grad(y, [x, w], g.to(f8))
            grads.append(gx)
            weights.append(gw)
    return tuple(outs + grads + weights)


# ---- what a pass cannot do without ---------------------------------------

def _pairs(case):
    """Visible (query, key) pairs over the batch (scattered padding counted)."""
    lens = _lengths(case)
    total = 0
    for size, off in zip(lens, _offsets(case, lens)):
        if case["causal"]:
            total += sum(min(size, max(0, i + off + 1)) for i in range(case["n"]))
        else:
            total += size * case["n"]
    return total


def work(case):
    es = 4 if case["dtype"] == "fp32" else 2
    B, n, H, K, d = (case[x] for x in ("B", "n", "H", "K", "d"))
    if case["op"].startswith("norm"):
        rows = B * n * (H + K)
        tables = B * n * (case["rot"] * 4 + 4)
        if case["op"] == "norm":
            return {"bytes": rows * d * es * 2 + tables + 8 * d, "flops": 8 * rows * d}
        return {"bytes": rows * d * es * 4 + tables + 16 * d, "flops": 24 * rows * d}
    dv = case["dv"]
    keys = sum(_lengths(case))
    pairs = _pairs(case) * H
    q_bytes, o_bytes = B * n * H * d * es, B * n * H * dv * es
    kv_bytes = keys * K * (d + dv) * es
    lse = B * n * H * 4
    if case["op"] == "attn":
        return {"bytes": q_bytes + o_bytes + kv_bytes + lse, "flops": 2 * pairs * (d + dv)}
    return {"bytes": 2 * (q_bytes + kv_bytes) + 2 * o_bytes + lse,
            "flops": pairs * (2 * (d + dv) + 2 * (3 * d + 2 * dv))}
