"""The attention of include/fs_attention.h and the preparation of its queries
and keys against their definitions in 64 bits (attention_reference.py, which
derives the bounds)."""
import math

import pytest
import torch

from attention_reference import check, norm_reference, reference

pytestmark = pytest.mark.gpu

BF, HF, F4 = torch.bfloat16, torch.float16, torch.float32


def randn(g, *shape, dtype=F4, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def gpu(x):
    return x.cuda() if isinstance(x, torch.Tensor) else x


def run_case(fs, q, k, v, d_o=None, d_lse=None, views=None, poison=False, **kw):
    """Forward (and backward with d_o) through the binding; outputs on the CPU.
    views(t): the device tensor to pass in t's place (same values)."""
    views = views or (lambda t: t)
    dev = {x: gpu(y) for x, y in kw.items()}
    Q, K, V = (views(gpu(t)) for t in (q, k, v))
    B, n, H, _ = q.shape
    fill = lambda *s, dtype=q.dtype: torch.full(s, math.nan, dtype=dtype, device="cuda")
    o = views(fill(B, n, H, v.shape[3]))
    lse = fill(B, H, n, dtype=F4)
    fs.fs_attention_forward(Q, K, V, o, lse, **dev)
    out = {"o": o, "lse": lse}
    if d_o is not None:
        out["d_q"], out["d_k"], out["d_v"] = (views(fill(*t.shape)) for t in (q, k, v))
        if kw.get("bias") is not None:
            out["d_bias"] = fill(*kw["bias"].shape, dtype=F4)
        fs.fs_attention_backward(Q, K, V, o, lse, views(gpu(d_o)), out["d_q"], out["d_k"],
                                 out["d_v"], d_lse=gpu(d_lse), d_bias=out.get("d_bias"), **dev)
    torch.cuda.synchronize()
    return {x: y.cpu() for x, y in out.items()}


def compare(out, ref):
    worst = {x: check(x, out[x], ref[x]) for x in ref}
    print({x: round(y, 3) for x, y in worst.items()})


# dtype, B, n, m, H, K, d, dv, options
CASES = [
    (BF, 2, 1, 1, 2, 2, 64, 64, {}),
    (BF, 1, 1, 700, 8, 2, 128, 128, {}),
    (HF, 3, 7, 133, 6, 3, 80, 80, {"ragged": True}),
    (F4, 2, 3, 65, 4, 1, 48, 48, {"mask": True}),
    (BF, 2, 130, 257, 4, 2, 64, 64, {"ragged": True, "mask": True}),
    (HF, 1, 200, 199, 2, 1, 128, 128, {"causal": True}),
    (F4, 1, 133, 140, 2, 2, 64, 32, {"causal": True, "mask": True}),
    (F4, 1, 61, 70, 2, 1, 128, 128, {}),
    (BF, 1, 100, 90, 1, 1, 256, 256, {"ragged": True}),
    (HF, 1, 40, 333, 2, 1, 192, 128, {"q_len": True}),
    (HF, 1, 50, 70, 2, 2, 200, 256, {"causal": True}),
    (BF, 2, 33, 31, 3, 3, 37, 21, {}),
    (HF, 1, 65, 64, 2, 2, 1, 3, {}),
    (BF, 2, 150, 161, 2, 2, 64, 64, {"buckets": (16, 60), "two_sided": True}),
    (HF, 2, 150, 333, 4, 2, 32, 32, {"buckets": (8, 128), "causal": True}),
    (F4, 1, 77, 150, 2, 1, 40, 40, {"buckets": (32, 100), "two_sided": True, "mask": True}),
    (BF, 2, 5, 1100, 4, 2, 128, 64, {"buckets": (32, 128), "causal": True, "ragged": True}),
    (BF, 1, 2, 300, 4, 1, 64, 64, {"buckets": (16, 64), "two_sided": True, "offset": 290}),
    (BF, 1, 300, 80, 2, 2, 64, 64, {"buckets": (64, 1024), "two_sided": True, "offset": -37}),
    (HF, 1, 300, 310, 2, 1, 128, 128, {"buckets": (4, 7), "two_sided": False}),
    (BF, 1, 1100, 130, 2, 1, 64, 64, {"ragged": True}),  # query ranges split
    (BF, 1, 140, 2100, 2, 2, 64, 64, {"mask": True}),    # key ranges split
    # each form of every pass at each width of tile (workgroups of 128 rows)
    (BF, 3, 257, 300, 16, 16, 64, 64, {"ragged": True, "mask": True}),
    (HF, 2, 390, 390, 11, 11, 64, 64, {"causal": True, "buckets": (16, 50)}),
    (F4, 2, 250, 270, 33, 33, 20, 20, {"mask": True}),
    (BF, 1, 520, 1030, 8, 8, 128, 128, {"mask": True, "buckets": (16, 50), "two_sided": True}),
    (HF, 1, 1030, 1030, 8, 4, 96, 96, {"causal": True}),
    (BF, 1, 300, 4600, 2, 1, 128, 128, {"mask": True, "ragged": True}),  # masks of 64 tiles and more
    (HF, 1, 3, 20000, 2, 2, 64, 64, {"mask": True}),
    (F4, 1, 200, 210, 6, 6, 100, 100, {"causal": True, "buckets": (8, 20), "two_sided": True}),
]


def inputs(case, seed=0):
    dtype, B, n, m, H, K, d, dv, opt = case
    g = torch.Generator().manual_seed(seed + 17 * n + m)
    q, k, v = (randn(g, *s, dtype=dtype) for s in ((B, n, H, d), (B, m, K, d), (B, m, K, dv)))
    kw = {"causal": opt.get("causal", False), "offset": opt.get("offset", 0)}
    i32 = torch.int32
    if opt.get("ragged"):
        kw["kv_len"] = torch.randint(1, m + 1, (B,), generator=g, dtype=i32)
    if opt.get("q_len"):
        kw["q_len"] = torch.randint(1, n + 1, (B,), generator=g, dtype=i32)
    if opt.get("mask"):
        kw["key_mask"] = (torch.rand(B, m, generator=g) > 0.3).to(torch.uint8)
    if kw["causal"]:
        kw["offsets"] = torch.randint(-3, max(m - n, 0) + 4, (B,), generator=g, dtype=i32)
    if "buckets" in opt:
        from streaming_sinkhorn_solver_amd import binding

        kw["two_sided"] = opt.get("two_sided", False)
        kw["edges"] = binding.fs_bucket_edges(*opt["buckets"])
        kw["bias"] = randn(g, opt["buckets"][0] * (2 if kw["two_sided"] else 1), H)
    return q, k, v, randn(g, B, n, H, dv, dtype=dtype, std=0.1), kw


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:8]))
def test_forward_backward(fs, case):
    q, k, v, d_o, kw = inputs(case)
    d_lse = randn(torch.Generator().manual_seed(3), q.shape[0], q.shape[2], q.shape[1], std=0.1)
    print(case, flush=True)
    out = run_case(fs, q, k, v, d_o, d_lse, **kw)
    compare(out, reference(q, k, v, d_o=d_o, d_lse=d_lse, **kw))


def heads_first(t):
    return t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)


def fused(t):
    """Rows as the middle slice of a wider buffer."""
    b, n, h, w = t.shape
    buf = torch.full((b, n, h, 3 * w), math.nan, dtype=t.dtype, device=t.device)
    buf[..., w:2 * w] = t
    return buf[..., w:2 * w]


def unaligned(t):
    """The same rows one element off a 16-byte boundary."""
    buf = torch.full((t.numel() + 1,), math.nan, dtype=t.dtype, device=t.device)
    buf[1:] = t.reshape(-1)
    return buf[1:].view(t.shape)


@pytest.mark.parametrize("views", [heads_first, fused, unaligned])
@pytest.mark.parametrize("case", [CASES[1], CASES[4], CASES[6], CASES[9], CASES[11]],
                         ids=lambda c: "-".join(str(x) for x in c[:8]))
def test_layouts(fs, case, views):
    q, k, v, d_o, kw = inputs(case, seed=5)
    out = run_case(fs, q, k, v, d_o, views=views, **kw)
    compare(out, reference(q, k, v, d_o=d_o, **kw))


@pytest.mark.parametrize("n,dtype", [(3, BF), (150, BF), (150, HF), (70, F4)])
def test_rows_without_keys_and_poisoned_padding(fs, n, dtype):
    """Sequences of no keys, masks that hide all, causal rows before the first
    key; NaN and infinities wherever nothing may be read."""
    g = torch.Generator().manual_seed(n)
    B, m, H, K, d = 4, 97, 4, 2, 64
    q, k, v, d_o = (randn(g, B, r, h, d, dtype=dtype)
                    for r, h in ((n, H), (m, K), (m, K), (n, H)))
    kw = {"kv_len": torch.tensor([0, m, 40, m], dtype=torch.int32),
          "q_len": torch.tensor([n, n, n - 1, n], dtype=torch.int32),
          "key_mask": torch.ones(B, m, dtype=torch.uint8), "causal": True,
          "offsets": torch.tensor([50, m, 50, -2], dtype=torch.int32)}
    kw["key_mask"][1] = 0
    kw["key_mask"][2, ::3] = 0
    ref = reference(q, k, v, d_o=d_o, **kw)
    k, v, q, d_o = k.clone(), v.clone(), q.clone(), d_o.clone()
    for t in (k, v):
        t[0] = math.nan
        t[1] = math.inf
        t[2, 40:] = math.nan
        t[2, ::3] = -math.inf
    q[2, n - 1] = math.nan
    d_o[2, n - 1] = math.inf
    out = run_case(fs, q, k, v, d_o, **kw)
    compare(out, ref)
    assert torch.all(out["o"][:2] == 0) and torch.all(out["lse"][:2] == -math.inf)
    for x in ("d_q", "d_k", "d_v"):
        assert torch.all(out[x][:2] == 0)


@pytest.mark.parametrize("n", [2, 140])
def test_bias_without_weight(fs, n):
    """Buckets at -inf and at the type's lowest hide their pairs; a row that has
    no other pairs is empty."""
    g = torch.Generator().manual_seed(1)
    q, k, v, d_o = (randn(g, 1, r, 2, 64, dtype=BF) for r in (n, 150, 150, n))
    bias = randn(g, 12, 2)
    bias[3] = -math.inf
    bias[5] = torch.finfo(F4).min
    bias[:6, 1] = -math.inf  # the second head sees later keys only
    bias[6:, 1] = torch.finfo(F4).min
    kw = {"bias": bias, "edges": [1, 2, 4, 9, 30], "two_sided": True}
    out = run_case(fs, q, k, v, d_o, **kw)
    compare(out, reference(q, k, v, d_o=d_o, **kw))
    assert torch.all(out["lse"][:, 1] == -math.inf) and torch.all(out["o"][:, :, 1] == 0)


@pytest.mark.parametrize("edges,two_sided", [([], False), ([], True), ([1], True), ([2, 2, 5], True),
                                             ([1024], False), (list(range(1, 256)), True)])
def test_bucket_shapes(fs, edges, two_sided):
    g = torch.Generator().manual_seed(2)
    q, k, v, d_o = (randn(g, 1, r, 2, 32, dtype=BF) for r in (70, 90, 90, 70))
    bias = randn(g, (len(edges) + 1) * (1 + two_sided), 2)
    kw = {"bias": bias, "edges": edges, "two_sided": two_sided, "offset": 4}
    out = run_case(fs, q, k, v, d_o, **kw)
    compare(out, reference(q, k, v, d_o=d_o, **kw))


@pytest.mark.parametrize("n,m", [(0, 5), (5, 0), (200, 0), (0, 0)])
def test_lengths_of_zero(fs, n, m):
    g = torch.Generator().manual_seed(1)
    q, k, v, d_o = (randn(g, 2, r, 2, 64, dtype=BF) for r in (n, m, m, n))
    kw = {"bias": randn(g, 4, 2), "edges": [1, 2, 4], "two_sided": False}
    out = run_case(fs, q, k, v, d_o, **kw)
    assert torch.all(out["o"] == 0) and torch.all(out["lse"] == -math.inf)
    for x in ("d_q", "d_k", "d_v", "d_bias"):
        assert torch.all(out[x] == 0)


def test_large_scores_and_scale(fs):
    """Scores of a few hundred: the running reference, and fp16's weights."""
    g = torch.Generator().manual_seed(4)
    for dtype in (BF, HF, F4):
        q, k, v, d_o = (randn(g, 1, r, 2, 64, dtype=dtype) for r in (140, 300, 300, 140))
        k[:, 100:] *= 3
        k[:, 250:] *= 3
        out = run_case(fs, q, k, v, d_o, scale=1.5)
        compare(out, reference(q, k, v, d_o=d_o, scale=1.5))


@pytest.mark.parametrize("size", [1e-6, 1e-3, 200.0])
def test_half_gradients_of_any_size(fs, size):
    """fp16 gradients far from 1 keep their digits as long as the outputs can."""
    g = torch.Generator().manual_seed(6)
    q, k, v, d_o = (randn(g, 1, r, 2, 64, dtype=HF) for r in (200, 600, 600, 200))
    d_o = (randn(g, 1, 200, 2, 64) * size).to(HF)
    out = run_case(fs, q, k, v, d_o)
    compare(out, reference(q, k, v, d_o=d_o))


def test_broadcast_inputs(fs):
    """k and v of one sequence read by the whole batch (stride 0): each copy's
    gradient is written."""
    g = torch.Generator().manual_seed(7)
    q, d_o = randn(g, 3, 50, 4, 64, dtype=BF), randn(g, 3, 50, 4, 64, dtype=BF)
    k1, v1 = randn(g, 1, 70, 2, 64, dtype=BF), randn(g, 1, 70, 2, 64, dtype=BF)
    k, v = k1.expand(3, -1, -1, -1), v1.expand(3, -1, -1, -1)
    kc, vc = k1.cuda().expand(3, -1, -1, -1), v1.cuda().expand(3, -1, -1, -1)
    o, lse = torch.empty(3, 50, 4, 64, dtype=BF, device="cuda"), torch.empty(3, 4, 50, device="cuda")
    dk, dv = (torch.empty(3, 70, 2, 64, dtype=BF, device="cuda") for _ in range(2))
    dq = torch.empty(3, 50, 4, 64, dtype=BF, device="cuda")
    fs.fs_attention_forward(q.cuda(), kc, vc, o, lse)
    fs.fs_attention_backward(q.cuda(), kc, vc, o, lse, d_o.cuda(), dq, dk, dv)
    ref = reference(q, k, v, d_o=d_o)
    compare({"o": o, "lse": lse, "d_q": dq, "d_k": dk, "d_v": dv}, ref)


def test_gradient_against_differences(fs):
    """fp32 gradients of sum(o c) + sum(lse e) against central differences of
    the definition in 64 bits."""
    g = torch.Generator().manual_seed(8)
    q, k, v = (randn(g, 1, r, 2, 8) for r in (5, 9, 9))
    bias = randn(g, 6, 2)
    c, e = randn(g, 1, 5, 2, 8), randn(g, 1, 2, 5)
    kw = {"edges": [1, 3], "two_sided": True}
    out = run_case(fs, q, k, v, c, e, bias=bias, **kw)

    def loss(q, k, v, bias):
        r = reference(q, k, v, bias=bias, **kw)
        return float((r["o"][0] * c).sum() + (r["lse"][0] * e).sum())

    leaves = {"d_q": q, "d_k": k, "d_v": v, "d_bias": bias}
    step = 1e-4
    for name, t in leaves.items():
        for _ in range(12):
            at = tuple(int(torch.randint(0, s, (1,), generator=g)) for s in t.shape)
            vals = []
            for sign in (1, -1):
                args = {x: y.double() for x, y in leaves.items()}
                args[name] = args[name].clone()
                args[name][at] += sign * step
                vals.append(loss(*args.values()))
            diff = (vals[0] - vals[1]) / (2 * step)
            # the difference is off by step^2 times a third derivative (of order
            # 10 here); the gradient by fp32's rounding
            assert abs(diff - float(out[name][at])) < 2e-5 * max(1.0, abs(diff)), (name, at)


def test_equal_calls_equal_bits_and_streams(fs):
    q, k, v, d_o, kw = inputs(CASES[13], seed=9)
    first = run_case(fs, q, k, v, d_o, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = run_case(fs, q, k, v, d_o, stream=side, **kw)
    with torch.cuda.stream(side):
        third = run_case(fs, q, k, v, d_o, **kw)
    for x in first:
        assert torch.equal(first[x], again[x]) and torch.equal(first[x], third[x]), x


@pytest.mark.parametrize("case", [CASES[1], CASES[16], CASES[20], CASES[21]],
                         ids=lambda c: "-".join(str(x) for x in c[:8]))
def test_graph_replays(fs, case):
    """A captured forward and backward, replayed on new inputs, against eager
    calls made between the replays."""
    q, k, v, d_o, kw = inputs(case)
    dev = {x: gpu(y) for x, y in kw.items()}
    Q, K, V, G = (t.cuda() for t in (q, k, v, d_o))
    o, lse = torch.empty_like(Q[..., :1].expand(*Q.shape[:3], V.shape[3])), \
        torch.empty(Q.shape[0], Q.shape[2], Q.shape[1], device="cuda")
    o = o.contiguous()
    outs = [o, lse, torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V)]
    bias = kw.get("bias")
    if bias is not None:
        outs.append(torch.empty_like(bias, device="cuda"))
    ws = torch.empty(fs.fs_attention_workspace_bytes(Q, K, V, edges=kw.get("edges"), backward=True),
                     dtype=torch.uint8, device="cuda")

    def step(w=None):
        fs.fs_attention_forward(Q, K, V, o, lse, workspace=w, **dev)
        fs.fs_attention_backward(Q, K, V, o, lse, G, *outs[2:5],
                                 d_bias=outs[5] if bias is not None else None, workspace=w, **dev)

    step(ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(ws)
    for seed in range(3):
        q2, k2, v2, d2, _ = inputs(case, seed=20 + seed)
        for t, s in ((Q, q2), (K, k2), (V, v2), (G, d2)):
            t.copy_(s)
        step()
        torch.cuda.synchronize()
        eager = [t.clone() for t in outs]
        for t in outs:
            t.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(eager, outs):
            assert torch.equal(x, y)


@pytest.mark.parametrize("case", [CASES[1], CASES[16], CASES[20], CASES[21], CASES[25]],
                         ids=lambda c: "-".join(str(x) for x in c[:8]))
def test_workspace_contents_do_not_matter(fs, case):
    """Whatever the workspace held, and with no bytes to spare."""
    q, k, v, d_o, kw = inputs(case)
    first = run_case(fs, q, k, v, d_o, **kw)
    need = fs.fs_attention_workspace_bytes(q, k, v, edges=kw.get("edges"), backward=True)
    ws = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in every type
    again = run_case(fs, q, k, v, d_o, workspace=ws[:need], **kw)
    for x in first:
        assert torch.equal(first[x], again[x]), x
    assert torch.all(ws[need:] == 0xFF)


def test_single_gradients(fs):
    """Each gradient alone is the one that comes with the others; keys' and
    values' without the queries' stay within the bounds."""
    q, k, v, d_o, kw = inputs(CASES[13])
    dev = {x: gpu(y) for x, y in kw.items()}
    Q, K, V, G = (t.cuda() for t in (q, k, v, d_o))
    full = run_case(fs, q, k, v, d_o, **kw)
    o, lse = full["o"].cuda(), full["lse"].cuda()
    ref = reference(q, k, v, d_o=d_o, **kw)
    for name, like in (("d_q", Q), ("d_k", K), ("d_v", V), ("d_bias", dev["bias"])):
        out = torch.full_like(like, math.nan)
        fs.fs_attention_backward(Q, K, V, o, lse, G, **{name: out}, **dev)
        torch.cuda.synchronize()
        check(name, out, ref[name])
        if name in ("d_q", "d_bias"):
            assert torch.equal(out.cpu(), full[name])


def test_binding_refuses(fs):
    q = torch.zeros(1, 4, 2, 32, device="cuda", dtype=BF)
    o, lse = torch.empty_like(q), torch.empty(1, 2, 4, device="cuda")
    ok = lambda **kw: fs.fs_attention_forward(q, q, q, o, lse, **kw)
    ok()
    i32 = torch.int32
    for bad, error in ((dict(kv_len=torch.tensor([4], dtype=i32)), TypeError),       # on the host
                       (dict(kv_len=torch.tensor([4], device="cuda")), TypeError),   # int64
                       (dict(kv_len=torch.zeros(2, dtype=i32, device="cuda")), ValueError),
                       (dict(key_mask=torch.ones(1, 4, device="cuda")), TypeError),
                       (dict(key_mask=torch.ones(1, 5, dtype=torch.bool, device="cuda")), ValueError),
                       (dict(bias=torch.zeros(3, 2, device="cuda"), edges=[1, 2]), ValueError),
                       (dict(scale=-1.0), fs.FsError), (dict(offset=1 << 30), fs.FsError),
                       (dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda")), fs.FsError)):
        with pytest.raises(error):
            ok(**bad)
    for args in ((q.float(), q, q, o), (q.double(), q, q, o), (q[0], q, q, o), (q, q[:, :3], q, o),
                 (q, q, q, o[..., :31]), (q, q, q, q), (q, q.cpu(), q, o),
                 (q, q, q, o[:, :1].expand(-1, 4, -1, -1)), (q.transpose(2, 3), q, q, o)):
        with pytest.raises((TypeError, ValueError, fs.FsError)):
            fs.fs_attention_forward(*args)
    with pytest.raises(fs.FsError):
        fs.fs_qk_norm_rotate(q, None, None, None, q, None)
    with pytest.raises(TypeError):
        fs.fs_qk_norm_rotate(q, None, None, None, o, None, cos=torch.ones(4, 16, device="cuda"))
    with pytest.raises(TypeError):
        fs.fs_qk_norm_rotate(None, None, None, None, None, None)


def test_offsets_beyond_32_bits(fs):
    """Keys of 2^32 bytes and more behind one another: the last heads against
    the same rows in a small tensor, bit for bit."""
    m, K, d = 1 << 18, 72, 128
    k = torch.empty(1, m, K, d, dtype=BF, device="cuda").normal_()
    assert k.numel() > 2 ** 31
    kv_len = torch.tensor([m - 5], dtype=torch.int32, device="cuda")
    for n in (1, 130):
        q = torch.randn(1, n, K, d, device="cuda").to(BF)
        o, lse = torch.empty_like(q), torch.empty(1, K, n, device="cuda")
        fs.fs_attention_forward(q, k, k, o, lse, kv_len=kv_len)
        part = k[:, -3000:, -2:].contiguous()
        o2, lse2 = torch.empty_like(o[:, :, -2:]), torch.empty(1, 2, n, device="cuda")
        mask = torch.zeros(1, m, dtype=torch.uint8, device="cuda")
        mask[:, -3000:] = 1
        fs.fs_attention_forward(q, k, k, o, lse, kv_len=kv_len, key_mask=mask)
        qs = q[:, :, -2:]
        fs.fs_attention_forward(qs, part, part, o2, lse2,
                                kv_len=torch.tensor([2995], dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        ref = reference(qs.cpu(), part[:, :2995].cpu(), part[:, :2995].cpu())
        check("o", o[:, :, -2:], ref["o"])
        check("lse", lse[:, -2:], ref["lse"])
        check("o2", o2, ref["o"])


def test_rows_behind_are_left(fs):
    """Memory around the outputs keeps its contents."""
    q, k, v, d_o, kw = inputs(CASES[4])
    B, n, H, d = q.shape
    big = torch.full((B, n + 2, H + 1, d + 8), 7.0, dtype=BF, device="cuda")
    o = big[:, :n, :H, :d]
    fs.fs_attention_forward(*(t.cuda() for t in (q, k, v)), o, **{x: gpu(y) for x, y in kw.items()})
    torch.cuda.synchronize()
    check("o", o, reference(q, k, v, **kw)["o"])
    assert torch.all(big[:, n:] == 7) and torch.all(big[:, :, H:] == 7) and torch.all(big[..., d:] == 7)


# ---- norm + rotation --------------------------------------------------------

NORM = [  # dtype, B, n, Hq, Hk, d, rot, interleaved, weights, offset or positions
    (BF, 2, 5, 4, 2, 128, 128, False, True, "positions"),
    (HF, 1, 33, 3, 1, 64, 64, True, True, 7),
    (F4, 2, 9, 2, 2, 48, 24, False, True, "positions"),
    (BF, 1, 70, 8, 8, 256, 128, True, False, 0),
    (HF, 3, 17, 5, 1, 80, 80, False, True, 3),
    (BF, 1, 4, 2, 0, 34, 10, False, True, "positions"),
    (F4, 1, 3, 0, 2, 2, 2, True, False, 0),
    (BF, 1, 600, 8, 2, 96, 0, False, True, 0),
    (F4, 1, 1, 1, 1, 256, 250, False, True, -4),
    # enough rows for the forms of several rows a lane group, heads not a multiple of them
    (BF, 2, 4700, 11, 3, 80, 32, False, True, "positions"),
    (HF, 1, 33000, 3, 1, 64, 48, True, True, "positions"),
]


@pytest.mark.parametrize("layout", ["plain", "heads_first", "unaligned"])
@pytest.mark.parametrize("case", NORM, ids=lambda c: "-".join(str(x) for x in c))
def test_norm_rotate(fs, case, layout):
    dtype, B, n, Hq, Hk, d, rot, inter, weights, where = case
    g = torch.Generator().manual_seed(d + n)
    view = {"plain": lambda t: t, "heads_first": heads_first, "unaligned": unaligned}[layout]
    x = [randn(g, B, n, h, d, dtype=dtype, std=2.0) if h else None for h in (Hq, Hk)]
    dy = [randn(g, B, n, h, d, dtype=dtype) if h else None for h in (Hq, Hk)]
    w = [1 + randn(g, d, std=0.3) if weights else None for _ in range(2)]
    cos = sin = pos = None
    kw = {"eps": 1e-5, "interleaved": inter}
    if rot:
        ang = torch.rand(50, rot // 2, generator=g) * 6
        cos, sin = ang.cos(), ang.sin()
        kw.update(cos=cos.cuda(), sin=sin.cuda())
    if where == "positions":
        # positions outside the tables stand for the nearest row
        pos = torch.randint(-2, 53, (B, n), generator=g, dtype=torch.int32)
        kw["positions"] = pos.cuda()
    else:
        pos = (torch.arange(n) + where)[None].expand(B, n)
        kw["offset"] = where
    dev = lambda t: None if t is None else view(t.cuda())
    nan = lambda t: None if t is None else view(torch.full_like(t, math.nan).cuda())
    wd = [None if t is None else t.cuda() for t in w]
    y, dx = [nan(t) for t in x], [nan(t) for t in x]
    dw = [torch.full((d,), math.nan, device="cuda") if h else None for h in (Hq, Hk)]
    fs.fs_qk_norm_rotate(dev(x[0]), dev(x[1]), *wd, *y, **kw)
    fs.fs_qk_norm_rotate_backward(dev(x[0]), dev(x[1]), *wd, dev(dy[0]), dev(dy[1]), *dx, *dw, **kw)
    torch.cuda.synchronize()
    for i in range(2):
        if x[i] is None:
            continue
        ref = norm_reference(x[i], w[i], cos, sin, pos, 1e-5, inter, dy[i])
        compare({"y": y[i], "dx": dx[i], "dw": dw[i]}, ref)


def test_norm_of_zeros(fs):
    """A row of zeros gives zeros (eps > 0), its gradient w g / sqrt(eps)."""
    x = torch.zeros(1, 2, 1, 64, device="cuda")
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(64, device="cuda")
    fs.fs_qk_norm_rotate(x, None, None, None, y, None, eps=1e-4)
    fs.fs_qk_norm_rotate_backward(x, None, None, None, torch.ones_like(x), None, dx, None, dw,
                                  eps=1e-4)
    assert torch.all(y == 0) and torch.allclose(dx, torch.full_like(dx, 100.0)) and torch.all(dw == 0)


# ---- as they are used together ----------------------------------------------

def test_descriptors_into_a_transport_loss(fs):
    """Two sets of states attend to one another (norm, rotation, cross
    attention with a learned bias) and the result is matched to the other set
    by the solver; the loss's gradient runs back through all of it."""
    g = torch.Generator().manual_seed(11)
    n, m, H, w = 150, 170, 2, 32
    x, y = randn(g, 1, n, H, w), randn(g, 1, m, H, w)
    vals = randn(g, 1, m, H, w, std=0.5)
    ang = torch.rand(200, w // 2, generator=g) * 3
    bias = randn(g, 6, H, std=0.5)
    target = randn(g, m, H * w, std=0.5)
    eps, iters = 0.5, 60
    rot = dict(cos=ang.cos().cuda(), sin=ang.sin().cuda())
    att = dict(bias=bias.cuda(), edges=[2, 9], two_sided=True)
    X, Y, V, T = x.cuda(), y.cuda(), vals.cuda(), target.cuda()
    qn, o = torch.empty_like(X), torch.empty_like(X)
    kn = torch.empty_like(Y)
    lse = torch.empty(1, H, n, device="cuda")
    a, b = torch.full((n,), 1 / n, device="cuda"), torch.full((m,), 1 / m, device="cuda")
    fs.fs_qk_norm_rotate(X, None, None, None, qn, None, **rot)
    fs.fs_qk_norm_rotate(None, Y, None, None, None, kn, **rot)
    fs.fs_attention_forward(qn, kn, V, o, lse, **att)
    cloud = o.reshape(n, H * w)
    p, f, gp, _ = fs.solve(cloud, T, a, b, eps=eps, iters=iters, dv_max=H * w)
    gx = torch.empty_like(cloud)
    fs.fs_gradient(p, eps, f, gp, cloud, T, gx, None)
    value = torch.empty(1, dtype=torch.float64, device="cuda")
    fs.fs_dual_value(p, f, gp, value)
    dq, dk, dv, dx = (torch.empty_like(t) for t in (X, Y, V, X))
    db = torch.empty(6, H, device="cuda")
    fs.fs_attention_backward(qn, kn, V, o, lse, gx.view_as(o), dq, dk, dv, d_bias=db, **att)
    fs.fs_qk_norm_rotate_backward(X, None, None, None, dq, None, dx, None, **rot)
    torch.cuda.synchronize()

    # the same chain in 64 bits, differentiated automatically
    F8 = torch.float64
    leaves = [t.to(F8).requires_grad_() for t in (x, vals, bias)]
    x8, v8, b8 = leaves

    def prep(t):
        z = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)
        c, s = ang.cos().to(F8), ang.sin().to(F8)
        c, s = c[: t.shape[1]][None, :, None], s[: t.shape[1]][None, :, None]
        e, h = z[..., : w // 2], z[..., w // 2:]
        return torch.cat((e * c - h * s, h * c + e * s), -1)

    q8, k8 = prep(x8), prep(y.to(F8))
    rel = torch.arange(m)[None] - torch.arange(n)[:, None]
    place = (rel.abs() >= 2).long() + (rel.abs() >= 9) + 3 * (rel > 0)
    s = torch.einsum("bnhd,bmhd->bhnm", q8, k8) / math.sqrt(w) + b8[place].permute(2, 0, 1)[None]
    o8 = torch.einsum("bhnm,bmhd->bnhd", s.softmax(-1), v8).reshape(n, H * w)
    t8 = target.to(F8)
    C = (o8.square().sum(1)[:, None] + t8.square().sum(1)[None] - 2 * o8 @ t8.t())
    with torch.no_grad():
        f8, g8 = torch.zeros(n, dtype=F8), torch.zeros(m, dtype=F8)
        for _ in range(iters):
            f8 = -eps * torch.logsumexp((g8[None] - C) / eps - math.log(m), 1)
            g8 = -eps * torch.logsumexp((f8[:, None] - C) / eps - math.log(n), 0)
        P = torch.exp((f8[:, None] + g8[None] - C) / eps) / (n * m)
    grads = torch.autograd.grad((P * C).sum(), leaves)
    dual = float(f8.mean() + g8.mean())
    assert abs(float(value) - dual) <= 2e-3 * eps
    # the solver's gradient is within 1e-3 of its terms (its transport's bar);
    # the terms here are of the gradient's own size
    for got, want in ((dx, grads[0]), (dv, grads[1]), (db, grads[2])):
        got = got.cpu().to(F8)
        assert float((got - want).norm() / want.norm()) < 5e-3
