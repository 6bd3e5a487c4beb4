"""Attention where rows, keys or sizes are at the edge of what a call allows, against
the definition in 64 bits.  A few heads are checked; a problem is made large enough
for the other forms of the kernels by repeating them, and each copy has to give the
same bits."""
import math

import pytest
import torch

from attention_reference import check, norm_reference, reference
from test_attention_gpu import BF, F4, HF, gpu, randn

pytestmark = pytest.mark.gpu

NAN, INF = math.nan, math.inf


def run(fs, q, k, v, d_o=None, d_lse=None, copies=1, view=None, **kw):
    """Outputs of the first heads, on the CPU, as a dict; with copies > 1 every
    head stands that many times in the call and all copies are compared.
    view(t): the device tensor to pass in t's place (same values)."""
    view = view or (lambda t: t)
    rep = lambda t: view(t.cuda().repeat(1, 1, copies, 1))
    Q, K, V = rep(q), rep(k), rep(v)
    dev = {x: gpu(y) for x, y in kw.items()}
    B, n, H, _ = Q.shape
    nan = lambda *s, dtype=q.dtype: torch.full(s, NAN, dtype=dtype, device="cuda")
    if kw.get("bias") is not None:
        dev["bias"] = dev["bias"].repeat(1, copies)
    out = {"o": view(nan(B, n, H, v.shape[3])), "lse": nan(B, H, n, dtype=F4)}
    fs.fs_attention_forward(Q, K, V, out["o"], out["lse"], **dev)
    if d_o is not None:
        out["d_q"], out["d_k"], out["d_v"] = (view(nan(*t.shape)) for t in (Q, K, V))
        if kw.get("bias") is not None:
            out["d_bias"] = nan(*dev["bias"].shape, dtype=F4)
        g = None if d_lse is None else d_lse.cuda().repeat(1, copies, 1)
        fs.fs_attention_backward(Q, K, V, out["o"], out["lse"], rep(d_o), out["d_q"], out["d_k"],
                                 out["d_v"], d_lse=g, d_bias=out.get("d_bias"), **dev)
    torch.cuda.synchronize()
    heads = {"lse": 1, "d_bias": 1}
    for x, t in out.items():
        axis = heads.get(x, 2)
        parts = t.chunk(copies, axis)
        same = torch.stack([torch.equal(p.nan_to_num(), parts[0].nan_to_num()) and
                            torch.equal(p.isnan(), parts[0].isnan()) and torch.tensor(True)
                            for p in parts[1:]] or [torch.tensor(True)])
        assert same.all(), f"{x}: copies of a head differ"
        out[x] = parts[0].cpu()
    return out


def compare(out, ref):
    print({x: round(check(x, out[x], ref[x]), 3) for x in ref})


# copies of two heads, so that few and many workgroups (the 32-row and the 128-row
# forms of the backward passes) both occur
EMPTY = [(BF, 3, 64, 1), (BF, 150, 64, 1), (BF, 150, 64, 66), (BF, 150, 128, 1), (BF, 150, 128, 66),
         (HF, 140, 64, 66), (HF, 140, 200, 1), (F4, 70, 40, 1), (F4, 130, 64, 66), (F4, 40, 128, 1)]


@pytest.mark.parametrize("dtype,n,d,copies", EMPTY)
def test_rows_that_see_no_key_poison_nothing(fs, dtype, n, d, copies):
    """Rows before the first key of a causal limit, or behind a left padding of
    masked keys, hold NaN and infinities in q, d_o and d_lse."""
    g = torch.Generator().manual_seed(n + d)
    B, m, H = 2, n + 9, 2
    q, k, v, d_o = (randn(g, B, r, H, d, dtype=dtype) for r in (n, m, m, n))
    d_lse = randn(g, B, H, n)
    # entry 0: the first rows stand before the keys; entry 1: left padding
    lost = max(1, n // 3)
    kw = {"causal": True, "offsets": torch.tensor([-lost, 0], dtype=torch.int32),
          "key_mask": torch.ones(B, m, dtype=torch.uint8)}
    kw["key_mask"][1, :lost] = 0
    ref = reference(q, k, v, d_o=d_o, d_lse=d_lse, **kw)
    assert torch.all(ref["lse"][0][:, :, :lost] == -INF) and torch.all(ref["lse"][0][:, :, lost:] > -INF)
    q[0, :lost], q[1, :lost] = NAN, INF
    d_o[0, :lost], d_o[1, :lost] = INF, NAN
    d_lse[:, :, :lost] = NAN
    out = run(fs, q, k, v, d_o, d_lse, copies, **kw)
    compare(out, ref)
    assert torch.all(out["d_q"][:, :lost] == 0)


@pytest.mark.parametrize("dtype,n,d,copies", EMPTY)
def test_rows_emptied_by_the_bias_poison_nothing(fs, dtype, n, d, copies):
    """Rows whose every key stands in a bucket without weight: d_o and d_lse there
    may hold anything."""
    g = torch.Generator().manual_seed(n + d)
    m, H = max(2, n // 2), 2
    q, k, v, d_o = (randn(g, 2, r, H, d, dtype=dtype) for r in (n, m, m, n))
    d_lse = randn(g, 2, H, n)
    bias = randn(g, 8, H)
    bias[:4, 1] = -INF  # the second head sees later keys only
    kw = {"bias": bias, "edges": [1, 3, 8], "two_sided": True}
    ref = reference(q, k, v, d_o=d_o, d_lse=d_lse, **kw)
    empty = ref["lse"][0] == -INF
    assert empty[:, 1, m - 1:].all() and not empty[:, 1, :m - 1].any() and not empty[:, 0].any()
    d_o[:, m - 1:, 1] = torch.where(torch.arange(n - m + 1) % 2 == 0, NAN, INF)[:, None].to(dtype)
    d_lse[:, 1, m - 1:] = NAN
    out = run(fs, q, k, v, d_o, d_lse, copies, **kw)
    compare(out, ref)
    assert torch.all(out["d_q"][:, m - 1:, 1] == 0)


@pytest.mark.parametrize("dtype,n,d,copies", EMPTY)
def test_keys_that_no_row_sees_poison_nothing(fs, dtype, n, d, copies):
    """A causal limit and lengths of the queries alone: keys behind the last query
    row are seen by padding only and may hold anything."""
    g = torch.Generator().manual_seed(n + d)
    B, m, H = 3, n + 9, 2
    q, k, v, d_o = (randn(g, B, r, H, d, dtype=dtype) for r in (n, m, m, n))
    lens = [max(1, n // 2), n - 1, 0]
    kw = {"causal": True, "offsets": torch.tensor([0, 3, 5], dtype=torch.int32),
          "q_len": torch.tensor(lens, dtype=torch.int32)}
    ref = reference(q, k, v, d_o=d_o, **kw)
    for t in (k, v):
        t[0, lens[0]:] = NAN
        t[1, lens[1] + 3:] = INF
        t[2] = -INF
    out = run(fs, q, k, v, d_o, copies=copies, **kw)
    compare(out, ref)
    for x in ("d_k", "d_v"):
        assert torch.all(out[x][0, lens[0]:] == 0) and torch.all(out[x][1, lens[1] + 3:] == 0)


@pytest.mark.parametrize("B,n", [(2, 0), (0, 3), (0, 0)])
def test_norm_of_no_tokens(fs, B, n):
    """Nothing to write but the weights' gradients, sums of nothing."""
    q, k = torch.empty(B, n, 4, 64, device="cuda"), torch.empty(B, n, 2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    dw = [torch.full_like(w, NAN) for _ in range(2)]
    empty = [torch.empty_like(t) for t in (q, k)]
    fs.fs_qk_norm_rotate(q, k, w, w, *empty)
    fs.fs_qk_norm_rotate_backward(q, k, w, w, q, k, *empty, *dw)
    # (and with a workspace full of NaN)
    ws = torch.full((fs.fs_qk_norm_workspace_bytes(q, k),), 0xFF, dtype=torch.uint8, device="cuda")
    fs.fs_qk_norm_rotate_backward(q, k, w, None, q, k, *empty, dw[0], None, workspace=ws)
    torch.cuda.synchronize()
    assert torch.all(dw[0] == 0) and torch.all(dw[1] == 0)


def test_numbers_beyond_32_bits_are_refused(fs):
    """An offset, an edge or a size that 32 bits do not hold is no other number."""
    q = torch.randn(1, 4, 2, 32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(1, 2, 4, device="cuda")
    bias = torch.zeros(3, 2, device="cuda")
    for kw in (dict(offset=1 << 32), dict(offset=-(1 << 32) - 1),
               dict(bias=bias, edges=[1, (1 << 32) + 2], two_sided=False)):
        with pytest.raises(ValueError, match="32 bits"):
            fs.fs_attention_forward(q, q, q, o, lse, causal=True, **kw)
        with pytest.raises(ValueError, match="32 bits"):
            fs.fs_attention_backward(q, q, q, o, lse, o, torch.empty_like(q), causal=True, **kw)
    many = q[:, :1].expand(-1, (1 << 32) + 4, -1, -1)
    with pytest.raises(ValueError, match="32 bits"):
        fs.fs_attention_forward(q, many, many, o, lse)
    with pytest.raises(ValueError, match="32 bits"):
        fs.fs_qk_norm_rotate(q, None, None, None, o, None, offset=1 << 32)
    with pytest.raises(ValueError, match="32 bits"):
        fs.fs_qk_norm_rotate(many, None, None, None, many, None)


@pytest.mark.parametrize("dtype,B,n,H,d", [(F4, 2, 5, 3, 64), (BF, 1, 40, 5, 128), (HF, 2, 9, 1, 256),
                                           (BF, 1, 12000, 11, 96), (F4, 1, 7, 3, 34)])
def test_norm_without_eps(fs, dtype, B, n, H, d):
    """eps = 0 is allowed; heads that do not fill the lanes of a wave leave no trace in
    the weights' gradients."""
    g = torch.Generator().manual_seed(d)
    x, dy = randn(g, B, n, H, d, dtype=dtype, std=2.0), randn(g, B, n, H, d, dtype=dtype)
    w = 1 + randn(g, d, std=0.3)
    y, dx = (torch.full_like(x, NAN, device="cuda") for _ in range(2))
    dw = torch.full((d,), NAN, device="cuda")
    fs.fs_qk_norm_rotate(x.cuda(), None, w.cuda(), None, y, None, eps=0.0)
    fs.fs_qk_norm_rotate_backward(x.cuda(), None, w.cuda(), None, dy.cuda(), None, dx, None, dw, None,
                                  eps=0.0)
    torch.cuda.synchronize()
    compare({"y": y, "dx": dx, "dw": dw}, norm_reference(x, w, None, None, None, 0.0, False, dy))


@pytest.mark.parametrize("low", [-1e9, -3e12, -1e25])
@pytest.mark.parametrize("dtype,n,d,copies", EMPTY)
def test_bias_far_below_every_score(fs, dtype, n, d, copies, low):
    """Buckets with an entry that stands for a mask: no weight next to other keys, and
    none in rows that have no others, whose scores fp32 would have lost beside it."""
    g = torch.Generator().manual_seed(n + d)
    m, H = max(2, n // 2), 2
    q, k, v, d_o = (randn(g, 2, r, H, d, dtype=dtype) for r in (n, m, m, n))
    d_lse = randn(g, 2, H, n)
    bias = randn(g, 8, H)
    bias[:4, 1] = low  # the second head sees later keys only
    kw = {"edges": [1, 3, 8], "two_sided": True, "scale": 1.5}
    out = run(fs, q, k, v, d_o, d_lse, copies, bias=bias, **kw)
    bias[:4, 1] = -INF
    compare(out, reference(q, k, v, d_o=d_o, d_lse=d_lse, bias=bias, **kw))
    assert torch.all(out["lse"][:, 1, m - 1:] == -INF) and torch.all(out["o"][:, m - 1:, 1] == 0)


@pytest.mark.parametrize("dtype,n", [(BF, 5), (HF, 140), (F4, 33)])
def test_one_buffer_for_queries_keys_and_values(fs, dtype, n):
    """q, k, v as slices of a fused projection, their gradients as slices of its
    gradient; the columns between them keep their contents."""
    g = torch.Generator().manual_seed(n)
    B, H, K, d = 2, 4, 2, 64
    qkv = randn(g, B, n, H + 2 * K + 1, d, dtype=dtype)
    d_o = randn(g, B, n, H, d, dtype=dtype, std=0.1)
    part = lambda t: (t[:, :, :H], t[:, :, H:H + K], t[:, :, H + K:H + 2 * K])
    dev = qkv.cuda()
    grad = torch.full_like(dev, 7.0)
    o, lse = torch.empty(B, n, H, d, dtype=dtype, device="cuda"), torch.empty(B, H, n, device="cuda")
    fs.fs_attention_forward(*part(dev), o, lse, causal=True)
    fs.fs_attention_backward(*part(dev), o, lse, d_o.cuda(), *part(grad), causal=True)
    # the same through the norm, in place of the projection's columns for q and k
    y = torch.full_like(dev, 7.0)
    fs.fs_qk_norm_rotate(*part(dev)[:2], None, None, *part(y)[:2])
    torch.cuda.synchronize()
    ref = reference(*part(qkv), d_o=d_o, causal=True)
    compare(dict(zip(("d_q", "d_k", "d_v"), part(grad)), o=o, lse=lse), ref)
    assert torch.all(grad[:, :, H + 2 * K:] == 7) and torch.all(y[:, :, H + K:] == 7)
    for got, x in zip(part(y), part(qkv)[:2]):
        check("y", got, norm_reference(x, None, None, None, None, 1e-6, False)["y"])


def test_calls_on_two_streams_at_once(fs):
    """Two training steps in flight together, each with its own buffers."""
    g = torch.Generator().manual_seed(3)
    sets, refs = [], []
    for n, m in ((300, 700), (130, 2100)):
        q, k, v, d_o = (randn(g, 2, r, 4, 64, dtype=BF) for r in (n, m, m, n))
        refs.append(reference(q, k, v, d_o=d_o))
        sets.append([t.cuda() for t in (q, k, v, d_o)])
    outs = [[torch.full_like(t, NAN) for t in (s[0], s[0], s[1], s[2])] +
            [torch.full((2, 4, s[0].shape[1]), NAN, device="cuda")] for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for (q, k, v, d_o), (o, dq, dk, dv, lse), s in zip(sets, outs, streams):
            fs.fs_attention_forward(q, k, v, o, lse, stream=s)
            fs.fs_attention_backward(q, k, v, o, lse, d_o, dq, dk, dv, stream=s)
    torch.cuda.synchronize()
    for (o, dq, dk, dv, lse), ref in zip(outs, refs):
        compare({"o": o, "lse": lse, "d_q": dq, "d_k": dk, "d_v": dv}, ref)
