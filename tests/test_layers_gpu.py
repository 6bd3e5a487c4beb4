"""The operators of include/fs_layers.h against their definitions in 64 bits
(layers_reference.py, which derives the bounds)."""
import math

import pytest
import torch

from attention_reference import check
from layers_reference import (balance_reference, distill_reference, norm_reference,
                              product_reference, quantize_reference)

pytestmark = pytest.mark.gpu

BF, HF, F4 = torch.bfloat16, torch.float16, torch.float32
I4 = torch.int32
NAN = math.nan


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=F4, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def gpu(t):
    return t.cuda() if isinstance(t, torch.Tensor) else t


def fill(*shape, dtype=F4):
    if dtype.is_floating_point:
        return torch.full(shape, NAN, dtype=dtype, device="cuda")
    return torch.full(shape, -77, dtype=dtype, device="cuda")


def wider(t, by=5):
    """t's values in rows that stand further apart, from an odd address on."""
    shape = t.shape[:-1] + (t.shape[-1] + by,)
    buf = torch.full(shape, NAN, dtype=t.dtype, device=t.device) if t.dtype.is_floating_point \
        else torch.full(shape, 99, dtype=t.dtype, device=t.device)
    view = buf[..., 1:1 + t.shape[-1]]
    view.copy_(t)
    return view


def rows_first(t):
    """[batch, rows, width] whose batch stride is the smaller one."""
    return t.transpose(0, 1).contiguous().transpose(0, 1)


def compare(out, ref):
    torch.cuda.synchronize()
    worst = {}
    for name, r in ref.items():
        if isinstance(r, tuple):
            worst[name] = round(check(name, out[name], r), 3)
        else:
            assert torch.equal(out[name].cpu(), r), name
    print(worst)


# ---- layer norm -----------------------------------------------------------

def norm_run(fs, x, w, b, eps, residual=None, lengths=None, d_y=None, d_total=None, views=None):
    views = views or (lambda t: t)
    x, w, b, residual, lengths, d_y, d_total = map(gpu, (x, w, b, residual, lengths, d_y, d_total))
    at = lambda t: None if t is None else views(t)
    B, n, width = x.shape
    out = {"y": views(fill(*x.shape, dtype=x.dtype)), "mean": fill(B, n), "rstd": fill(B, n)}
    if residual is not None:
        out["total"] = views(fill(*x.shape, dtype=x.dtype))
    X = views(x)
    fs.fs_layer_norm(X, w, b, out["y"], residual=at(residual), total=out.get("total"),
                     mean=out["mean"], rstd=out["rstd"], eps=eps, lengths=lengths)
    if d_y is not None:
        z = X if residual is None else out["total"]
        out["d_x"] = views(fill(*x.shape, dtype=x.dtype))
        out["d_weight"], out["d_bias"] = fill(width), fill(width)
        fs.fs_layer_norm_backward(z, w, out["mean"], out["rstd"], views(d_y), out["d_x"],
                                  out["d_weight"], out["d_bias"], d_total=at(d_total),
                                  lengths=lengths)
    return out


# type, batch, rows, width, options
NORMS = [
    (BF, 1, 1, 1, {}),
    (F4, 2, 3, 5, {"residual": True}),
    (BF, 3, 7, 64, {"residual": True, "ragged": True}),
    (HF, 2, 33, 96, {"ragged": True}),
    (F4, 2, 40, 200, {"residual": True}),
    (BF, 1, 130, 256, {}),
    (HF, 4, 31, 512, {"residual": True, "shift": 30.0}),
    (F4, 3, 177, 777, {"ragged": True}),
    (BF, 2, 50, 1024, {"residual": True}),
    (HF, 2, 9, 1999, {"residual": True}),
    (BF, 1, 1100, 2048, {}),
    (F4, 1, 5, 4096, {"residual": True, "shift": 1000.0}),
    (BF, 32, 1, 4096, {"residual": True}),
    (BF, 2, 600, 2560, {"residual": True, "ragged": True}),
    (HF, 1, 20, 5000, {}),
    (BF, 2, 17, 8192, {"residual": True}),
    (BF, 1, 9, 16384, {"residual": True}),
    (F4, 1, 4, 16383, {"residual": True}),
    (BF, 9000, 1, 40, {}),
]


def norm_inputs(case):
    dtype, B, n, width, opt = case
    g = gen(17 * width + n)
    x = (randn(g, B, n, width, std=1.5) + opt.get("shift", 0.3)).to(dtype)
    kw = {"eps": 1e-5}
    if opt.get("residual"):
        kw["residual"] = randn(g, B, n, width, dtype=dtype)
        kw["d_total"] = randn(g, B, n, width, dtype=dtype, std=0.1)
    if opt.get("ragged"):
        kw["lengths"] = torch.randint(0, n + 1, (B,), generator=g, dtype=I4)
    w, b = 1 + randn(g, width, std=0.2), randn(g, width, std=0.2)
    return x, w, b, randn(g, B, n, width, dtype=dtype, std=0.1), kw


@pytest.mark.parametrize("case", NORMS, ids=lambda c: "-".join(str(x) for x in c[:4]))
def test_layer_norm(fs, case):
    x, w, b, d_y, kw = norm_inputs(case)
    print(case, flush=True)
    compare(norm_run(fs, x, w, b, d_y=d_y, **kw), norm_reference(x, w, b, d_y=d_y, **kw))


@pytest.mark.parametrize("views", [wider, rows_first], ids=["wider", "rows_first"])
@pytest.mark.parametrize("case", [NORMS[2], NORMS[7], NORMS[12], NORMS[13]],
                         ids=lambda c: "-".join(str(x) for x in c[:4]))
def test_layer_norm_strides(fs, case, views):
    x, w, b, d_y, kw = norm_inputs(case)
    print(case, flush=True)
    compare(norm_run(fs, x, w, b, d_y=d_y, views=views, **kw),
            norm_reference(x, w, b, d_y=d_y, **kw))


def test_layer_norm_without_weights(fs):
    x, _, _, d_y, kw = norm_inputs(NORMS[8])
    compare(norm_run(fs, x, None, None, d_y=d_y, **kw),
            norm_reference(x, None, None, d_y=d_y, **kw))


def test_layer_norm_padding_is_never_read(fs):
    x, w, b, d_y, kw = norm_inputs((BF, 3, 20, 512, {"residual": True}))
    kw["lengths"] = torch.tensor([20, 7, 0], dtype=I4)
    ref = norm_reference(x, w, b, d_y=d_y, **kw)
    for t in (x, kw["residual"], d_y, kw["d_total"]):
        t[1, 7:] = NAN
        t[2] = math.inf
    compare(norm_run(fs, x, w, b, d_y=d_y, **kw), ref)


def test_layer_norm_no_rows(fs):
    for B, n in ((0, 4), (3, 0)):
        out = norm_run(fs, torch.zeros(B, n, 64), torch.ones(64), torch.ones(64), 1e-5,
                       d_y=torch.zeros(B, n, 64))
        torch.cuda.synchronize()
        assert (out["d_weight"] == 0).all() and (out["d_bias"] == 0).all()


def test_layer_norm_broadcast_inputs(fs):
    """Inputs broadcast by a stride of 0: each row's gradient is written."""
    g = gen(5)
    x = randn(g, 1, 1, 128, dtype=BF).cuda().expand(2, 9, 128)
    d_y = randn(g, 2, 1, 128, dtype=BF).cuda().expand(2, 9, 128)
    w, b = 1 + randn(g, 128, std=0.2), randn(g, 128)
    out = {"y": fill(2, 9, 128, dtype=BF), "mean": fill(2, 9), "rstd": fill(2, 9),
           "d_x": fill(2, 9, 128, dtype=BF), "d_weight": fill(128), "d_bias": fill(128)}
    fs.fs_layer_norm(x, w.cuda(), b.cuda(), out["y"], mean=out["mean"], rstd=out["rstd"])
    fs.fs_layer_norm_backward(x, w.cuda(), out["mean"], out["rstd"], d_y, out["d_x"],
                              out["d_weight"], out["d_bias"])
    compare(out, norm_reference(x.cpu(), w, b, 1e-5, d_y=d_y.cpu()))


# ---- rows in 8-bit integers -----------------------------------------------

QUANTS = [(BF, 1, 1), (F4, 3, 7), (HF, 5, 64), (BF, 40, 128), (F4, 33, 200), (HF, 9, 512),
          (BF, 17, 1111), (F4, 8, 2048), (BF, 8, 4096), (HF, 3, 8192), (BF, 2, 20000),
          (F4, 2, 65536), (BF, 1500, 96)]


def quant_inputs(dtype, rows, width):
    x = randn(gen(rows + width), rows, width)
    x = (x * torch.logspace(-3, 3, rows)[:, None]).to(dtype)
    if width > 4:
        # halves of the largest are ties (63.5), as are its other odd multiples of 1 / 254
        top = x.abs().amax(1)
        x[:, 1], x[:, 2] = top / 2, -top / 2
        x[:, 3] = -top
    if rows > 2:
        x[2] = 0
    return x


def quant_run(fs, x, views=lambda t: t):
    q, s = views(fill(*x.shape, dtype=torch.int8)), fill(x.shape[0])
    fs.fs_quantize_rows(views(x.cuda()), q, s)
    torch.cuda.synchronize()
    return q.cpu(), s.cpu()


@pytest.mark.parametrize("views", [lambda t: t, wider], ids=["whole", "wider"])
@pytest.mark.parametrize("case", QUANTS, ids=str)
def test_quantize_rows(fs, case, views):
    x = quant_inputs(*case)
    print(case, flush=True)
    q, s = quant_run(fs, x, views)
    rq, rs = quantize_reference(x)
    assert torch.equal(q, rq) and torch.equal(s, rs)


def test_quantize_ties_and_borders(fs):
    """Every multiple of half a step, and its neighbours in fp32."""
    for top in (127.0, 254.0, 1.0, 2.0 ** -140, 3e38, 0.7):
        v = torch.arange(-254, 255, dtype=torch.float64) / 254 * top
        v = v.float()
        x = torch.cat((v, torch.nextafter(v, torch.full_like(v, math.inf)).clamp(-top, top),
                       torch.nextafter(v, torch.full_like(v, -math.inf)).clamp(-top, top)))[None]
        q, s = quant_run(fs, x.contiguous())
        rq, rs = quantize_reference(x)
        assert torch.equal(q, rq) and torch.equal(s, rs), top


def test_quantize_rows_that_are_not_finite(fs):
    x = randn(gen(1), 4, 100, dtype=BF)
    x[0, 3], x[1, 99], x[2, 0] = math.inf, NAN, -math.inf
    q, s = quant_run(fs, x)
    rq, rs = quantize_reference(x)
    assert torch.isnan(s[:3]).all() and (q[:3] == 0).all()
    assert torch.equal(q[3], rq[3]) and s[3] == rs[3]


# output type, m, n, k, bias
PRODUCTS = [
    (F4, 1, 1, 1, True), (BF, 1, 1, 0, True), (BF, 1, 17, 16, False), (F4, 3, 5, 100, True),
    (BF, 8, 700, 4096, False), (HF, 16, 33, 1111, True), (BF, 17, 64, 64, False),
    (F4, 32, 100, 300, True), (BF, 64, 129, 1000, False), (HF, 65, 64, 128, True),
    (BF, 65, 3, 31, False), (F4, 100, 333, 144, True), (BF, 300, 257, 257, False),
    (HF, 200, 190, 4112, True), (BF, 130, 130, 9000, True), (F4, 513, 500, 2048, False),
    (BF, 1500, 1900, 272, True), (HF, 2000, 1777, 333, False), (BF, 3500, 3400, 400, True),
    (F4, 70000, 65, 48, False), (BF, 66, 70000, 100, True),
]


def product_inputs(case):
    dtype, m, n, k, bias = case
    g = gen(m + 3 * n + k)
    q = lambda r: torch.randint(-128, 128, (r, k), generator=g, dtype=torch.int8)
    s = lambda r: 0.01 + torch.rand(r, generator=g)
    return q(m), s(m) / (k + 1), q(n), s(n) / 100, (randn(g, n, std=0.3) if bias else None)


def product_run(fs, dtype, q_x, s_x, q_w, s_w, bias, views=lambda t: t):
    y = views(fill(q_x.shape[0], q_w.shape[0], dtype=dtype))
    fs.fs_quantized_product(views(q_x.cuda()), s_x.cuda(), views(q_w.cuda()), s_w.cuda(), y,
                            bias=gpu(bias))
    torch.cuda.synchronize()
    return y


def product_check(y, dtype, q_x, s_x, q_w, s_w, bias):
    # (fp64 products of whole numbers below 2^53 are exact)
    p = (q_x.double() @ q_w.double().t()) * s_x.double()[:, None] * s_w.double()
    if max(y.shape) <= 64:
        ref = product_reference(q_x, s_x, q_w, s_w, dtype, bias)
        assert torch.equal(ref[0], p if bias is None else p + bias.double())
    from layers_reference import W, half_step, tiny_of
    v = p if bias is None else p + bias.double()
    print(check("y", y, (v, 3 * W * p.abs() + (W + half_step(dtype)) * v.abs() + tiny_of(dtype))))


@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: "-".join(str(x) for x in c))
def test_quantized_product(fs, case):
    print(case, flush=True)
    args = product_inputs(case)
    product_check(product_run(fs, case[0], *args), case[0], *args)


@pytest.mark.parametrize("case", [(BF, 8, 100, 320, True), (F4, 100, 200, 320, False),
                                  (HF, 1500, 2000, 160, True), (BF, 130, 130, 9008, True)],
                         ids=lambda c: "-".join(str(x) for x in c))
def test_quantized_product_strides(fs, case):
    print(case, flush=True)
    args = product_inputs(case)
    product_check(product_run(fs, case[0], *args, views=wider), case[0], *args)
    # rows further apart that are still aligned
    product_check(product_run(fs, case[0], *args, views=lambda t: torch.cat((t, t), 1)[:, :t.shape[1]]
                              if t.dtype == torch.int8 else t), case[0], *args)


def test_quantized_product_largest_sums(fs):
    """128 x 128 x 65536 is the largest sum: 2^30."""
    for m in (3, 70):
        q = torch.full((m, 65536), -128, dtype=torch.int8)
        s = torch.full((m,), 2.0 ** -15)
        y = product_run(fs, F4, q, s, q, s, None)
        assert (y == 1.0).all()


def test_quantized_product_scale_nan_poisons_its_row_alone(fs):
    args = list(product_inputs((BF, 70, 90, 64, False)))
    args[1] = args[1].clone()
    args[1][5] = NAN
    y = product_run(fs, BF, *args)
    assert torch.isnan(y[5]).all() and torch.isfinite(y[:5]).all() and torch.isfinite(y[6:]).all()


def test_quantized_product_no_rows(fs):
    for m, n in ((0, 5), (5, 0)):
        z = lambda r: torch.zeros(r, 32, dtype=torch.int8)
        product_run(fs, BF, z(m), torch.zeros(m), z(n), torch.zeros(n), None)


# ---- distillation -----------------------------------------------------------

# type, rows, classes, k, T, options
DISTILLS = [
    (F4, 1, 1, 1, 1.0, {}),
    (BF, 3, 2, 5, 2.0, {}),
    (BF, 7, 100, 3, 1.0, {"short": True}),
    (HF, 20, 1000, 8, 0.5, {"idle": True}),
    (F4, 9, 2049, 64, 4.0, {"short": True}),
    (BF, 5, 9000, 16, 1.0, {"mass": True}),
    (BF, 2, 32000, 300, 2.0, {"short": True, "idle": True}),
    (F4, 3, 50001, 20, 1.0, {"masked": True}),
    (HF, 1, 131072, 1024, 1.0, {"mass": True}),
    (F4, 1100, 515, 4, 1.0, {"masked": True, "short": True}),
    (BF, 1030, 4100, 33, 3.0, {"idle": True}),
]


def distill_inputs(case):
    dtype, R, V, k, T, opt = case
    g = gen(R + V + k)
    x = randn(g, R, V, dtype=dtype, std=2.0)
    ids = torch.randint(0, V, (R, k), generator=g, dtype=I4)  # some twice in a row
    t = randn(g, R, k, std=2.0) + 4
    kw = {}
    if opt.get("short"):
        ids[torch.rand(R, k, generator=g) < 0.3] = -1
        ids[0, 0] = V + 3
        t[-1, -1] = -math.inf
    if opt.get("masked"):
        x[torch.rand(R, V, generator=g) < 0.2] = -math.inf
        x.scatter_(1, ids.clamp(0, V - 1).long(), 1.25)
    if opt.get("idle"):
        kw["active"] = (torch.rand(R, generator=g) < 0.7).to(torch.uint8)
        kw["active"][0] = 1
    if opt.get("mass"):
        kw["teacher_lse"] = (torch.logsumexp(t.double() / T, 1) + 0.4).float()
    return x, ids, t, T, 0.5 + torch.rand(R, generator=g), kw


def distill_run(fs, x, ids, t, T, d_loss=None, views=lambda t: t, **kw):
    kw = {a: gpu(b) for a, b in kw.items()}
    X, ids, t = views(x.cuda()), ids.cuda(), t.cuda()
    R = x.shape[0]
    out = {"loss": fill(R), "lse": fill(R)}
    fs.fs_distill_loss(X, ids, t, out["loss"], out["lse"], temperature=T, **kw)
    if d_loss is None:
        return out, None
    g = d_loss.cuda()
    out["d_logits"] = views(fill(*x.shape, dtype=x.dtype))
    fs.fs_distill_loss_backward(X, ids, t, out["lse"], g, out["d_logits"], temperature=T, **kw)
    one = {"loss": fill(R), "lse": fill(R), "d_logits": views(fill(*x.shape, dtype=x.dtype))}
    fs.fs_distill_loss(X, ids, t, one["loss"], one["lse"], temperature=T, d_loss=g,
                       d_logits=one["d_logits"], **kw)
    return out, one


@pytest.mark.parametrize("views", [lambda t: t, wider], ids=["whole", "wider"])
@pytest.mark.parametrize("case", DISTILLS, ids=lambda c: "-".join(str(x) for x in c[:5]))
def test_distill(fs, case, views):
    x, ids, t, T, g, kw = distill_inputs(case)
    print(case, flush=True)
    out, one = distill_run(fs, x, ids, t, T, g, views, **kw)
    ref = distill_reference(x, ids, t, T, d_loss=g, **kw)
    compare(out, ref)
    compare(one, ref)


def test_distill_rows_without_anything(fs):
    """No entry, no finite logit, not active, no weight in the total: zeros, and rows
    that are not active are never read."""
    x, ids, t, T, g, _ = distill_inputs((BF, 8, 5000, 4, 2.0, {}))
    ids[0] = -1
    t[1] = -math.inf
    x[2] = -math.inf
    active = torch.ones(8, dtype=torch.bool)
    active[3] = False
    ref = distill_reference(x, ids, t, T, d_loss=g, active=active)
    x[3], t[3] = NAN, NAN
    g[4] = 0
    ref["d_logits"][0][4] = 0
    ref["d_logits"][1][4] = 0
    out, one = distill_run(fs, x, ids, t, T, g, active=active)
    for o in (out, one):
        compare(o, ref)
        assert (o["d_logits"][[0, 1, 2, 3, 4]] == 0).all()
        assert o["lse"][2] == -math.inf and o["lse"][3] == 0


def test_distill_masked_class_of_the_teacher(fs):
    """A teacher's class that the student masks: an infinite loss, a finite gradient."""
    x, ids, t, T, g, _ = distill_inputs((F4, 2, 300, 3, 1.0, {}))
    x[0, ids[0, 0]] = -math.inf
    out, one = distill_run(fs, x, ids, t, T, g)
    ref = distill_reference(x, ids, t, T, d_loss=g)
    for o in (out, one):
        assert o["loss"][0] == math.inf
        check("d_logits", o["d_logits"], ref["d_logits"])


def test_distill_nan_poisons_its_row_alone(fs):
    for R, V in ((4, 20000), (1500, 300)):
        x, ids, t, T, g, _ = distill_inputs((BF, R, V, 4, 1.0, {}))
        x[1, 77] = NAN
        for o in distill_run(fs, x, ids, t, T, g):
            assert torch.isnan(o["loss"][1]) and torch.isnan(o["d_logits"][1]).all()
            assert torch.isfinite(o["loss"][[0, 2, 3]]).all()
            assert torch.isfinite(o["d_logits"][[0, 2, 3]]).all()


def test_distill_large_logits(fs):
    """Logits far from zero: their differences count."""
    x, ids, t, T, g, _ = distill_inputs((F4, 4, 3000, 8, 1.0, {}))
    x = x + 1000
    ref = distill_reference(x, ids, t, T, d_loss=g)
    for o in distill_run(fs, x, ids, t, T, g):
        compare(o, ref)


# ---- balance ------------------------------------------------------------------

# type, batch, rows, experts, k, options
BALANCES = [
    (F4, 1, 1, 1, 1, {}),
    (BF, 2, 5, 3, 2, {"normalize": True}),
    (HF, 3, 40, 8, 8, {"ragged": True, "normalize": True}),
    (BF, 1, 64, 64, 8, {"normalize": True}),
    (F4, 2, 333, 16, 2, {"ragged": True}),
    (BF, 2, 1000, 32, 1, {}),
    (HF, 4, 301, 60, 4, {"ragged": True}),
    (F4, 1, 700, 128, 6, {"normalize": True}),
    (BF, 1, 3001, 160, 8, {"normalize": True, "ragged": True}),
    (BF, 3, 150, 256, 32, {"normalize": True}),
    (F4, 1, 90, 333, 9, {}),
    (HF, 2, 70, 512, 12, {"normalize": True}),
    (F4, 2, 33, 1024, 32, {"ragged": True}),
    (BF, 1, 50, 777, 5, {"normalize": True}),
    (BF, 700, 3, 40, 2, {"ragged": True}),
]


def balance_inputs(case):
    dtype, B, n, E, k, opt = case
    g = gen(n + E + k)
    x = (randn(g, B, n, E) + randn(g, E, std=0.7)).to(dtype)
    kw = {"normalize": opt.get("normalize", False)}
    if opt.get("ragged"):
        kw["lengths"] = torch.randint(0, n + 1, (B,), generator=g, dtype=I4)
    scale = 4096.0 if dtype == HF else 1.0
    d_loss = (torch.rand(B, 2, generator=g) - 0.3) * scale
    return x, k, d_loss, randn(g, B, n, k, std=0.1), kw


def balance_run(fs, x, k, d_loss=None, d_gates=None, views=lambda t: t, **kw):
    kw = {a: gpu(b) for a, b in kw.items()}
    B, n, E = x.shape
    X = views(x.cuda())
    out = {"ids": fill(B, n, k, dtype=I4), "gates": fill(B, n, k), "counts": fill(B, E, dtype=I4),
           "loss": fill(B, 2), "lse": fill(B, n)}
    fs.fs_balance_loss(X, out["ids"], out["gates"], out["counts"], out["loss"], out["lse"], **kw)
    if d_loss is not None:
        out["d_logits"] = views(fill(*x.shape, dtype=x.dtype))
        fs.fs_balance_loss_backward(X, out["ids"], out["counts"], out["lse"], out["d_logits"],
                                    d_loss=d_loss.cuda(), d_gates=gpu(d_gates), **kw)
    return out


@pytest.mark.parametrize("views", [lambda t: t, wider, rows_first],
                         ids=["whole", "wider", "rows_first"])
@pytest.mark.parametrize("case", BALANCES, ids=lambda c: "-".join(str(x) for x in c[:5]))
def test_balance(fs, case, views):
    x, k, d_loss, d_gates, kw = balance_inputs(case)
    print(case, flush=True)
    compare(balance_run(fs, x, k, d_loss, d_gates, views, **kw),
            balance_reference(x, k, d_loss=d_loss, d_gates=d_gates, **kw))


def test_balance_without_gates(fs):
    x, k, d_loss, _, kw = balance_inputs(BALANCES[7])
    compare(balance_run(fs, x, k, d_loss, None, **kw),
            balance_reference(x, k, d_loss=d_loss, **kw))


def test_balance_ties_masks_and_padding(fs):
    """Equal logits go to the lowest column; masked columns come last, rows of -inf take
    no part; padding is never read."""
    g = gen(9)
    x = torch.randint(-2, 3, (3, 40, 24), generator=g).float()
    x[x == 0] = -0.0
    x[0, :20] = x[0, :20].abs()  # 0 and -0 are equal
    x[1, :, 3:] = -math.inf      # fewer columns than are chosen
    x[0, 5] = -math.inf
    x[2] = 1.0
    kw = {"normalize": True, "lengths": torch.tensor([40, 30, 11], dtype=I4)}
    d_loss, d_gates = torch.ones(3, 2), randn(g, 3, 40, 4, std=0.1)
    ref = balance_reference(x, 4, d_loss=d_loss, d_gates=d_gates, **kw)
    assert (ref["ids"][2, :11] == torch.arange(4)).all() and (ref["ids"][0, 5] == -1).all()
    x[1, 30:], x[2, 11:] = NAN, math.inf
    compare(balance_run(fs, x, 4, d_loss, d_gates, **kw), ref)


def test_balance_nan_counts_as_masked_in_the_choice(fs):
    x = randn(gen(2), 1, 6, 12)
    x[0, 2, 3] = NAN
    out = balance_run(fs, x, 3)
    torch.cuda.synchronize()
    assert torch.equal(out["ids"].cpu(), balance_reference(x, 3, False)["ids"])
    assert torch.isnan(out["loss"]).all() and torch.isnan(out["gates"][0, 2]).all()
    assert torch.isfinite(out["gates"][0, [0, 1, 3, 4, 5]]).all()


def test_balance_no_rows(fs):
    out = balance_run(fs, torch.zeros(3, 0, 8), 2, torch.ones(3, 2))
    torch.cuda.synchronize()
    assert (out["loss"] == 0).all() and (out["counts"] == 0).all()
    x, k, d_loss, d_gates, kw = balance_inputs((BF, 2, 9, 8, 2, {}))
    kw["lengths"] = torch.zeros(2, dtype=I4)
    out = balance_run(fs, x, k, d_loss, d_gates, **kw)
    torch.cuda.synchronize()
    assert (out["loss"] == 0).all() and (out["counts"] == 0).all() and (out["ids"] == -1).all()
    assert (out["d_logits"] == 0).all() and (out["lse"] == 0).all() and (out["gates"] == 0).all()


@pytest.mark.parametrize("normalize", [False, True])
def test_balance_gradient_of_another_choice(fs, normalize):
    """ids from elsewhere: a column twice, rows that take no part."""
    g = gen(4)
    x = randn(g, 2, 50, 20, dtype=BF)
    ids = torch.randint(0, 20, (2, 50, 3), generator=g, dtype=I4)
    ids[0, 7], ids[1, 40:] = -1, -1
    d_loss, d_gates = torch.rand(2, 2, generator=g), randn(g, 2, 50, 3, std=0.1)
    ref = balance_reference(x, 3, normalize, d_loss=d_loss, d_gates=d_gates, ids=ids)
    out = {"d_logits": fill(2, 50, 20, dtype=BF)}
    lse = torch.logsumexp(x.double(), 2).float()
    fs.fs_balance_loss_backward(x.cuda(), ids.cuda(), ref["counts"].cuda(), lse.cuda(),
                                out["d_logits"], d_loss=d_loss.cuda(), d_gates=d_gates.cuda(),
                                normalize=normalize)
    compare(out, {"d_logits": ref["d_logits"]})
