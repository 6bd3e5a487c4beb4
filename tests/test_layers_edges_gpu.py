"""The operators of include/fs_layers.h at their edges: calls that the documentation
allows and few make, and the refusals of calls that it does not."""
import math

import pytest
import torch

from layers_reference import balance_reference, distill_reference
from test_layers_gpu import balance_run, compare, distill_run, fill, gen, gpu, randn

pytestmark = pytest.mark.gpu

BF, HF, F4 = torch.bfloat16, torch.float16, torch.float32
I4, I1 = torch.int32, torch.int8
NAN, INF = math.nan, math.inf
TYPES = pytest.mark.parametrize("dtype", [BF, HF, F4], ids=["bf16", "fp16", "fp32"])


@TYPES
def test_product_refuses_a_y_of_another_shape(fs, dtype):
    """Refused before any launch: what lies around such a y stays as it is."""
    for m, n, shape in ((70, 90, (10, 90)), (1, 90, (1, 64)), (90, 70, (70, 90))):
        q = lambda r: torch.ones(r, 32, dtype=I1, device="cuda")
        s = lambda r: torch.ones(r, device="cuda")
        buf = torch.full((4 * m * n,), 7.0, dtype=dtype, device="cuda")
        y = buf[:shape[0] * shape[1]].view(shape)
        with pytest.raises(ValueError, match="y must be"):
            fs.fs_quantized_product(q(m), s(m), q(n), s(n), y)
        torch.cuda.synchronize()
        assert (buf == 7).all()



@pytest.mark.parametrize("m,n,k", [(70, 90, 320), (1800, 1700, 256)])
def test_product_workspace_of_a_slice(fs, m, n, k):
    """A program that keeps its own workspace asks with the operands it has; the call
    writes nothing behind what was asked for."""
    g = gen(k)
    x = torch.randint(-128, 128, (m, k + 5), generator=g, dtype=I1).cuda()[:, 1:k + 1]
    w = torch.randint(-128, 128, (n, k), generator=g, dtype=I1).cuda()
    sx, sw = torch.rand(m, device="cuda"), torch.rand(n, device="cuda")
    small = fs.fs_quantized_product_workspace_bytes(m, n, k)
    need = fs.fs_quantized_product_workspace_bytes(m, n, k, q_x=x, q_w=w)
    assert need > small
    own, y = fill(m, n), fill(m, n)
    with pytest.raises(fs.FsError, match="workspace"):
        fs.fs_quantized_product(x, sx, w, sw, y,
                                workspace=torch.zeros(small, dtype=torch.uint8, device="cuda"))
    space = torch.full((need + 256,), 0x55, dtype=torch.uint8, device="cuda")
    fs.fs_quantized_product(x, sx, w, sw, y, workspace=space[:need])
    fs.fs_quantized_product(x, sx, w, sw, own)
    assert torch.equal(y, own) and (space[need:] == 0x55).all()
    p = (x.double() @ w.double().t().contiguous()) * sx.double()[:, None] * sw.double()
    assert ((y - p).abs() <= 4 * 2.0 ** -24 * p.abs()).all()


# ---- balance -----------------------------------------------------------------

def poison(x):
    """Rows of the first batch entry: of NaN alone, of NaN and -inf, with one NaN, with an
    infinity, of -inf alone (the only one of them that takes no part)."""
    E = x.shape[2]
    x[0, 1] = NAN
    x[0, 2] = -INF
    x[0, 2, E - 1] = NAN
    x[0, 4, E // 2] = NAN
    x[0, 5, 0] = INF
    x[0, 7] = -INF
    return [1, 2, 4, 5], 7


@TYPES
@pytest.mark.parametrize("n", [9, 700])  # one workgroup an entry, several
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (8, 1), (9, 3), (60, 4), (64, 8), (256, 8), (250, 9),
                                 (512, 2), (1000, 32), (1024, 8)])
def test_balance_rows_of_nan(fs, dtype, n, E, k):
    """A row that holds anything but -inf takes part: a NaN (of a whole row, too) shows in
    all that the row has a share in, and nowhere else."""
    print(dtype, n, E, k, flush=True)
    g = gen(E + k)
    x = randn(g, 2, n, E, dtype=dtype)
    bad, masked = poison(x)
    if E == 1:
        bad, masked = [1, 2, 4, 5], 7
        x[0, 2] = NAN
    rest = torch.ones(2, n, dtype=torch.bool)
    rest[0, bad] = False
    for normalize in (False, True):
        out = balance_run(fs, x, k, torch.rand(2, 2, generator=g), randn(g, 2, n, k), normalize=normalize)
        torch.cuda.synchronize()
        out = {a: t.cpu() for a, t in out.items()}
        # the choice: NaN as -inf, the lowest of equal columns
        order = torch.where(torch.isnan(x), torch.full_like(x, -INF), x).float()
        ids = torch.sort(order, dim=2, descending=True, stable=True)[1][..., :k].to(I4)
        ids[0, masked] = -1
        assert torch.equal(out["ids"], ids)
        for b in range(2):
            took = ids[b][ids[b, :, 0] >= 0]
            assert torch.equal(out["counts"][b], torch.bincount(took.flatten(), minlength=E).to(I4))
        for name in ("gates", "lse", "d_logits"):
            assert torch.isnan(out[name][0, bad]).all(), name
            assert torch.isfinite(out[name][rest]).all(), name
            assert (out[name][0, masked] == 0).all(), name
        assert torch.isnan(out["loss"][0]).all() and torch.isfinite(out["loss"][1]).all()


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("E,k", [(7, 2), (64, 8), (256, 8), (333, 12), (1024, 4)])
def test_balance_gradient_of_logits_far_from_zero(fs, normalize, E, k):
    """A row's common offset changes neither the choice nor a probability, nor then the
    gradient of the balance and of the gates.  Logits that are whole multiples of 2^-13
    stay what they are under an offset of 1000, so that the outputs are within the bound
    of those without it."""
    g = gen(E)
    x = torch.round(randn(g, 2, 60, E) * 8192) / 8192
    far = x + 1000
    assert torch.equal(far.double(), x.double() + 1000)
    d_loss, d_gates = torch.tensor([[3.0, 0.0], [50.0, 0.0]]), randn(g, 2, 60, k, std=0.1)
    ref = balance_reference(x, k, normalize, d_loss=d_loss, d_gates=d_gates)
    out = balance_run(fs, far, k, d_loss, d_gates, normalize=normalize)
    compare(out, {a: ref[a] for a in ("ids", "counts", "gates", "d_logits")})


# ---- distillation ------------------------------------------------------------

def distill_step(fs, x, ids, t, T, d_loss, teacher_lse=None, **kw):
    """Loss, lse and gradient of one call."""
    out = {"loss": fill(x.shape[0]), "lse": fill(x.shape[0]),
           "d_logits": fill(*x.shape, dtype=x.dtype)}
    fs.fs_distill_loss(gpu(x), gpu(ids), gpu(t), out["loss"], out["lse"], temperature=T,
                       teacher_lse=gpu(teacher_lse), d_loss=gpu(d_loss), d_logits=out["d_logits"], **kw)
    return out


def far_inputs(R, V, k, T, offset, step, mass):
    """Logits of a student and a teacher, a few T apart and whole multiples of `step`, and
    the same beside an offset that leaves them what they are.  (near, far): x, t,
    teacher_lse each."""
    g = gen(V + k)
    x, t = (torch.round(randn(g, *s, std=2 * T) / step) * step for s in ((R, V), (R, k)))
    ids = torch.randint(0, V, (R, k), generator=g, dtype=I4)
    ids[0, -1] = -1
    x.scatter_(1, ids.clamp(0).long(), t)  # (a student that begins to know)
    fx, ft = x + offset, t + offset
    assert torch.equal(fx.double(), x.double() + offset)
    assert torch.equal(ft.double(), t.double() + offset)
    lse = far = None
    if mass:
        far = (torch.logsumexp(ft.double() / T, 1) + 0.4).float()
        lse = far.double() - offset / T  # what the rounded one stands for
    return (x, t.double(), lse), (fx, ft, far), ids, 0.5 + torch.rand(R, generator=g)


# temperature, offset, the logits' step: an fp32 number at the offset holds it
FAR = [(1.0, 1000.0, 2.0 ** -13), (0.3, -300.0, 2.0 ** -14), (1e-3, 14.0, 2.0 ** -20),
       (2.0 ** -10, 14.0, 2.0 ** -20), (2.0 ** -20, 14.0, 2.0 ** -20), (1e5, 3e6, 0.5)]


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("R,V,k", [(5, 300, 8), (3, 9000, 200), (2, 40001, 3), (2, 70000, 16), (140, 40000, 3)],
                         ids=str)
@pytest.mark.parametrize("T,offset,step", FAR, ids=str)
def test_distill_logits_far_from_zero(fs, T, offset, step, R, V, k, mass):
    """A common offset of a row's logits changes no probability: loss and gradient of one
    call are within the bounds of the logits without it, whatever offset / T is."""
    print(T, offset, R, V, k, mass, flush=True)
    near, far, ids, d_loss = far_inputs(R, V, k, float(torch.tensor(T)), offset, step, mass)
    T = float(torch.tensor(T))  # as the call's fp32 holds it
    ref = distill_reference(near[0], ids, near[1], T, teacher_lse=near[2], d_loss=d_loss)
    out = distill_step(fs, far[0], ids, far[1], T, d_loss, teacher_lse=far[2])
    compare(out, {a: ref[a] for a in ("loss", "d_logits")})
    compare(out, {"lse": distill_reference(far[0], ids, far[1], T)["lse"]})


@TYPES
@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("T", [0.25, 1.0, 2.0])
def test_distill_teacher_masked_by_the_lowest_number(fs, dtype, mass, T):
    """Entries and columns that hold the type's lowest number weigh nothing, also where
    their quotient by the temperature is no fp32 number."""
    g = gen(6)
    x, t = randn(g, 4, 500, dtype=dtype, std=2.0), randn(g, 4, 6)
    ids = torch.stack([torch.randperm(500, generator=g)[:6] for _ in range(4)]).to(I4)
    t[:, 4:] = torch.finfo(F4).min
    lse = (torch.logsumexp(t[:, :4].double() / T, 1) + 0.3).float() if mass else None
    dl = 0.5 + torch.rand(4, generator=g)
    ref = distill_reference(x, ids[:, :4], t[:, :4], T, teacher_lse=lse, d_loss=dl)
    compare(distill_step(fs, x, ids, t, T, dl, teacher_lse=lse), ref)
    x[:, 400:] = torch.finfo(dtype).min
    ids = ids % 400
    ref = distill_reference(x[:, :400], ids[:, :4], t[:, :4], T, teacher_lse=lse, d_loss=dl)
    out = distill_step(fs, x, ids, t, T, dl, teacher_lse=lse)
    assert (out["d_logits"][:, 400:] == 0).all()
    out["d_logits"] = out["d_logits"][:, :400]
    compare(out, ref)


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_distill_teacher_that_is_not_finite(fs, bad, mass):
    """A NaN or +inf of the teacher's shows in its row's loss and gradient, and in no
    other row."""
    g = gen(7)
    x, t = randn(g, 4, 700), randn(g, 4, 5)
    ids = torch.randint(0, 700, (4, 5), generator=g, dtype=I4)
    t[2, 3] = bad
    lse = torch.full((4,), 3.0) if mass else None
    out = distill_step(fs, x, ids, t, 1.5, torch.ones(4), teacher_lse=lse)
    torch.cuda.synchronize()
    assert torch.isnan(out["loss"][2]) and torch.isnan(out["d_logits"][2]).all()
    for name in ("loss", "d_logits"):
        assert torch.isfinite(out[name][[0, 1, 3]]).all()
    assert torch.isfinite(out["lse"]).all()


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("R,V,k", [(5, 300, 8), (3, 9000, 200), (2, 70000, 16), (1100, 4100, 3)], ids=str)
@pytest.mark.parametrize("T,offset,step", FAR, ids=str)
def test_distill_gradient_alone_of_logits_far_from_zero(fs, T, offset, step, R, V, k, mass):
    """With what the stored lse lacks in fp32 the gradient call, too, is within the bound
    of the logits without their offset; rows that take no part, or hold -inf alone, have
    no such rest."""
    print(T, offset, R, V, k, mass, flush=True)
    T = float(torch.tensor(T))
    near, far, ids, d_loss = far_inputs(R, V, k, T, offset, step, mass)
    if R > 1000:  # (their reference is slow)
        near, far, ids, d_loss = ([t if t is None else t[::50] for t in near], far, ids, d_loss)
        keep = torch.arange(0, R, 50)
    else:
        keep = torch.arange(R)
    loss, lse, rest, dx = fill(R), fill(R), fill(R), fill(R, V)
    x, t, tl = map(gpu, far)
    active = torch.ones(R, dtype=torch.uint8)
    active[R // 2 + 1:R // 2 + 2] = 0
    kw = dict(temperature=T, teacher_lse=tl, active=gpu(active), lse_rest=rest)
    fs.fs_distill_loss(x, gpu(ids), t, loss, lse, **kw)
    fs.fs_distill_loss_backward(x, gpu(ids), t, lse, gpu(d_loss), dx, **kw)
    ref = distill_reference(near[0], ids[keep], near[1], T, teacher_lse=near[2], d_loss=d_loss[keep],
                            active=active[keep])
    compare({"loss": loss[gpu(keep)], "d_logits": dx[gpu(keep)]}, {a: ref[a] for a in ("loss", "d_logits")})
    assert (rest.abs() <= 2.0 ** -24 * lse.abs() + 1e-37).all()
    assert (rest[gpu(active) == 0] == 0).all()


def test_distill_rest_of_an_lse_that_is_not_finite(fs):
    x, ids, t = randn(gen(1), 3, 50), torch.zeros(3, 1, dtype=I4), torch.zeros(3, 1)
    x[0], x[1, 7] = -INF, NAN
    loss, lse, rest, dx = fill(3), fill(3), fill(3), fill(3, 50)
    fs.fs_distill_loss(gpu(x), gpu(ids), gpu(t), loss, lse, lse_rest=rest)
    fs.fs_distill_loss_backward(gpu(x), gpu(ids), gpu(t), lse, torch.ones(3, device="cuda"), dx,
                                lse_rest=rest)
    torch.cuda.synchronize()
    assert lse[0] == -INF and rest[0] == 0 and rest[1] == 0 and (dx[0] == 0).all()
    assert torch.isnan(dx[1]).all() and torch.isfinite(dx[2]).all()


def test_distill_gradient_alone_at_a_small_temperature(fs):
    """Below 2^-10 the stored lse alone does not carry the gradient: refused."""
    x, t = gpu(randn(gen(1), 3, 50)), torch.zeros(3, 1, device="cuda")
    ids = torch.zeros(3, 1, dtype=I4, device="cuda")
    lse, one, dx = torch.zeros(3, device="cuda"), torch.ones(3, device="cuda"), torch.zeros_like(x)
    with pytest.raises(fs.FsError, match="lse_rest"):
        fs.fs_distill_loss_backward(x, ids, t, lse, one, dx, temperature=2.0 ** -11)
    with pytest.raises(ValueError, match="lse_rest"):
        fs.fs_distill_loss_backward(x, ids, t, lse, one, dx, lse_rest=one[:2].clone())


@TYPES
@pytest.mark.parametrize("rows,classes", [(1024, 8200), (1030, 8201), (1024, 10240), (1100, 10241),
                                          (1024, 16384), (2048, 8200), (2300, 8203)], ids=str)
def test_distill_many_rows_of_medium_length(fs, dtype, rows, classes):
    """From 1024 rows on, rows of 8193 to 10240 classes (fp32: of 70 MB in all; to 16384
    for the loss alone) are kept in part and read again."""
    print(dtype, rows, classes, flush=True)
    g = gen(classes)
    x = randn(g, rows, classes, dtype=dtype, std=2.0)
    ids = torch.randint(0, classes, (rows, 3), generator=g, dtype=I4)
    ids[0, 0] = classes - 1
    t, dl = randn(g, rows, 3), 0.5 + torch.rand(rows, generator=g)
    keep = torch.arange(0, rows, 97)
    ref = distill_reference(x[keep], ids[keep], t[keep], 1.5, d_loss=dl[keep])
    for out in distill_run(fs, x, ids, t, 1.5, dl):
        compare({k: v[keep.cuda()] for k, v in out.items()}, ref)
