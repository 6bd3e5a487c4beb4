"""Refusals of include/fs_layers.h (bad arguments are reported on the host, before
any device is looked at: no compute calls, so they run without a GPU), and the
references' gradients against differences of their values."""
import ctypes
import math

import pytest
import torch

from layers_reference import (balance_reference, distill_reference, norm_reference,
                              product_reference, quantize_reference)
from streaming_sinkhorn_solver_amd import binding
from streaming_sinkhorn_solver_amd.binding import (BalanceDesc, DistillDesc, LayerNormDesc,
                                                   QuantizedProductDesc, Rows)

F8 = torch.float64
A = [x << 20 for x in range(1, 16)]  # addresses; no call gets as far as using them
NONE = Rows(None, 0, 0, 0)


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def refused(lib, status, word, want=binding.FS_ERR_INVALID_ARG):
    assert status == want, binding.fs_last_error()
    assert word in binding.fs_last_error(), binding.fs_last_error()


def view(at, n, w):
    return Rows(at, n * w, w, 0)


# ---- layer norm ----------------------------------------------------------------

def norm(lib, x=None, r=NONE, w=A[2], b=A[3], z=NONE, y=None, mean=A[6], rstd=A[7], **kw):
    a = LayerNormDesc(1, 2, 5, 64, 1e-5)
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.fs_layer_norm(ctypes.byref(a), x or view(A[0], 5, 64), r, w, b, z,
                             y or view(A[5], 5, 64), mean, rstd, None)


def norm_back(lib, z=None, mean=A[6], rstd=A[7], g=None, gz=NONE, gx=None, dw=A[10], db=A[11],
              ws=A[12], size=1 << 20, **kw):
    a = LayerNormDesc(1, 2, 5, 64, 1e-5)
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.fs_layer_norm_backward(ctypes.byref(a), z or view(A[0], 5, 64), A[2], mean, rstd,
                                      g or view(A[8], 5, 64), gz, gx or view(A[9], 5, 64), dw, db,
                                      ws, size, None)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=3), "fs_dtype"), (dict(batch=-1), "batch"), (dict(batch=1 << 16, n=1 << 15), "2^31"),
    (dict(width=0), "width"), (dict(width=16385), "width"), (dict(eps=-1.0), "eps"),
    (dict(eps=math.nan), "eps"), (dict(eps=math.inf), "eps")], ids=str)
def test_layer_norm_bad_sizes(lib, kw, word):
    refused(lib, norm(lib, **kw), word)
    refused(lib, norm_back(lib, **kw), word)
    a = LayerNormDesc(1, 2, 5, 64, 1e-5)
    for k, v in kw.items():
        setattr(a, k, v)
    assert lib.fs_layer_norm_workspace_bytes(ctypes.byref(a)) == 0


def test_layer_norm_bad_tensors(lib):
    refused(lib, norm(lib, x=Rows(None, 320, 64, 0)), "x must be")
    refused(lib, norm(lib, x=view(A[0] + 1, 5, 64)), "aligned")
    refused(lib, norm(lib, y=Rows(A[5], 320, 63, 0)), "overlap")
    refused(lib, norm(lib, y=Rows(A[5], 0, 64, 0)), "overlap")
    refused(lib, norm(lib, x=Rows(A[0], 320, -64, 0)), "stride")
    refused(lib, norm(lib, y=view(A[0] + 64, 5, 64)), "y overlaps")
    refused(lib, norm(lib, r=view(A[1], 5, 64)), "both or neither")
    refused(lib, norm(lib, z=view(A[4], 5, 64)), "both or neither")
    refused(lib, norm(lib, r=view(A[1], 5, 64), z=view(A[5], 5, 64)), "overlaps y")
    refused(lib, norm(lib, r=view(A[1], 5, 64), z=view(A[1], 5, 64)), "total overlaps")
    refused(lib, norm(lib, mean=A[2] + 8), "mean overlaps")
    refused(lib, norm(lib, mean=A[7]), "rstd overlaps mean")
    refused(lib, norm(lib, w=A[2] + 2), "weight is not aligned")
    refused(lib, norm_back(lib, mean=None), "mean must be")
    refused(lib, norm_back(lib, rstd=None), "rstd must be")
    refused(lib, norm_back(lib, gx=view(A[8], 5, 64)), "d_x overlaps")
    refused(lib, norm_back(lib, db=A[10] + 4), "d_bias overlaps d_weight")
    refused(lib, norm_back(lib, ws=A[12] + 8), "workspace", binding.FS_ERR_WORKSPACE)
    refused(lib, norm_back(lib, size=255), "workspace", binding.FS_ERR_WORKSPACE)
    refused(lib, norm_back(lib, ws=A[9]), "d_x overlaps")
    assert lib.fs_layer_norm(None, NONE, NONE, None, None, NONE, NONE, None, None, None) == \
        binding.FS_ERR_INVALID_ARG


# ---- rows in 8-bit integers ------------------------------------------------------

def test_quantize_refusals(lib):
    def call(dtype=1, rows=4, width=64, x=A[0], sx=64, q=A[1], sq=64, s=A[2]):
        return lib.fs_quantize_rows(dtype, rows, width, x, sx, q, sq, s, None)
    refused(lib, call(dtype=5), "fs_dtype")
    refused(lib, call(rows=-1), "rows")
    refused(lib, call(width=0), "width")
    refused(lib, call(width=65537), "width")
    refused(lib, call(x=None), "x must be")
    refused(lib, call(x=A[0] + 1), "aligned")
    refused(lib, call(sq=63), "overlap")
    refused(lib, call(q=A[0] + 16), "q overlaps")
    refused(lib, call(s=A[1]), "scale overlaps")
    refused(lib, call(s=None), "scale must be")


def product(lib, ws=A[6], size=1 << 20, **kw):
    a = QuantizedProductDesc(1, 4, 6, 32, A[0], 32, A[1], A[2], 32, A[3], A[4], A[5], 6)
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.fs_quantized_product(ctypes.byref(a), ws, size, None)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=-1), "fs_dtype"), (dict(m=-1), "needs"), (dict(k=65537), "needs"),
    (dict(n=(1 << 24) + 1), "needs"), (dict(m=1 << 20, n=1 << 20), "2^36"),
    (dict(q_x=None), "q_x must be"), (dict(q_w=None), "q_w must be"), (dict(y=None), "y must be"),
    (dict(y=A[5] + 1), "aligned"), (dict(y_stride=5), "overlap"), (dict(y=A[2]), "y overlaps"),
    (dict(scale_x=None), "scale_x must be"), (dict(scale_w=A[3] + 2), "aligned"),
    (dict(q_x_stride=-1), "stride")], ids=str)
def test_product_refusals(lib, kw, word):
    refused(lib, product(lib, **kw), word)


def test_product_workspace(lib):
    refused(lib, product(lib, ws=None), "workspace", binding.FS_ERR_WORKSPACE)
    refused(lib, product(lib, size=64), "workspace", binding.FS_ERR_WORKSPACE)
    bad = QuantizedProductDesc(1, -1, 3, 3)
    assert lib.fs_quantized_product_workspace_bytes(ctypes.byref(bad)) == 0
    assert lib.fs_quantized_product_workspace_bytes(None) == 0
    assert binding.fs_quantized_product_workspace_bytes(8, 8192, 4096) >= 256
    assert lib.fs_quantized_product(None, A[0], 256, None) == binding.FS_ERR_INVALID_ARG


# ---- losses ----------------------------------------------------------------------

def distill(lib, x=None, loss=A[3], lse=A[4], g=None, gx=NONE, ws=A[7], size=1 << 20, **kw):
    a = DistillDesc(1, 4, 64, 3, 1.0, A[1], A[2])
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.fs_distill_loss(ctypes.byref(a), x or Rows(A[0], 0, 64, 0), loss, lse, g, gx, ws,
                               size, None)


def distill_back(lib, x=None, lse=A[4], g=A[5], gx=None, **kw):
    a = DistillDesc(1, 4, 64, 3, 1.0, A[1], A[2])
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.fs_distill_loss_backward(ctypes.byref(a), x or Rows(A[0], 0, 64, 0), lse, g,
                                        gx or Rows(A[6], 0, 64, 0), None)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=7), "fs_dtype"), (dict(rows=-1), "rows"), (dict(classes=0), "classes"),
    (dict(classes=(1 << 24) + 1), "classes"), (dict(k=0), "k must"), (dict(k=1025), "k must"),
    (dict(temperature=0.0), "temperature"), (dict(temperature=math.nan), "temperature"),
    (dict(temperature=math.inf), "temperature"), (dict(temperature=-1.0), "temperature"),
    (dict(ids=None), "ids must"), (dict(teacher=None), "teacher must"),
    (dict(ids=A[1] + 1), "aligned")], ids=str)
def test_distill_bad_sizes(lib, kw, word):
    refused(lib, distill(lib, **kw), word)
    refused(lib, distill_back(lib, **kw), word)


def test_distill_bad_tensors(lib):
    grad = Rows(A[6], 0, 64, 0)
    refused(lib, distill(lib, g=A[5]), "both or neither")
    refused(lib, distill(lib, gx=grad), "both or neither")
    refused(lib, distill(lib, g=A[5], gx=Rows(A[6], 0, 63, 0)), "overlap")
    refused(lib, distill(lib, g=A[5], gx=Rows(A[0], 0, 64, 0)), "d_logits overlaps")
    refused(lib, distill(lib, g=A[5], gx=Rows(A[4] - 64, 0, 64, 0)), "d_logits overlaps lse")
    refused(lib, distill(lib, loss=None), "loss must")
    refused(lib, distill(lib, lse=None), "lse must")
    refused(lib, distill(lib, loss=A[4]), "lse overlaps loss")
    refused(lib, distill(lib, loss=A[2] + 4), "loss overlaps")
    refused(lib, distill(lib, ws=A[7] + 4), "workspace", binding.FS_ERR_WORKSPACE)
    refused(lib, distill(lib, size=0), "workspace", binding.FS_ERR_WORKSPACE)
    refused(lib, distill_back(lib, lse=None), "lse must")
    refused(lib, distill_back(lib, g=None), "d_loss must")
    refused(lib, distill_back(lib, gx=Rows(A[4] - 64, 0, 64, 0)), "d_logits overlaps")
    assert lib.fs_distill_loss(None, NONE, None, None, None, NONE, None, 0, None) == \
        binding.FS_ERR_INVALID_ARG


def balance(lib, x=None, ids=A[1], gates=A[2], counts=A[3], loss=A[4], lse=A[5], ws=A[6],
            size=1 << 20, **kw):
    a = BalanceDesc(1, 2, 5, 8, 2, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.fs_balance_loss(ctypes.byref(a), x or view(A[0], 5, 8), ids, gates, counts, loss,
                               lse, ws, size, None)


def balance_back(lib, ids=A[1], counts=A[3], lse=A[5], g=A[4], gg=A[2], gx=None, **kw):
    a = BalanceDesc(1, 2, 5, 8, 2, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.fs_balance_loss_backward(ctypes.byref(a), view(A[0], 5, 8), ids, counts, lse, g, gg,
                                        gx or view(A[7], 5, 8), None)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=3), "fs_dtype"), (dict(batch=-1), "batch"), (dict(batch=65536), "batch"),
    (dict(batch=65535, n=1 << 20), "2^31"), (dict(experts=0), "experts"),
    (dict(experts=1025), "experts"), (dict(k=0), "k must"), (dict(k=9), "k must"),
    (dict(experts=64, k=33), "k must"), (dict(batch=1, n=1 << 30, k=2), "n * k")], ids=str)
def test_balance_bad_sizes(lib, kw, word):
    refused(lib, balance(lib, **kw), word)
    refused(lib, balance_back(lib, **kw), word)


def test_balance_bad_tensors(lib):
    for name in ("ids", "gates", "counts", "loss", "lse"):
        refused(lib, balance(lib, **{name: None}), f"{name} must")
        refused(lib, balance(lib, **{name: A[0] + 4}), f"{name} overlaps")
    refused(lib, balance(lib, gates=A[1]), "gates overlaps ids")
    refused(lib, balance(lib, size=8), "workspace", binding.FS_ERR_WORKSPACE)
    refused(lib, balance_back(lib, ids=None), "ids must")
    refused(lib, balance_back(lib, g=None), "d_loss must")
    refused(lib, balance_back(lib, gx=view(A[0], 5, 8)), "d_logits overlaps")
    refused(lib, balance_back(lib, gx=Rows(A[7], 40, 4, 0)), "overlap")


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 2, 8)
    with pytest.raises(TypeError, match="device tensor"):
        binding.fs_layer_norm(x, None, None, x)
    with pytest.raises(TypeError, match="device tensor"):
        binding.fs_quantize_rows(x[0], x[0], x[0])
    with pytest.raises(TypeError, match="device tensor"):
        binding.fs_distill_loss(x[0], x[0], x[0], x[0], x[0])
    with pytest.raises(TypeError, match="device tensor"):
        binding.fs_balance_loss(x, torch.zeros(1, 2, 1, dtype=torch.int32), x, x, x, x)


# ---- the references' gradients against differences ----------------------------------

def differences(f, x, step=1e-5):
    """Central differences of the scalar f at x (64 bits)."""
    out = torch.zeros_like(x)
    for i in range(x.numel()):
        at = x.clone().view(-1)
        at[i] += step
        hi = f(at.view_as(x))
        at[i] -= 2 * step
        out.view(-1)[i] = (hi - f(at.view_as(x))) / (2 * step)
    return out


def test_norm_gradient():
    g = torch.Generator().manual_seed(1)
    x, w, b, d = (torch.randn(*s, generator=g) for s in ((2, 3, 5), (5,), (5,), (2, 3, 5)))
    lens = torch.tensor([3, 1], dtype=torch.int32)
    ref = norm_reference(x, w, b, 1e-2, lengths=lens, d_y=d)
    from layers_reference import inside, norm_values

    def value(X, Wt, Bs):
        return float((norm_values(X, Wt, Bs, 1e-2, inside(2, 3, lens))[0] * d.to(F8)).sum())
    X, Wt, Bs = x.to(F8), w.to(F8), b.to(F8)
    assert torch.allclose(ref["d_x"][0], differences(lambda t: value(t, Wt, Bs), X), atol=1e-7)
    assert torch.allclose(ref["d_weight"][0], differences(lambda t: value(X, t, Bs), Wt), atol=1e-7)
    assert torch.allclose(ref["d_bias"][0], differences(lambda t: value(X, Wt, t), Bs), atol=1e-7)


@pytest.mark.parametrize("mass", [False, True])
def test_distill_gradient(mass):
    g = torch.Generator().manual_seed(2)
    x = torch.randn(3, 7, generator=g, dtype=F8)
    ids = torch.tensor([[1, 4, 1], [6, -1, 2], [0, 9, 3]], dtype=torch.int32)
    t, dl = torch.randn(3, 3, generator=g), torch.rand(3, generator=g)
    tl = torch.logsumexp(t.to(F8) / 1.7, 1).float() + 0.3 if mass else None
    ref = distill_reference(x, ids, t, 1.7, teacher_lse=tl, d_loss=dl)

    def value(X):
        return float((distill_reference(X, ids, t, 1.7, teacher_lse=tl)["loss"][0] * dl.to(F8)).sum())
    assert torch.allclose(ref["d_logits"][0], differences(value, x), atol=1e-7)
    if not mass:
        # a mean of logarithms against the definition: not negative, zero where they agree
        same = torch.full((3, 7), -math.inf, dtype=F8)
        ids = torch.tensor([[1, 4, 2], [6, 0, 2], [0, 5, 3]], dtype=torch.int32)
        same.scatter_(1, ids.long(), t.to(F8))
        assert (ref["loss"][0] >= 0).all()
        assert distill_reference(same, ids, t, 1.7)["loss"][0].abs().max() < 1e-12


@pytest.mark.parametrize("normalize", [False, True])
def test_balance_gradient(normalize):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 4, 5, generator=g, dtype=F8)
    lens = torch.tensor([4, 3], dtype=torch.int32)
    dl, dg = torch.rand(2, 2, generator=g), torch.randn(2, 4, 2, generator=g)
    ref = balance_reference(x, 2, normalize, lens, dl, dg)

    def value(X):
        r = balance_reference(X, 2, normalize, lens)
        assert torch.equal(r["ids"], ref["ids"])
        return float((r["loss"][0] * dl.to(F8)).sum() + (r["gates"][0] * dg.to(F8)).sum())
    assert torch.allclose(ref["d_logits"][0], differences(value, x), atol=1e-7)
    assert (ref["counts"].sum(1) == 2 * lens).all()


def test_quantized_rows_stand_for_their_values():
    x = torch.randn(9, 33, generator=torch.Generator().manual_seed(4))
    x[3] = 0
    q, s = quantize_reference(x)
    assert (q.to(F8) * s.to(F8)[:, None] - x.to(F8)).abs().max() <= 0.5001 * s.max()
    assert ((q.abs().amax(1) == 127) | (s == 0)).all()
    y, bound = product_reference(q, s, q, s, torch.float32)
    assert ((y - x.to(F8) @ x.to(F8).t()).abs() <= 33 * (s[:, None] * s * 127 * 1.01 + 1e-12)).all()
    # a half goes to the even one: 63.5 to 64, 31.5 (a quarter of the largest, less
    # half a step) to 32
    q, _ = quantize_reference(torch.tensor([[254.0, 127.0, -127.0, 63.0, 1.0, 3.0, 5.0]]))
    assert q.tolist() == [[127, 64, -64, 32, 0, 2, 2]]
