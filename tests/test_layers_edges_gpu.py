"""The operators of include/fs_layers.h at their edges: calls that the documentation
allows and few make, and the refusals of calls that it does not."""
import math

import pytest
import torch

from layers_reference import balance_reference
from test_layers_gpu import balance_run, compare, gen, randn

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
