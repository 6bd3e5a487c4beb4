"""What the binding and the host library of include/fs_layers.h answer at their edges:
calls that a user may get wrong, and sizes asked for before there is memory.  No
kernel runs."""
import ctypes

import pytest
import torch

from streaming_sinkhorn_solver_amd import binding
from streaming_sinkhorn_solver_amd.binding import DistillDesc, Rows

F4, I1 = torch.float32, torch.int8
A = [x << 20 for x in range(1, 16)]  # addresses; no call gets as far as using them
NONE = Rows(None, 0, 0, 0)


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def refused(status, word):
    assert status == binding.FS_ERR_INVALID_ARG, binding.fs_last_error()
    assert word in binding.fs_last_error(), binding.fs_last_error()


@pytest.fixture
def calls(monkeypatch):
    """The binding on host tensors, with nothing behind it: the calls that it would
    have passed on to the library."""
    seen = []
    monkeypatch.setattr(binding, "_dtype_of", lambda t, name: binding._DTYPES[t.dtype])
    monkeypatch.setattr(binding, "_on", lambda t, name, dev: None)
    monkeypatch.setattr(binding, "_call", lambda fn, where, *args: seen.append(where))
    return seen


# m, n and the shape of a y that is not [m, n]: too few rows, too narrow, transposed, one
# row or column too few or too many
@pytest.mark.parametrize("m,n,shape", [
    (70, 90, (10, 90)), (70, 90, (70, 80)), (1, 90, (1, 64)), (90, 70, (70, 90)), (70, 90, (69, 90)),
    (70, 90, (71, 90)), (70, 1, (70, 2)), (4, 4, (4, 0))], ids=str)
def test_product_refuses_a_y_of_another_shape(calls, m, n, shape):
    q = lambda r: torch.zeros(r, 32, dtype=I1)
    work = torch.zeros(1 << 16, dtype=torch.uint8)

    def call(y):
        binding.fs_quantized_product(q(m), torch.zeros(m), q(n), torch.zeros(n), y, workspace=work)
    with pytest.raises(ValueError, match="y must be"):
        call(torch.zeros(shape))
    assert not calls
    call(torch.zeros(m, n))
    assert calls == ["fs_quantized_product"]


def test_distill_rest_refusals(lib):
    """lse_rest is an output of the loss and an input of the gradient, which needs it
    below a temperature of 2^-10."""
    def desc(rest, T=1.0):
        return ctypes.byref(DistillDesc(1, 4, 64, 3, T, A[1], A[2], None, None, rest))

    def loss(rest):
        return lib.fs_distill_loss(desc(rest), Rows(A[0], 0, 64, 0), A[3], A[4], None, NONE, A[7],
                                   1 << 20, None)

    def back(rest, T=1.0, gx=A[6]):
        return lib.fs_distill_loss_backward(desc(rest, T), Rows(A[0], 0, 64, 0), A[4], A[5],
                                            Rows(gx, 0, 64, 0), None)
    refused(loss(A[8] + 2), "lse_rest is not aligned")
    refused(loss(A[4]), "lse_rest overlaps lse")
    refused(loss(A[1]), "lse_rest overlaps an input")
    refused(back(A[6]), "d_logits overlaps an input")
    refused(back(A[8] + 2), "lse_rest is not aligned")
    refused(back(None, 2.0 ** -11), "lse_rest")
