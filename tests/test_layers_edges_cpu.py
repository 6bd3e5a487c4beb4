"""What the binding and the host library of include/fs_layers.h answer at their edges:
calls that a user may get wrong, and sizes asked for before there is memory.  No
kernel runs."""
import pytest
import torch

from streaming_sinkhorn_solver_amd import binding

F4, I1 = torch.float32, torch.int8


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
