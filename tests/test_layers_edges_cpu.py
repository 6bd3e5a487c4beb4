"""What the binding and the host library of include/fs_layers.h answer at their edges:
calls that a user may get wrong, and sizes asked for before there is memory.  No
kernel runs."""
import ctypes
import random

import pytest
import torch

from streaming_sinkhorn_solver_amd import binding
from streaming_sinkhorn_solver_amd.binding import DistillDesc, LayerNormDesc, QuantizedProductDesc, Rows

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


def product_bytes(lib, m, n, k, x, sx, w, sw):
    a = QuantizedProductDesc(0, m, n, k, x, sx, None, w, sw)
    return int(lib.fs_quantized_product_workspace_bytes(ctypes.byref(a)))


@pytest.mark.parametrize("m,n,k", [(33, 40, 64), (1800, 1700, 256), (70, 90, 8192), (2000, 33, 16)])
def test_product_workspace_before_there_is_memory(lib, m, n, k):
    """An operand that is not there yet may come to stand anywhere: the answer is enough
    for every address that its stride allows."""
    asked = product_bytes(lib, m, n, k, None, k, None, k)
    for x in (A[0], A[0] + 1, A[0] + 8):
        for w in (A[1], A[1] + 2):
            need = product_bytes(lib, m, n, k, x, k, w, k)
            assert need <= asked
            assert (need < asked) == (x == A[0] or w == A[1])
            assert need <= product_bytes(lib, m, n, k, x, k, None, k) <= asked
    # few rows are read as they stand, and nothing is to be formed without rows
    assert product_bytes(lib, 8, n, k, None, k, None, k) == 256
    assert product_bytes(lib, m, 0, k, None, k, None, k) == 256


def test_product_workspace_of_given_operands(lib, calls):
    """The binding answers for contiguous, aligned operands, or for those it is given."""
    m, n, k = 70, 90, 320
    x, w = torch.zeros(m, k + 16, dtype=I1), torch.zeros(n, k + 5, dtype=I1)
    aligned = binding.fs_quantized_product_workspace_bytes(m, n, k)
    assert aligned == product_bytes(lib, m, n, k, A[0], k, A[1], k)
    for qx, qw in ((x[:, :k], None), (x[:, 1:k + 1], None), (None, w[:, :k]), (x[:, :k], w[:, 1:k + 1]),
                   (x[:, 3:k + 3], w[:, 1:k + 1])):
        p = [(t.data_ptr(), t.stride(0)) if t is not None else (A[0], k) for t in (qx, qw)]
        assert binding.fs_quantized_product_workspace_bytes(m, n, k, q_x=qx, q_w=qw) == \
            product_bytes(lib, m, n, k, *p[0], *p[1])
    assert binding.fs_quantized_product_workspace_bytes(m, n, k, q_w=w[:, 1:k + 1]) > aligned
    with pytest.raises(ValueError, match="q_x must be"):
        binding.fs_quantized_product_workspace_bytes(m, n, k, q_x=x)


def two_outputs(lib, batch, n, width, at_y, y, at_total, total):
    """What the layer norm says of y and total as these views (offsets and strides in
    elements); a call that it allows is refused for its rstd, which is its mean."""
    a = LayerNormDesc(0, batch, n, width, 1e-5)
    view = lambda base, s: Rows(base, s[0], s[1], 0)
    flat = (n * width, width)
    status = lib.fs_layer_norm(ctypes.byref(a), view(A[0], flat), view(A[1], flat), None, None,
                               view(A[2] + 4 * at_total, total), view(A[2] + 4 * at_y, y), A[3], A[3],
                               None)
    assert status == binding.FS_ERR_INVALID_ARG
    return binding.fs_last_error()


def elements(batch, n, width, at, strides):
    rows = [at + b * strides[0] + i * strides[1] for b in range(batch) for i in range(n)]
    all_ = [r + e for r in rows for e in range(width)]
    return set(all_), len(set(all_)) == len(all_)


def test_two_output_views_of_one_buffer(lib):
    """Rows 0..9 and 5..14 of one buffer overlap; slices side by side, rows or batches in
    turn do not."""
    flat = (640, 64)
    assert "total overlaps y" in two_outputs(lib, 1, 10, 64, 0, flat, 5 * 64, flat)
    assert "total overlaps y" in two_outputs(lib, 2, 10, 64, 0, flat, 64, flat)
    assert "total overlaps y" in two_outputs(lib, 1, 10, 64, 5 * 64 + 3, flat, 0, flat)
    assert "total overlaps y" in two_outputs(lib, 1, 10, 64, 0, (0, 100), 32, (0, 100))
    assert "total overlaps y" in two_outputs(lib, 1, 10, 64, 0, (0, 128), 64, (0, 192))
    # (the second batch entry of one is the first of the other)
    assert "total overlaps y" in two_outputs(lib, 2, 10, 64, 0, flat, 640, flat)
    for y, total, s in ((0, 1280, flat), (0, 64, (1280, 128)), (64, 0, (1280, 128)),
                        (0, 64, (1440, 144)), (8, 72, (1584, 144)), (0, 640, (1280, 64)),
                        (0, 1 << 16, flat), (0, 64, (128, 640))):
        assert "rstd overlaps mean" in two_outputs(lib, 2, 10 if s[1] != 640 else 3, 64, y, s, total, s)


def test_two_output_views_of_any_strides(lib):
    """Against the sets of their elements: views that share one are refused, views of equal
    strides that share none are not."""
    rng = random.Random(5)
    seen = {True: 0, False: 0}
    while min(seen.values()) < 3000:
        batch, n, width = rng.randint(1, 4), rng.randint(1, 4), rng.randint(1, 5)
        s = (rng.randint(1, 40), rng.randint(1, 40))
        t = s if rng.random() < 0.8 else (rng.randint(1, 40), rng.randint(1, 40))
        at = rng.randint(0, 60), rng.randint(0, 60)
        (one, fits), (other, fits2) = (elements(batch, n, width, x, y) for x, y in zip(at, (s, t)))
        if not (fits and fits2):
            continue
        said = two_outputs(lib, batch, n, width, at[0], s, at[1], t)
        if "is written and its strides overlap" in said:
            continue  # (rows and batches that interleave: refused for themselves)
        meet = bool(one & other)
        used = [x for x, size in ((0, batch), (1, n)) if size > 1]
        alike = all(s[x] == t[x] for x in used)
        apart = max(one) < min(other) or max(other) < min(one)
        if meet or alike or apart:
            assert ("total overlaps y" in said) == meet, (batch, n, width, at, s, t, said)
            assert meet or "rstd overlaps mean" in said
            seen[meet] += 1
