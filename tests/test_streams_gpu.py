"""Calls on a stream that is not the current one: the order a caller has to give,
and temporary memory that belongs to the call's stream."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture
def side():
    return torch.cuda.Stream()


class Allocations:
    """The streams that torch.empty's device memory was taken from, and where."""

    def __init__(self, monkeypatch):
        self.seen, real = [], torch.empty

        def empty(*args, **kw):
            t = real(*args, **kw)
            if t.is_cuda:
                self.seen.append((torch.cuda.current_stream().cuda_stream, t.data_ptr(), t.nbytes))
            return t

        monkeypatch.setattr(torch, "empty", empty)

    def check(self, side, freed):
        """Some memory was taken, all of it from the side stream's pool, none of it
        a block that the current stream has just given back."""
        assert self.seen
        for stream, at, size in self.seen:
            assert stream == side.cuda_stream
            for lo, n in freed:
                assert at + size <= lo or lo + n <= at


def give_back(sizes):
    """Blocks of these sizes returned to the current stream's pool."""
    blocks = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in sizes]
    return [(b.data_ptr(), b.nbytes) for b in blocks]


def attention(fs, stream=None, order=lambda: None):
    """Forward with split keys, and backward; every output."""
    g = torch.Generator(device="cuda").manual_seed(1)
    q, d_o = (torch.randn(2, 40, 4, 64, generator=g, device="cuda").to(BF) for _ in range(2))
    k, v = (torch.randn(2, 2500, 2, 64, generator=g, device="cuda").to(BF) for _ in range(2))
    o, dq, dk, dv = (torch.full_like(t, float("nan")) for t in (q, q, k, v))
    lse = torch.full((2, 4, 40), float("nan"), device="cuda")
    order()
    fs.fs_attention_forward(q, k, v, o, lse, stream=stream)
    fs.fs_attention_backward(q, k, v, o, lse, d_o, dq, dk, dv, stream=stream)
    return o, lse, dq, dk, dv


def norm(fs, stream=None, order=lambda: None):
    g = torch.Generator(device="cuda").manual_seed(2)
    x, gy = (torch.randn(2, 300, 4, 64, generator=g, device="cuda") for _ in range(2))
    w = torch.rand(64, generator=g, device="cuda")
    dx, dw = torch.full_like(x, float("nan")), torch.full_like(w, float("nan"))
    order()
    fs.fs_qk_norm_rotate_backward(x, None, w, None, gy, None, dx, None, dw, stream=stream)
    return dx, dw


def solver(fs, stream=None, order=lambda: None):
    """Every solver call that allocates something for itself."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n, m, d, eps = 300, 260, 3, 0.5
    X, V = (torch.rand(n, d, generator=g, device="cuda") for _ in range(2))
    Y = torch.rand(m, d, generator=g, device="cuda")
    a, b = torch.full((n,), 1 / n, device="cuda"), torch.full((m,), 1 / m, device="cuda")
    f, gp, HV = (torch.zeros(s, device="cuda") for s in (n, m, (n, d)))
    pick = torch.arange(20, dtype=torch.int32, device="cuda")
    order()
    kw = {"stream": stream}
    Xs, ws, perm = fs.fs_morton_sort(X, a, **kw)
    back = fs.fs_unpermute(Xs, perm, **kw)
    C, W = fs.fs_centroids(Xs, ws, 8, **kw)
    lifted = fs.fs_lift(W, n, 8, **kw)
    p = fs.fs_potentials_init(X, Y, a, b, dv_max=d + 2, f=f, g=gp, **kw)
    fs.fs_bs_attach(p, **kw)
    fs.fs_sinkhorn_solve(p, f, gp, eps_end=eps, iters_per_stage=20, **kw)
    value = fs.fs_dual_value(p, f, gp, **kw)
    errs = fs.fs_sampled_marginal_error(X, Y, a, b, f, gp, eps, pick, pick, **kw)
    fs.fs_hvp(p, eps, f, gp, X, Y, V, HV, **kw)
    return Xs, ws, perm, back, C, W, lifted, f, gp, value, errs, HV


@pytest.mark.parametrize("work", [attention, norm, solver])
def test_temporary_memory_is_the_streams_own(fs, monkeypatch, side, work):
    """Each workspace that a call allocates for itself comes from the pool of the
    stream that it runs on, given as a stream or as its handle."""
    assert fs.fs_attention_workspace_bytes(*(torch.empty(2, r, h, 64, device="cuda", dtype=BF)
                                             for r, h in ((40, 4), (2500, 2), (2500, 2)))) > 256
    want = work(fs)
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        freed, allocations = [], None

        def order():
            nonlocal freed, allocations
            freed = give_back([1 << x for x in range(9, 25)])
            side.wait_stream(torch.cuda.current_stream())
            allocations = Allocations(monkeypatch)

        got = work(fs, stream, order)
        monkeypatch.undo()
        torch.cuda.synchronize()
        allocations.check(side, freed)
        for x, y in zip(want, got):
            assert torch.equal(x, y)


@pytest.mark.parametrize("work", [attention, norm, solver])
def test_other_stream_in_order(fs, side, work):
    """The side stream waits for the fills and the current one for the side
    stream, with no wait of the host between: equal bits."""
    want = work(fs)
    got = work(fs, side, lambda: side.wait_stream(torch.cuda.current_stream()))
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(want, got):
        assert torch.equal(x, y)
