"""The operators of include/fs_layers.h as a program uses them: together, captured,
on other streams, side by side, on memory beyond 32 bits, with workspaces of any
content; and the binding's refusals."""
import math

import pytest
import torch

from attention_reference import check
from layers_reference import (balance_reference, distill_reference, norm_reference,
                              product_reference, quantize_reference)
from test_layers_gpu import BF, F4, HF, I4, fill, gen, randn

pytestmark = pytest.mark.gpu

NAN = math.nan


class Use:
    """Inputs, outputs and workspaces of every operator; step() runs them all.  small:
    sizes of single launches, else of ranges, parts and joins."""

    def __init__(self, fs, small, dtype=BF, seed=0):
        self.fs, self.small = fs, small
        self.rows = 12 if small else 700
        self.width, self.classes, self.experts, self.k = (96, 500, 16, 2) if small else \
            (1000, 40000, 72, 4)
        self.m, self.n = (20, 50) if small else (70, 130)
        self.kk = 512 if small else 9001
        self.dtype = dtype
        R, W, V, E = self.rows, self.width, self.classes, self.experts
        D = 12 if small else 40  # rows of the distillation
        dev = dict(device="cuda")
        e = lambda *s, dtype=dtype: torch.empty(*s, dtype=dtype, **dev)
        self.x, self.r, self.dy, self.dz = (e(2, R, W) for _ in range(4))
        self.w, self.b = e(W, dtype=F4), e(W, dtype=F4)
        self.a, self.c = e(self.m, self.kk), e(self.n, self.kk)
        self.logits, self.ids, self.t = e(D, V), e(D, 6, dtype=I4), e(D, 6, dtype=F4)
        self.dl = e(D, dtype=F4)
        self.route = e(2, R, E)
        self.d_loss, self.d_gates = e(2, 2, dtype=F4), e(2, R, self.k, dtype=F4)
        self.fill(seed)
        f = lambda *s, dtype=F4: fill(*s, dtype=dtype)
        self.outs = dict(
            y=f(2, R, W, dtype=dtype), z=f(2, R, W, dtype=dtype), mean=f(2, R), rstd=f(2, R),
            dx=f(2, R, W, dtype=dtype), dw=f(W), db=f(W),
            qa=f(self.m, self.kk, dtype=torch.int8), sa=f(self.m),
            qc=f(self.n, self.kk, dtype=torch.int8), sc=f(self.n),
            scores=f(self.m, self.n, dtype=dtype),
            loss=f(D), lse=f(D), dlogits=f(D, V, dtype=dtype),
            loss2=f(D), lse2=f(D), dlogits2=f(D, V, dtype=dtype),
            chosen=f(2, R, self.k, dtype=I4), gates=f(2, R, self.k), counts=f(2, E, dtype=I4),
            balance=f(2, 2), blse=f(2, R), droute=f(2, R, E, dtype=dtype))

    def fill(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (self.x, self.r, self.dy, self.dz, self.w, self.b, self.a, self.c, self.t,
                  self.logits, self.route, self.d_loss, self.d_gates):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        self.dl.copy_(torch.rand(self.dl.shape, generator=g, device="cuda") + 0.5)
        self.ids.copy_(torch.randint(0, self.classes, self.ids.shape, generator=g, device="cuda"))

    def sizes(self):
        import ctypes
        fs = self.fs
        need = fs.QuantizedProductDesc(0, self.m, self.n, self.kk, None, self.kk, None, None, self.kk)
        return [fs.fs_layer_norm_workspace_bytes(self.x),
                int(fs.load().fs_quantized_product_workspace_bytes(ctypes.byref(need))),
                fs.fs_distill_workspace_bytes(self.logits, 6),
                fs.fs_balance_workspace_bytes(self.route, self.k)]

    def step(self, spaces=(None,) * 4, stream=None):
        fs, o, st = self.fs, self.outs, {"stream": stream}
        fs.fs_layer_norm(self.x, self.w, self.b, o["y"], residual=self.r, total=o["z"],
                         mean=o["mean"], rstd=o["rstd"], **st)
        fs.fs_layer_norm_backward(o["z"], self.w, o["mean"], o["rstd"], self.dy, o["dx"], o["dw"],
                                  o["db"], d_total=self.dz, workspace=spaces[0], **st)
        fs.fs_quantize_rows(self.a, o["qa"], o["sa"], **st)
        fs.fs_quantize_rows(self.c, o["qc"], o["sc"], **st)
        fs.fs_quantized_product(o["qa"], o["sa"], o["qc"], o["sc"], o["scores"], workspace=spaces[1],
                                **st)
        fs.fs_distill_loss(self.logits, self.ids, self.t, o["loss"], o["lse"], temperature=2.0,
                           d_loss=self.dl, d_logits=o["dlogits"], workspace=spaces[2], **st)
        fs.fs_distill_loss(self.logits, self.ids, self.t, o["loss2"], o["lse2"], temperature=2.0,
                           workspace=spaces[2], **st)
        fs.fs_distill_loss_backward(self.logits, self.ids, self.t, o["lse2"], self.dl,
                                    o["dlogits2"], temperature=2.0, **st)
        fs.fs_balance_loss(self.route, o["chosen"], o["gates"], o["counts"], o["balance"], o["blse"],
                           normalize=True, workspace=spaces[3], **st)
        fs.fs_balance_loss_backward(self.route, o["chosen"], o["counts"], o["blse"], o["droute"],
                                    d_loss=self.d_loss, d_gates=self.d_gates, normalize=True, **st)

    def results(self):
        torch.cuda.synchronize()
        return {x: t.clone() for x, t in self.outs.items()}

    def clear(self):
        for t in self.outs.values():
            t.fill_(NAN) if t.dtype.is_floating_point else t.fill_(-77)


def same(a, b):
    for x in a:
        assert torch.equal(a[x], b[x]), x


@pytest.mark.parametrize("small", [True, False])
def test_workspace_contents_do_not_matter(fs, small):
    """Equal calls give equal bits, whatever the workspace held, without a byte to
    spare and nothing written behind it."""
    use = Use(fs, small)
    use.step()
    first = use.results()
    assert all(not torch.isnan(t).any() for t in first.values() if t.dtype.is_floating_point)
    need = use.sizes()
    if not small:
        assert min(need) > 256
    spaces = [torch.full((n + 512,), 0xFF, dtype=torch.uint8, device="cuda") for n in need]
    for _ in range(2):
        use.clear()
        use.step([s[:n] for s, n in zip(spaces, need)])
        same(first, use.results())
    for s, n in zip(spaces, need):
        assert (s[n:] == 0xFF).all()


@pytest.mark.parametrize("small", [True, False])
def test_graph_replays(fs, small):
    """A captured step, replayed on new inputs, against eager steps between the replays."""
    use = Use(fs, small)
    spaces = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in use.sizes()]
    use.step(spaces)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        use.step(spaces)
    for seed in range(1, 4):
        use.fill(seed)
        use.step()
        eager = use.results()
        use.clear()
        graph.replay()
        same(eager, use.results())


@pytest.mark.parametrize("small", [True, False])
def test_other_stream_and_two_at_once(fs, small):
    """On a stream given as such or as a handle, in the order that the caller gives;
    and two steps in flight on two streams."""
    use = Use(fs, small)
    use.step()
    want = use.results()
    side = [torch.cuda.Stream() for _ in range(2)]
    for st in (side[0], side[0].cuda_stream):
        use.clear()
        side[0].wait_stream(torch.cuda.current_stream())
        use.step(stream=st)
        torch.cuda.current_stream().wait_stream(side[0])
        same(want, use.results())
    uses = [Use(fs, small, seed=x) for x in (5, 6)]
    for u in uses:
        u.step()
    wants = [u.results() for u in uses]
    for u in uses:
        u.clear()
    torch.cuda.synchronize()
    for u, s in zip(uses, side):
        for _ in range(3):
            u.step(stream=s)
    for u, w in zip(uses, wants):
        same(w, u.results())


def test_temporary_memory_is_the_streams_own(fs, monkeypatch):
    use = Use(fs, False)
    side, seen, real = torch.cuda.Stream(), [], torch.empty

    def empty(*args, **kw):
        t = real(*args, **kw)
        if t.is_cuda:
            seen.append(torch.cuda.current_stream().cuda_stream)
        return t

    side.wait_stream(torch.cuda.current_stream())
    monkeypatch.setattr(torch, "empty", empty)
    use.step(stream=side)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert seen and set(seen) == {side.cuda_stream}


@pytest.mark.parametrize("dtype", [BF, HF, F4], ids=["bf16", "fp16", "fp32"])
def test_a_student_of_a_plan(fs, dtype):
    """A cheaper matcher learns a converged plan's largest entries: the solver's
    potentials give the teacher's logits, layer norm the student's states, their
    8-bit scores the logits; distillation and a balance loss over the same scores
    give gradients that go back through the layer norm.  Every step is within its
    bound on what the step before it gave."""
    n, m, d, top = 150, 170, 96, 6
    g = gen(3)
    # the solver on the teacher's features
    X, Y = randn(g, n, 8, std=0.4).cuda(), randn(g, m, 8, std=0.4).cuda()
    a, b = torch.full((n,), 1 / n, device="cuda"), torch.full((m,), 1 / m, device="cuda")
    eps = 0.3
    _, f, pot, _ = fs.solve(X, Y, a, b, eps=eps, iters=100)
    plan = (f[:, None] + pot[None] - torch.cdist(X.double(), Y.double()).square().float()) / eps \
        + b.log()
    teacher, ids = plan.topk(top, dim=1)
    teacher, ids = teacher.contiguous(), ids.to(I4).contiguous()
    assert (plan.logsumexp(1).abs() < 0.05).all()  # rows of log-probabilities
    whole = torch.zeros(n, device="cuda")
    # the student
    x, r = randn(g, 1, n, d, dtype=dtype).cuda(), randn(g, 1, n, d, dtype=dtype).cuda()
    keys = randn(g, m, d, dtype=dtype).cuda()
    w, bias = (1 + randn(g, d, std=0.1)).cuda(), randn(g, d, std=0.1).cuda()
    z, y = fill(1, n, d, dtype=dtype), fill(1, n, d, dtype=dtype)
    mean, rstd = fill(1, n), fill(1, n)
    fs.fs_layer_norm(x, w, bias, y, residual=r, total=z, mean=mean, rstd=rstd)
    q, s, qk, sk = fill(n, d, dtype=torch.int8), fill(n), fill(m, d, dtype=torch.int8), fill(m)
    fs.fs_quantize_rows(y[0], q, s)
    fs.fs_quantize_rows(keys, qk, sk)
    scores = fill(n, m, dtype=F4)
    fs.fs_quantized_product(q, s, qk, sk, scores)
    loss, lse, d_scores = fill(n), fill(n), fill(n, m)
    share = torch.full((n,), 1 / n, device="cuda")
    fs.fs_distill_loss(scores, ids, teacher, loss, lse, temperature=2.0, teacher_lse=whole,
                       d_loss=share, d_logits=d_scores)
    chosen, gates, counts = fill(1, n, 2, dtype=I4), fill(1, n, 2), fill(1, m, dtype=I4)
    even, elz, d_even = fill(1, 2), fill(1, n), fill(1, n, m)
    d_loss = torch.tensor([[0.1, 0.01]], device="cuda")
    fs.fs_balance_loss(scores[None], chosen, gates, counts, even, elz)
    fs.fs_balance_loss_backward(scores[None], chosen, counts, elz, d_even, d_loss=d_loss)
    d_y = ((d_scores + d_even[0]) @ (qk.float() * sk[:, None]))[None].to(dtype)
    dx, dw, db = fill(1, n, d, dtype=dtype), fill(d), fill(d)
    fs.fs_layer_norm_backward(z, w, mean, rstd, d_y, dx, dw, db)
    torch.cuda.synchronize()
    c = lambda t: t.cpu()
    ref = norm_reference(c(x), c(w), c(bias), 1e-5, residual=c(r))
    for name, t in (("y", y), ("total", z), ("mean", mean), ("rstd", rstd)):
        check(name, t, ref[name])
    for t, qt, st in ((y[0], q, s), (keys, qk, sk)):
        rq, rs = quantize_reference(c(t))
        assert torch.equal(c(qt), rq) and torch.equal(c(st), rs)
    check("scores", scores, product_reference(c(q), c(s), c(qk), c(sk), F4))
    ref = distill_reference(c(scores), c(ids), c(teacher), 2.0, teacher_lse=c(whole),
                            d_loss=c(share))
    for name, t in (("loss", loss), ("lse", lse), ("d_logits", d_scores)):
        check(name, t, ref[name])
    ref = balance_reference(c(scores)[None], 2, False, d_loss=c(d_loss))
    assert torch.equal(c(chosen), ref["ids"]) and torch.equal(c(counts), ref["counts"])
    for name, t in (("gates", gates), ("loss", even), ("lse", elz), ("d_logits", d_even)):
        check(name, t, ref[name])
    ref = norm_reference(c(z), c(w), c(bias), 1e-5, d_y=c(d_y))
    for name, t in (("d_x", dx), ("d_weight", dw), ("d_bias", db)):
        check(name, t, ref[name])


def test_slices_of_one_buffer(fs):
    """Outputs side by side in one buffer; only rows of the call are written."""
    g = gen(8)
    x, r = randn(g, 2, 9, 64, dtype=BF).cuda(), randn(g, 2, 9, 64, dtype=BF).cuda()
    buf = fill(2, 11, 144, dtype=BF)
    y, z = buf[:, 1:10, 8:72], buf[:, 1:10, 72:136]
    fs.fs_layer_norm(x, None, None, y, residual=r, total=z)
    ref = norm_reference(x.cpu(), None, None, 1e-5, residual=r.cpu())
    check("y", y, ref["y"])
    check("total", z, ref["total"])
    rest = buf.clone()
    rest[:, 1:10, 8:136] = NAN
    assert torch.isnan(rest).all()


def test_offsets_beyond_32_bits(fs):
    """Views that span more than 2^32 elements: the last rows equal those of a call on
    them alone."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    far = (1 << 32) + 4096
    buf = torch.empty(far + (1 << 20), dtype=BF, device="cuda")
    tail = buf[-(1 << 20):]
    g = torch.Generator(device="cuda").manual_seed(4)
    buf[:4096].normal_(generator=g)
    tail.normal_(generator=g)
    stride = (far + 4096) // 2 // 8 * 8
    x = buf.as_strided((1, 3, 1024), (0, stride, 1))
    x[0, 1].normal_(generator=g)
    close = x.contiguous()

    def norm(t):
        y, dx = fill(1, 3, 1024, dtype=BF), fill(1, 3, 1024, dtype=BF)
        m, s = fill(1, 3), fill(1, 3)
        fs.fs_layer_norm(t, None, None, y, mean=m, rstd=s)
        fs.fs_layer_norm_backward(t, None, m, s, y, dx)
        return y, dx
    for p, q in zip(norm(x), norm(close)):
        assert torch.equal(p, q)

    def quant(t):
        q, s = fill(3, 1024, dtype=torch.int8), fill(3)
        fs.fs_quantize_rows(t[0], q, s)
        return q, s
    for p, q in zip(quant(x), quant(close)):
        assert torch.equal(p, q)

    def route(t):
        ids, gates, counts = fill(1, 3, 4, dtype=I4), fill(1, 3, 4), fill(1, 1024, dtype=I4)
        loss, lse, dx = fill(1, 2), fill(1, 3), fill(1, 3, 1024, dtype=BF)
        fs.fs_balance_loss(t, ids, gates, counts, loss, lse)
        fs.fs_balance_loss_backward(t, ids, counts, lse, dx, d_loss=torch.ones(1, 2, device="cuda"))
        return ids, gates, counts, loss, lse, dx
    for p, q in zip(route(x), route(close)):
        assert torch.equal(p, q)
    ids = torch.arange(15, device="cuda", dtype=I4).view(3, 5)
    te = torch.ones(3, 5, device="cuda")

    def distill(t):
        loss, lse, dx = fill(3), fill(3), fill(3, 1024, dtype=BF)
        fs.fs_distill_loss(t[0], ids, te, loss, lse, d_loss=torch.ones(3, device="cuda"), d_logits=dx)
        return loss, lse, dx
    for p, q in zip(distill(x), distill(close)):
        assert torch.equal(p, q)
    del x, buf, tail
    # a product with more than 2^32 outputs, its last block against a product alone
    m, n, k = 70000, 62000, 32
    y = torch.empty(m, n, dtype=BF, device="cuda")
    qx = torch.randint(-128, 128, (m, k), device="cuda", dtype=torch.int8, generator=g)
    qw = torch.randint(-128, 128, (n, k), device="cuda", dtype=torch.int8, generator=g)
    sx, sw = torch.rand(m, device="cuda", generator=g), torch.rand(n, device="cuda", generator=g)
    fs.fs_quantized_product(qx, sx, qw, sw, y)
    part = fill(200, 300, dtype=BF)
    fs.fs_quantized_product(qx[-200:], sx[-200:].clone(), qw[-300:], sw[-300:].clone(), part)
    assert torch.equal(y[-200:, -300:], part)


def test_many_rows(fs):
    """More rows than a grid has workgroups, and batches of one row."""
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(300000, 1, 24, generator=g, device="cuda")
    y, m, s, dx = torch.empty_like(x), fill(300000, 1), fill(300000, 1), torch.empty_like(x)
    dw, db = fill(24), fill(24)
    fs.fs_layer_norm(x, None, None, y, mean=m, rstd=s)
    fs.fs_layer_norm_backward(x, None, m, s, torch.ones_like(x), dx, dw, db)
    far = x.double() - x.double().mean(-1, keepdim=True)
    h = far / (far.square().mean(-1, keepdim=True) + 1e-5).sqrt()
    assert (y - h).abs().max() < 1e-5 and (db == 300000).all() and dx.abs().max() < 1e-4
    assert (dw - h.sum((0, 1))).abs().max() < 300000 * 2.0 ** -22
    x = torch.randn(1, 300000, 5, generator=g, device="cuda").to(HF)
    ids, gates, counts = fill(1, 300000, 2, dtype=I4), fill(1, 300000, 2), fill(1, 5, dtype=I4)
    loss, lse = fill(1, 2), fill(1, 300000)
    fs.fs_balance_loss(x, ids, gates, counts, loss, lse)
    want = torch.bincount(torch.sort(x.float(), dim=-1, descending=True, stable=True)[1][..., :2].flatten(),
                          minlength=5)
    assert torch.equal(counts[0].long(), want) and int(counts.sum()) == 600000
    t = torch.zeros(300000, 1, device="cuda")
    loss, lse = fill(300000), fill(300000)
    fs.fs_distill_loss(x[0], ids[0, :, :1].contiguous(), t, loss, lse)
    assert (loss - (lse - x[0].float().amax(1))).abs().max() < 1e-5


def test_binding_refuses(fs):
    x = torch.zeros(2, 3, 64, device="cuda", dtype=BF)
    v, i = torch.zeros(64, device="cuda"), torch.zeros(2, 3, 2, device="cuda", dtype=I4)
    st = torch.zeros(2, 3, device="cuda")
    with pytest.raises(TypeError, match="float32"):
        fs.fs_layer_norm(x, v.to(BF), None, x.clone())
    with pytest.raises(fs.FsError, match="y must be non-NULL"):
        fs.fs_layer_norm(x, v, None, None)
    with pytest.raises(TypeError, match="as the others"):
        fs.fs_layer_norm(x, v, None, x.float())
    with pytest.raises(ValueError, match="must be"):
        fs.fs_layer_norm(x, v[:32], None, x.clone())
    with pytest.raises(ValueError, match="contiguous"):
        fs.fs_layer_norm(x.transpose(1, 2).contiguous().transpose(1, 2), v, None, x.clone())
    with pytest.raises(fs.FsError, match="overlaps"):
        fs.fs_layer_norm(x, v, None, x)
    with pytest.raises(fs.FsError, match="mean must be non-NULL"):
        fs.fs_layer_norm_backward(x, v, None, st, x.clone(), x.clone())
    with pytest.raises(TypeError, match="device tensor"):
        fs.fs_layer_norm(x, v.cpu(), None, x.clone())
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        fs.fs_layer_norm(x.double(), v, None, x.clone())
    with pytest.raises(ValueError, match="width"):
        fs.fs_quantize_rows(x, x, v)
    with pytest.raises(TypeError, match="int8"):
        fs.fs_quantize_rows(x[0], x[0].clone(), v[:3].clone())
    q = torch.zeros(3, 64, device="cuda", dtype=torch.int8)
    with pytest.raises(ValueError, match="scale_w"):
        fs.fs_quantized_product(q, v[:3].clone(), q, v[:2].clone(), torch.zeros(3, 3, device="cuda"))
    with pytest.raises(TypeError, match="y must be float32"):
        fs.fs_quantized_product(q, v[:3].clone(), q, v[:3].clone(),
                                torch.zeros(3, 3, device="cuda", dtype=I4))
    with pytest.raises(fs.FsError, match="workspace"):
        big = torch.zeros(1800, 64, device="cuda", dtype=torch.int8)[:, :33]
        s = torch.zeros(1800, device="cuda")
        fs.fs_quantized_product(big, s, big, s, torch.zeros(1800, 1800, device="cuda"),
                                workspace=torch.zeros(512, device="cuda", dtype=torch.uint8))
    t = torch.zeros(3, 2, device="cuda")
    with pytest.raises(fs.FsError, match="both or neither"):
        fs.fs_distill_loss(x[0], i[0], t, st[0].clone(), st[1].clone(), d_loss=v[:3].clone())
    with pytest.raises(fs.FsError, match="temperature"):
        fs.fs_distill_loss(x[0], i[0], t, st[0].clone(), st[1].clone(), temperature=0.0)
    with pytest.raises(TypeError, match="active"):
        fs.fs_distill_loss(x[0], i[0], t, st[0].clone(), st[1].clone(), active=t)
    with pytest.raises(TypeError, match="int32"):
        fs.fs_distill_loss(x[0], i[0].long(), t, st[0].clone(), st[1].clone())
    with pytest.raises(ValueError, match="ids must be"):
        fs.fs_balance_loss(x, i[0], st, st, st, st)
    with pytest.raises(ValueError, match="counts"):
        fs.fs_balance_loss(x, i, i.float(), i[:, 0].contiguous(), st, st)
    with pytest.raises(fs.FsError, match="k must be"):
        bad = torch.zeros(2, 3, 33, device="cuda", dtype=I4)
        fs.fs_balance_loss(x, bad, bad.float(), torch.zeros(2, 64, device="cuda", dtype=I4),
                           torch.zeros(2, 2, device="cuda"), st)
