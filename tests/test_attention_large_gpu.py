"""Attention and norm + rotation at row counts whose launches pass 2^32 threads in one
dimension if laid out flat."""
import pytest
import torch

from attention_reference import check, norm_reference, reference
from test_attention_gpu import BF

pytestmark = pytest.mark.gpu


def test_single_rows_of_many_sequences(fs):
    """One query row for each of 65536 x 32 heads: the backward pass pads its row
    terms to whole tiles, 2^28 in all."""
    B, H, m, d = 1 << 16, 32, 2, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    q, d_o = (torch.randn(B, 1, H, d, generator=g, device="cuda").to(BF) for _ in range(2))
    k, v = (torch.randn(B, m, H, d, generator=g, device="cuda").to(BF) for _ in range(2))
    o, dq, dk, dv = (torch.full_like(t, float("nan")) for t in (q, q, k, v))
    lse = torch.full((B, H, 1), float("nan"), device="cuda")
    fs.fs_attention_forward(q, k, v, o, lse)
    fs.fs_attention_backward(q, k, v, o, lse, d_o, dq, dk, dv)
    torch.cuda.synchronize()
    for t in (o, lse, dq, dk, dv):
        assert torch.isfinite(t).all()
    # every row of o against the definition: the weights and the result are rounded
    # to bf16 (2^-8 each of values up to max |v|), the rest is fp32
    s = (q.float() * k.float()).sum(-1) * d ** -0.5
    want = (torch.softmax(s, 1)[..., None] * v.float()).sum(1, keepdim=True)
    assert torch.all((o.float() - want).abs() <= 2.5 * 2.0 ** -8 * v.float().abs().amax(1, keepdim=True))
    at = torch.tensor([0, 1, 4095, 32767, 32768, 65534, 65535], device="cuda")
    pick = lambda t: t[at].cpu()
    ref = reference(*(pick(t) for t in (q, k, v)), d_o=pick(d_o))
    for x, t in (("o", o), ("lse", lse), ("d_q", dq), ("d_k", dk), ("d_v", dv)):
        check(x, pick(t), ref[x])


def test_norm_of_many_tokens(fs):
    """2^26 tokens of one head, the most that a call takes."""
    n, d = 1 << 26, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(1, n, 1, d, generator=g, device="cuda").to(BF)
    y = torch.full_like(x, float("nan"))
    w = torch.rand(d, generator=g, device="cuda") + 0.5
    fs.fs_qk_norm_rotate(x, None, w, None, y, None, eps=1e-5)
    torch.cuda.synchronize()
    for lo in range(0, n, n // 8):
        part = x[:, lo:lo + n // 8].float()
        want = part * torch.rsqrt((part * part).mean(-1, keepdim=True) + 1e-5) * w
        # one rounding to bf16, fp32 before it
        assert torch.all((y[:, lo:lo + n // 8].float() - want).abs() <= want.abs() * 1.01 * 2.0 ** -8)
    ends = torch.cat((x[:, :3], x[:, -3:]), 1).cpu()
    ref = norm_reference(ends, w.cpu(), None, None, None, 1e-5, False)
    check("y", torch.cat((y[:, :3], y[:, -3:]), 1), ref["y"])
