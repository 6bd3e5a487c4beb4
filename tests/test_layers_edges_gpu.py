"""The operators of include/fs_layers.h at their edges: calls that the documentation
allows and few make, and the refusals of calls that it does not."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, HF, F4 = torch.bfloat16, torch.float16, torch.float32
I4, I1 = torch.int32, torch.int8


@pytest.mark.parametrize("dtype", [BF, HF, F4], ids=["bf16", "fp16", "fp32"])
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
