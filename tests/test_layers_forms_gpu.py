"""Every form of the kernels of include/fs_layers.h (shapes by width, rows that are
whole 16-byte chunks or not, types, ranges) on a few rows, against the
definitions in 64 bits."""
import pytest
import torch

from layers_reference import (balance_reference, distill_reference, norm_reference,
                              quantize_reference)
from test_layers_gpu import (BF, F4, HF, I4, balance_run, compare, distill_run, gen, norm_run,
                             product_check, product_inputs, product_run, quant_inputs, quant_run,
                             randn)

pytestmark = pytest.mark.gpu

TYPES = [BF, HF, F4]
IDS = ["bf16", "fp16", "fp32"]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("rows", [1, 70])
def test_layer_norm_forms(fs, dtype, rows):
    for width in (8, 63, 64, 65, 128, 129, 250, 256, 512, 515, 1024, 1031, 2048, 2051, 4096, 4100, 8192,
                  8200, 16376, 16384):
        if rows > 1 and width > 5000:
            continue
        g = gen(width)
        x, r, d_y, d_z = (randn(g, 1, rows, width, dtype=dtype) for _ in range(4))
        w, b = 1 + randn(g, width, std=0.2), randn(g, width, std=0.2)
        kw = {"eps": 1e-5, "residual": r, "d_total": d_z}
        print(dtype, rows, width, flush=True)
        compare(norm_run(fs, x, w, b, d_y=d_y, **kw), norm_reference(x, w, b, d_y=d_y, **kw))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_quantize_forms(fs, dtype):
    for width in (1, 16, 127, 128, 129, 512, 513, 2048, 2049, 8192, 8193, 65535, 65536):
        x = quant_inputs(dtype, 3, width)
        print(dtype, width, flush=True)
        q, s = quant_run(fs, x)
        rq, rs = quantize_reference(x)
        assert torch.equal(q, rq) and torch.equal(s, rs)


# m, n, k: few rows (one and two blocks of 16, from dwords on and not), tiles of 64
# (ranges of k), 128 (four and two buffers) and 256, laid out first and not
PRODUCTS = [(16, 40, 64), (16, 40, 1000), (5, 40, 1001), (32, 70, 2048), (20, 70, 2047),
            (8, 48, 4096), (8, 8200, 640), (16, 8193, 1003), (32, 8195, 700), (20, 8192, 129), (33, 64, 128), (64, 64, 4096), (40, 80, 8193), (1700, 1800, 256),
            (1700, 1801, 250), (2100, 2200, 144), (3500, 3600, 272), (3500, 3601, 257),
            (70, 90, 16), (70, 90, 1)]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", PRODUCTS, ids=str)
def test_product_forms(fs, dtype, case):
    print(dtype, case, flush=True)
    args = product_inputs((dtype,) + case + (True,))
    product_check(product_run(fs, dtype, *args), dtype, *args)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("rows", [1, 130])
def test_distill_forms(fs, dtype, rows):
    """With 130 rows one workgroup a row whatever its length, with one row ranges of it
    from 32769 classes on."""
    for classes in (8, 511, 512, 520, 2048, 2049, 4096, 4104, 8192, 8193, 16384, 16392, 32768, 32776,
                    40001, 65536, 65544, 70001, 131072, 131080, 300000):
        if rows > 1 and (classes < 30000 or classes > 80000):
            continue
        g = gen(classes)
        x = randn(g, rows, classes, dtype=dtype, std=2.0)
        ids = torch.randint(0, classes, (rows, 5), generator=g, dtype=I4)
        t, dl = randn(g, rows, 5), 0.5 + torch.rand(rows, generator=g)
        # the last class, and one twice
        ids[0, 0], ids[0, 1], ids[0, 2] = classes - 1, 3, 3
        print(dtype, rows, classes, flush=True)
        ref = distill_reference(x, ids, t, 1.5, d_loss=dl)
        for out in distill_run(fs, x, ids, t, 1.5, dl):
            compare(out, ref)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_distill_many_rows(fs, dtype):
    """From 512 rows on, rows of 8193 to 10240 classes (to 16384 for the loss alone) are
    kept in part."""
    for classes in (8200, 8201, 10241, 16384):
        g = gen(classes)
        x = randn(g, 512, classes, dtype=dtype, std=2.0)
        ids = torch.randint(0, classes, (512, 3), generator=g, dtype=I4)
        ids[0, 0] = classes - 1
        t, dl = randn(g, 512, 3), 0.5 + torch.rand(512, generator=g)
        print(dtype, classes, flush=True)
        keep = torch.arange(0, 512, 37)
        outs = distill_run(fs, x, ids, t, 1.5, dl)
        ref = distill_reference(x[keep], ids[keep], t[keep], 1.5, d_loss=dl[keep])
        for out in outs:
            compare({k: v[keep.cuda()] for k, v in out.items()}, ref)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("normalize", [False, True])
def test_balance_forms(fs, dtype, normalize):
    for n in (3, 300):  # one workgroup, several
        for E in (7, 8, 15, 16, 31, 32, 60, 64, 100, 128, 250, 256, 511, 512, 1000, 1024):
            for k in {1, min(E, 8), min(E, 9), min(E, 32)}:
                if n > 3 and k not in (1, 8, 32):
                    continue
                g = gen(E + k)
                x = randn(g, 2, n, E, dtype=dtype)
                dl, dg = torch.rand(2, 2, generator=g) * 30, randn(g, 2, n, k, std=0.1)
                print(dtype, n, E, k, flush=True)
                compare(balance_run(fs, x, k, dl, dg, normalize=normalize),
                        balance_reference(x, k, normalize, d_loss=dl, d_gates=dg))
