"""Every form of the attention's kernels, at each width of tile and type, with and
without a bias, against the definition in 64 bits (attention_cases.py says which
case reaches which form)."""
import pytest
import torch

from attention_cases import (BF, F4, FORMS, HF, LONG, LONG_ROWS, SPLIT, bias_gradient, case_id,
                             case_inputs, coherent)
from attention_reference import check, reference
from test_attention_edges_gpu import compare, run
from test_attention_gpu import fused, heads_first, unaligned

pytestmark = pytest.mark.gpu

LAYOUTS = {"plain": None, "heads_first": heads_first, "fused": fused, "unaligned": unaligned}


def full(fs, case, view=None, seed=0):
    q, k, v, d_o, d_lse, kw = case_inputs(case, seed)
    print(case_id(case), flush=True)
    out = run(fs, q, k, v, d_o, d_lse, case[8], view, **kw)
    compare(out, reference(q, k, v, d_o=d_o, d_lse=d_lse, **kw))
    if kw.get("bias") is not None:
        print("d_bias", check("d_bias", out["d_bias"], bias_gradient(q, k, v, d_o, d_lse, **kw)))


@pytest.mark.parametrize("case", FORMS, ids=case_id)
def test_forms(fs, case):
    full(fs, case)


@pytest.mark.parametrize("case", SPLIT, ids=case_id)
@pytest.mark.parametrize("layout", LAYOUTS)
def test_split_keys_and_queries(fs, case, layout):
    """Ranges of keys and of queries, joined into outputs of any strides."""
    full(fs, case, LAYOUTS[layout], seed=1)


@pytest.mark.parametrize("layout", ["heads_first", "fused", "unaligned"])
@pytest.mark.parametrize("case", [c for c in FORMS if c[9]["buckets"]][::2], ids=case_id)
def test_layouts_with_a_bias(fs, case, layout):
    full(fs, case, LAYOUTS[layout], seed=2)


@pytest.mark.parametrize("case", LONG, ids=case_id)
def test_masks_of_many_words(fs, case):
    full(fs, case)


@pytest.mark.parametrize("case", LONG_ROWS, ids=case_id)
def test_masks_of_many_words_few_rows(fs, case):
    """Half a million keys and more: a wave of the few-row form takes over 64 tiles."""
    q, k, v, _, _, kw = case_inputs(case)
    print(case_id(case), flush=True)
    compare(run(fs, q, k, v, **kw), reference(q, k, v, **kw))


@pytest.mark.parametrize("copies", [1, 16, 64])
@pytest.mark.parametrize("n", [3, 140])
@pytest.mark.parametrize("dtype", [BF, HF, F4])
def test_bias_gradient_with_fp32_row_sums(fs, dtype, n, copies):
    """Inputs whose rounded o would show in the bias's gradient."""
    q, k, v, d_o, d_lse, kw = coherent(dtype, n)
    out = run(fs, q, k, v, d_o, d_lse, copies, **kw)
    print(check("d_bias", out["d_bias"], bias_gradient(q, k, v, d_o, d_lse, **kw)))
