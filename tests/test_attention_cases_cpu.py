"""The attention's cases reach every form of its kernels, and the bias gradient's bound
tells a row sum from a rounded output."""
import pytest
import torch

from attention_cases import (BF, F4, FORMS, HF, LONG, LONG_ROWS, SPLIT, all_forms, bias_gradient,
                             case_forms, case_id, case_inputs, coherent)
from attention_reference import reference


def test_every_form_has_a_case():
    got = set()
    for case in FORMS + SPLIT + LONG + LONG_ROWS:
        got |= case_forms(case)
    missing = all_forms() - got
    assert not missing, sorted(missing, key=str)
    # every backward form of a mask ring is one of the cases that run backward
    back = set()
    for case in FORMS + SPLIT + LONG:
        back |= case_forms(case)
    assert all(x in back for x in all_forms() if x[0].startswith(("q ", "kv ")) or
               x[0] == "refill" and x[1].startswith("q "))


def test_cases_have_the_shapes_that_the_rules_see():
    for case in FORMS + SPLIT:
        q, k, v, d_o, d_lse, kw = case_inputs(case)
        assert q.shape[2] == case[4] and k.shape[2] == case[5] and v.shape[3] == case[7]
        assert d_o.shape == q.shape[:3] + v.shape[3:] and d_lse.shape == (case[1], case[4], case[2])


@pytest.mark.parametrize("case", [c for c in FORMS if c[9]["buckets"] and c[8] == 1], ids=case_id)
def test_bias_gradient_is_the_references(case):
    q, k, v, d_o, d_lse, kw = case_inputs(case)
    val, bound = bias_gradient(q, k, v, d_o, d_lse, **kw)
    want, wide = reference(q, k, v, d_o=d_o, d_lse=d_lse, **kw)["d_bias"]
    assert torch.allclose(val, want, rtol=1e-10, atol=1e-12)
    if q.dtype != F4:
        assert torch.all(bound <= wide)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n", [3, 140])
def test_the_bound_tells_a_rounded_row_sum(dtype, n):
    """The gradient with its row sums taken from the rounded o is out of bounds."""
    q, k, v, d_o, d_lse, kw = coherent(dtype, n)
    val, bound = bias_gradient(q, k, v, d_o, d_lse, **kw)
    wrong, _ = bias_gradient(q, k, v, d_o, d_lse, stored_o=True, **kw)
    assert float(((wrong - val).abs() / bound).max()) > 2
