"""The check of the experts' precision (a16_norm.py) on the CPU: it takes what the kernels are to compute
and rejects the same with fewer bits anywhere."""
import pytest

import a16_norm as norm


@pytest.mark.parametrize("case", norm.CASES, ids=str)
def test_fewer_bits_are_rejected(case):
    args = norm.make(case)
    want = norm.experts(*args)
    norm.check_norm(norm.rounded(norm.experts(*args, how="kernel")), want, "two terms")
    for how in norm.MUTANTS:
        with pytest.raises(AssertionError):
            norm.check_norm(norm.rounded(norm.experts(*args, how=how)), want, how)


@pytest.mark.parametrize("b", [4, 8, 24])
def test_one_term_changes_h(b):
    args = norm.make_low_rank(b)
    want = norm.experts(*args)
    assert norm.changed(norm.rounded(norm.experts(*args, how="kernel")), want) <= 0.05
    assert norm.changed(norm.rounded(norm.experts(*args, how="one term")), want) > 0.1
