"""assert_values lets numbers in the tolerance pass, and nothing else."""
import numpy as np
import pytest

from _close import assert_values

REF = np.array([[1.0, -2.0, 0.0]])


def test_numbers_within_the_tolerance_pass():
    assert_values(REF * (1 + 2.0 ** -12), REF, "f16", 0.0)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 1.01])
@pytest.mark.parametrize("at", [0, 2])
def test_what_is_no_number_or_is_off_fails(bad, at):
    got = REF.copy()
    got[0, at] = bad
    with pytest.raises(AssertionError):
        assert_values(got, REF, "bf16", 2.0 ** -10)


def test_all_nan_fails():
    with pytest.raises(AssertionError):
        assert_values(np.full_like(REF, np.nan), REF, "f32", 1.0, extra=10.0)
