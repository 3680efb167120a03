"""The comparison that smoke() makes (no GPU): a NaN anywhere fails it, whichever result it is in."""
import numpy as np
import pytest

import __graft_entry__ as entry


def test_worst_is_the_largest_error():
    want = {"a": np.array([3.0, 4.0]), "b": np.array([1.0])}
    got = {"a": np.array([3.0, 4.5]), "b": np.array([1.2])}
    assert entry.worst_rel_err(got, want) == pytest.approx(0.2)
    assert entry.worst_rel_err(want, want) == 0.0


@pytest.mark.parametrize("bad", ["a", "b", "c"])
def test_a_nan_in_any_result_fails_the_bar(bad):
    want = {k: np.ones(4) for k in "abc"}
    got = {k: v.copy() for k, v in want.items()}
    got[bad][2] = np.nan
    assert not entry.worst_rel_err(got, want) <= 1e-5
