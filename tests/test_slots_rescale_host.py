"""The cases of a moving reference tell a right walk over the pages from wrong ones (on the CPU)."""
import numpy as np
import pytest

import slots_rescale_testlib as cases


@pytest.mark.parametrize("name", cases.HEIGHTS)
@pytest.mark.parametrize("repeat", [1, 3])
def test_a_right_walk_passes_and_wrong_ones_do_not(name, repeat):
    H, heights = 24, cases.HEIGHTS[name]
    q, kv = cases.case(1, heights, H, repeat)
    n = 64 * len(kv) - 9
    table = np.arange(len(kv))
    out, lse, weights, tol_out, tol_lse, tol_w = cases.expected(q, kv, table, n, len(kv))
    assert (tol_out <= 0.01 * np.abs(out)).all()       # a row of zeros is wrong in every value
    assert (tol_lse <= 2e-3).all() and (tol_w <= 2e-3 * weights).all()
    got = cases.walk(q, kv, table, n)
    assert (np.abs(got[0] - out) <= tol_out).all() and (np.abs(got[1] - lse) <= tol_lse).all()
    rising = np.arange(H) % 7 != 6
    for mistake in ("rows left", "half the dims left", "the next head's factor", "rows dropped"):
        wrong = (np.abs(cases.walk(q, kv, table, n, mistake)[0] - out) > tol_out).any(1)
        assert wrong[rising].all(), mistake
    if name in ("one step", "a step a page"):  # (later slots outweigh what is left in the sum elsewhere)
        wrong = np.abs(cases.walk(q, kv, table, n, "sum left")[1] - lse) > tol_lse
        assert wrong[rising].all()
