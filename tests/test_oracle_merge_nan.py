"""The oracle's merge of partials keeps NaN: a row whose LSEs are NaN is not one
without keys (CPU)."""
import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("bad", [[0], [1], [2], [0, 1], [0, 1, 2]])
@pytest.mark.parametrize("others", [0.5, -np.inf])
def test_nan_lse(bad, others):
    po = np.ones((2, 3, 4))
    pl = np.full((2, 3), others)
    pl[0, bad] = np.nan
    out, lse = oracle.merge_partials(po, pl)
    assert np.isnan(out[0]).all() and np.isnan(lse[0])
    if others == -np.inf:
        assert not out[1].any() and lse[1] == -np.inf
    else:
        assert np.allclose(out[1], 1.0, rtol=1e-15) and np.isclose(lse[1], 0.5 + np.log(3), rtol=1e-15)


def test_nan_behind_the_valid_partials_is_not_read():
    po, pl = np.ones((1, 3, 4)), np.zeros((1, 3))
    pl[0, 2] = po[0, 2] = np.nan
    out, lse = oracle.merge_partials(po, pl, nvalid=np.array([2]))
    assert np.allclose(out, 1.0, rtol=1e-15) and np.isclose(lse[0], np.log(2), rtol=1e-15)
