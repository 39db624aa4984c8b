"""The comparisons of tests/strict.py reject NaN, and what else is wrong (CPU)."""
import math

import pytest

torch = pytest.importorskip("torch")
from tests.strict import assert_attention, assert_within


def test_within():
    x = torch.tensor([1.0, -math.inf, 0.0])
    assert_within(x, x, 0.0)
    assert_within(x + torch.tensor([0.5, 0.0, -0.5]), x, 0.5)
    for i, bad in ((0, math.nan), (0, 1.6), (1, math.nan), (1, 0.0), (1, math.inf), (2, math.inf)):
        y = x.clone()
        y[i] = bad
        with pytest.raises(AssertionError):
            assert_within(y, x, 0.5)


@pytest.mark.parametrize("what", ["right", "nan out", "nan lse", "all nan out", "empty row not zero", "empty row lse"])
def test_attention(what):
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(n, 128, generator=g).double() for n in (3, 5, 5))
    seen = torch.ones(3, 5, dtype=torch.bool)
    seen[2] = False                                        # a row that sees nothing
    s = q @ k.T / math.sqrt(128)
    out = torch.softmax(s, 1) @ v
    lse = torch.logsumexp(s, 1)
    out[2], lse[2] = 0.0, -math.inf
    if what == "nan out":
        out[1, 5] = math.nan
    elif what == "nan lse":
        lse[0] = math.nan
    elif what == "all nan out":
        out[:] = math.nan
    elif what == "empty row not zero":
        out[2, 0] = math.nan
    elif what == "empty row lse":
        lse[2] = math.nan
    if what == "right":
        assert_attention(out, lse, q, k, v, seen, 1 / math.sqrt(128))
    else:
        with pytest.raises(AssertionError):
            assert_attention(out, lse, q, k, v, seen, 1 / math.sqrt(128))
