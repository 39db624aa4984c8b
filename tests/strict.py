"""Comparisons that NaN fails: every entry has to be within its tolerance, where
"no entry is outside it" would let NaN pass."""
import math

import torch

from tests import cache_ref as R


def assert_within(got, want, tolerance, what=""):
    """|got - want| <= tolerance, entry by entry; where `want` is infinite, equal to it."""
    got, want = got.double(), want.double()
    same = got == want                                     # (infinities)
    ok = same | ((got - want).abs() <= torch.as_tensor(tolerance).double())
    assert bool(ok.all()), (what, int((~ok).sum()), float(torch.where(ok, 0.0, (got - want).abs()).max()))


def assert_attention(got, got_lse, rows, k, v, seen, scale, tolerance=R.out_tolerance, what=""):
    """One KV head's rows [R, 128] over keys k, v [n, 128] (64 bits) as `seen` [R, n] lets
    them: outputs and LSEs within their tolerances, rows that see nothing 0 and -inf."""
    o, l, wabs, mag = R.attention_rows(rows, k, v, seen, scale)
    some = ~l.isinf()
    tol = torch.where(some[:, None], tolerance(o, wabs, mag), 0.0)
    assert_within(got, torch.where(some[:, None], o, 0.0), tol, (what, "out"))
    lse_tol = torch.where(some, R.lse_tolerance(l, mag), 0.0)
    assert_within(got_lse, l, lse_tol, (what, "lse"))
    assert not bool((l == math.inf).any())
