"""More than 128 query rows per KV head over bf16 caches: large values, and rows whose
scores rise from one step of 128 keys to the next, against plain 64-bit references."""
import math

import pytest

torch = pytest.importorskip("torch")
from tests import cache_ref as R
from tests.strict import assert_within
from tests.test_gpu_cache_ops import D, bf16, gen
from tests.test_gpu_tree_ops import da, ints  # noqa: F401

pytestmark = pytest.mark.gpu
LN2 = math.log(2.0)  # (as a scale: q . k are the scores in log2 units)


def rising(T, L, at, v, q0, k0, k1=None):
    """Row t's score of key j is q0[t] * k0[j] (+ k1[j]) in log2 units, the value v[j]."""
    q = torch.zeros(1, T, 1, D, dtype=torch.bfloat16)
    k = torch.zeros(1, L, 1, D, dtype=torch.bfloat16)
    q[0, :, 0, at] = q0.to(torch.bfloat16)
    k[0, :, 0, at] = k0.to(torch.bfloat16)
    if k1 is not None:
        q[0, :, 0, at + 1] = 1.0
        k[0, :, 0, at + 1] = k1.to(torch.bfloat16)
    return q, k, v.to(torch.bfloat16).view(1, L, 1, D)


def call(da, q, k, v, splits):  # noqa: F811
    L = k.shape[1]
    return da.cross_attn(q.cuda(), k.cuda(), v.cuda(), None, ints([L]), max_seq_len=L, scale=LN2, num_splits=splits)


def reference(q, k, v):
    rows, kk, vv = q[0, :, 0].double(), k[0, :, 0].double(), v[0, :, 0].double()
    return (*R.attention_rows(rows, kk, vv, torch.ones(rows.shape[0], kk.shape[0], dtype=torch.bool), LN2), vv)


@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("size", [2.0 ** 70, 1e30])
@pytest.mark.parametrize("rise", [7, 9, 40, 60, 64])
def test_large_values_behind_rising_scores(da, rise, size, splits):  # noqa: F811
    """The later a key, the more it weighs, and its value stays finite in the product: a row's weights are kept within
    2^8 of its largest score so far.  (384 keys: 384 x 2^8 x 4e30 is 2^119.)"""
    T, L = 200, 384
    k0 = torch.zeros(L)
    k0[200], k0[300] = rise, 2 * rise
    v = bf16(gen(rise), L, D).float().clamp(-4, 4) * size
    q, k, v = rising(T, L, 5, v, torch.linspace(0.1, 1.0, T), k0)
    out, lse = call(da, q, k, v, splits)
    o, l, wabs, mag, _ = reference(q, k, v)
    assert_within(out[0, :, 0].cpu(), o, R.bf16_p_tolerance(o, wabs, mag))
    assert_within(lse[0, :, 0].cpu(), l, R.lse_tolerance(l, mag))


def rounded_weights_tolerance(o, w_off, mag):
    """Where the sum that divides O is that of the weights as rounded to bf16 (2^-8 of each), those applied sum to one:
    sum_j w_j (1 + d_j) v_j / sum_j w_j (1 + d_j) - o = sum_j w_j d_j (v_j - o) / (1 + sum_j w_j d_j), so the weights'
    roundings and the errors of the scores (as in cache_ref) count only by w_off = sum_j w_j |v_j - o|.  On top come the
    output's own rounding, 2^-8, and 2^-18 for the sums in fp32."""
    rel = 2.0 ** -8 / (1 - 2.0 ** -8) + 2 * 2.0 ** -16 * mag + 2.0 ** -18
    return (2.0 ** -8 + 2.0 ** -18) * o.abs() + rel[:, None] * w_off


@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("first", [0, 200])
@pytest.mark.parametrize("most", [8, 60])
def test_rows_that_one_key_dominates(da, most, first, splits):  # noqa: F811
    """One key's score is 0.3 to 60 (log2) above another's of an earlier step, and all others are far below: the output
    is off by its own rounding and by what the two keys' weights leave open, not by the rounding of the larger weight."""
    T, L = 256, 512
    k0, k1 = torch.zeros(L), torch.full((L,), -40.0)
    k1[first + 3] = k1[first + 150] = 0.0
    k0[first + 150] = 1.0
    rise = torch.linspace(0.3, most, T)
    v = bf16(gen(most), L, D).float() * 8
    q, k, v = rising(T, L, 5, v, rise, k0, k1)
    out, lse = call(da, q, k, v, splits)
    o, l, _, mag, vv = reference(q, k, v)
    s = (q[0, :, 0].double() @ k[0, :, 0].double().T) * LN2
    w = torch.exp(s - l[:, None])
    w_off = torch.stack([(w[t, :, None] * (vv - o[t]).abs()).sum(0) for t in range(T)])
    assert_within(out[0, :, 0].cpu(), o, rounded_weights_tolerance(o, w_off, mag))
    assert_within(lse[0, :, 0].cpu(), l, R.lse_tolerance(l, mag))
