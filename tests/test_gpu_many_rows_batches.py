"""More than 128 query rows per KV head in large ragged batches: a few long requests among
many short ones, and lengths that are out of range among them."""
import random

import pytest

torch = pytest.importorskip("torch")
from tests.test_gpu_cache_ops import D, Paged, bf16, gen, status_word
from tests.test_gpu_tree_ops import check_rows, cross_call, da, ints  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("B,heads,at", [(300, 2, [0, 1, 150, 299]), (257, 1, [128]), (40, 3, [39]), (33, 1, [])])
def test_few_long_requests_among_many(da, kind, B, heads, at):  # noqa: F811
    """Requests of one token or none, with keys or without, around those at `at`, one of which has no keys: the walk
    over the pairs of row tiles passes over all others."""
    r = random.Random(B)
    T, G = 330, 2
    lens = [r.choice([0, 1, 40, 129, 300]) for _ in range(B)]
    own = [r.choice([0, 1, 1, 2]) for _ in range(B)]
    for i, b in enumerate(at):
        own[b] = T - i
        lens[b] = 300 if i != 1 else 0
    lens[-1] = 300
    c = Paged(kind, lens, heads, 16, 500 + B).gpu()
    q = bf16(gen(B), B, T, heads * G, D, std=2.0)
    status = status_word()
    out, lse = cross_call(da, c, q.cuda(), q_lens=ints(own), num_splits=1, status=status)
    check_rows(c, q, out, lse, own, None)
    assert int(status) == 0
    # rows that are out of range count as T, or as none
    bad = list(own)
    bad[3], bad[7] = T + 5, -4
    own[3], own[7] = T, 0
    out, lse = cross_call(da, c, q.cuda(), q_lens=ints(bad), num_splits=1, status=status)
    check_rows(c, q, out, lse, own, None)
    assert int(status) == 2
