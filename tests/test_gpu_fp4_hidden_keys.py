"""NaN block scales of a 4-bit cache in keys that the mask hides, and in slots behind the
sequence, in trees of every form of the kernels."""
import math

import pytest

torch = pytest.importorskip("torch")
from tests import cache_ref as R
from tests.strict import assert_attention
from tests.test_gpu_cache_ops import D, Paged, bf16, gen, status_word
from tests.test_gpu_tree_ops import SCALE, da, ints, pack, tolerance_for  # noqa: F401

pytestmark = pytest.mark.gpu
NAN = 0x7f


@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("lens", [[300, 133], [2100, 1500]])
@pytest.mark.parametrize("G,T", [(4, 4), (2, 15), (4, 16), (4, 32), (4, 40), (4, 100)])
def test_nan_block_scales_of_hidden_keys(da, G, T, lens, splits):  # noqa: F811
    """Token 2's key is NaN and is seen by token 2 alone; rows of 16 to 400 per KV head, in calls that are cut into groups of
    16 rows and in those that are not, converted in the kernel and copied first."""
    lens, own = lens + [T], [T, T - 1, T - 1]
    c = Paged("fp4", lens, 2, 16, 40 + T).gpu()
    q = bf16(gen(T), 3, T, 2 * G, D, std=2.0)
    seen = torch.zeros(T, T, dtype=torch.bool)
    seen[:, 0] = seen[:, 1] = True
    seen[2, 2] = True
    for b in range(3):
        j = lens[b] - own[b] + 2
        c.dk_sf[int(c.bt[b, j // 16]), :, j % 16] = NAN
        for j in range(lens[b], -(-lens[b] // 16) * 16):
            for x in (c.dk_sf, c.dv_sf):
                x[int(c.bt[b, j // 16]), :, j % 16] = NAN
    q[1, own[1]:] = math.nan
    q[2, own[2]:] = math.inf
    status = status_word()
    out, lse = da.decode_attn_tree(q.cuda(), c.dk, c.dv, c.dbt, c.dlens, pack(seen)[None].cuda(), max_seq_len=c.max_len, num_splits=splits,
                                   new_lens=ints(own), status=status, **c.scales())
    assert int(status) == 0
    kv, vv = (c.values(w) * s for w, s in (("k", c.ks), ("v", c.vs)))
    keep = [t for t in range(T) if t != 2]
    for b, n in enumerate(lens):
        m = own[b]
        assert bool(out[b, 2].isnan().all()) and bool(lse[b, 2].isnan().all())
        assert bool((out[b, m:] == 0).all()) and bool((lse[b, m:] == -math.inf).all())
        rows = [t for t in keep if t < m]
        k, v = R.gather(kv, c.bt, b, n), R.gather(vv, c.bt, b, n)
        see = torch.ones(len(rows), n, dtype=torch.bool)
        see[:, n - m:] = seen[rows][:, :m]
        for h in range(2):
            at = slice(h * G, (h + 1) * G)
            assert_attention(out[b, rows, at].double().cpu().reshape(-1, D), lse[b, rows, at].double().cpu().reshape(-1),
                             q[b, rows, at].double().reshape(-1, D), k[:, h], v[:, h], see.repeat_interleave(G, 0), SCALE,
                             tolerance_for("fp4", G, T), (b, h))
