"""Chunks behind a request's last token, in contiguous caches whose slots there hold NaN:
they weigh nothing, however their CTA's copies fall."""
import math

import pytest

torch = pytest.importorskip("torch")
from tests import cache_ref as R
from tests.strict import assert_attention
from tests.test_gpu_cache_ops import D, Paged, bf16, gen, status_word

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(D)


@pytest.fixture(scope="module")
def da():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from split_kv_decode_attention_gb300 import binding as B
    from split_kv_decode_attention_gb300 import build as cuda_build
    cuda_build.build()
    B.lib()
    return B


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("op", ["decode", "cross"])
@pytest.mark.parametrize("batch,T,splits", [(33, 4, 2), (33, 1, 2), (3, 2, 8), (5, 3, 16), (33, 4, 0), (20, 16, 2)])
def test_empty_chunks_of_a_poisoned_cache(da, kind, op, batch, T, splits):
    lens = [[1, 257, 129, 33, 500][b % 5] for b in range(batch)]
    lens[-1] = 1030
    heads = 4 if T == 16 else 8
    c = Paged(kind, lens, heads, 0, 30).gpu()
    for b, n in enumerate(lens):
        if kind == "fp4":
            c.dk_sf[b, :, n:] = 0x7f
            c.dv_sf[b, :, n:] = 0x7f
        else:
            for x in (c.dk, c.dv):
                x[b, n:] = 0x7f if kind == "fp8" else float("nan")
    q = bf16(gen(31), batch, T, heads, D, std=2.0)
    dq, status = q.cuda(), status_word()
    runs = []
    for _ in range(12):
        if op == "decode":
            runs.append(da.decode_attn(dq, c.dk, c.dv, None, c.dlens, max_seq_len=c.max_len, num_splits=splits, status=status,
                                       **(c.scales() if kind != "bf16" else {})))
        else:
            runs.append(da.cross_attn(dq, c.dk, c.dv, None, c.dlens, max_seq_len=c.max_len, num_splits=splits, status=status,
                                      **c.scales()))
    assert int(status) == 0
    out, lse = runs[0]
    for o, l in runs:
        assert bool(o.isfinite().all()) and bool(l.isfinite().all())
        assert torch.equal(o, out) and torch.equal(l, lse)
    out, lse = out.double().cpu(), lse.double().cpu()
    kv, vv = (c.values(w) * s for w, s in (("k", c.ks), ("v", c.vs)))
    tol = R.bf16_p_tolerance if kind == "bf16" else R.out_tolerance
    for b in (0, 1, 2, batch - 1):
        n = lens[b]
        for h in (0, heads - 1):
            assert_attention(out[b, :, h], lse[b, :, h], q[b, :, h].double(), kv[b, :n, h], vv[b, :n, h],
                             torch.ones(T, n, dtype=torch.bool), SCALE, tol, (b, h))
