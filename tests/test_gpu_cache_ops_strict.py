"""Attention over 4-bit caches and over selected pages into outputs that hold NaN
before the call: every entry has to be written, and within its tolerance."""
import math

import pytest

torch = pytest.importorskip("torch")
from tests import cache_ref as R
from tests.strict import assert_attention
from tests.test_gpu_cache_ops import FP4_CASES, Paged, bf16, gen, longer

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def da():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from split_kv_decode_attention_gb300 import binding as B
    from split_kv_decode_attention_gb300 import build as cuda_build
    cuda_build.build()
    B.lib()
    return B


def nan_outputs(q):
    return dict(out=torch.full(q.shape, math.nan, dtype=torch.bfloat16, device="cuda"),
                lse=torch.full(q.shape[:3], math.nan, device="cuda"))


def tolerance(kind):
    return R.bf16_p_tolerance if kind == "bf16" else R.out_tolerance


def check_dense(pc, q, out, lse, causal):
    B, T, Hq, _ = q.shape
    G = Hq // pc.heads
    out, lse = out.cpu().double(), lse.cpu().double()
    k64, v64 = pc.values("k") * pc.ks, pc.values("v") * pc.vs
    for b, n in enumerate(pc.lens):
        kb, vb = R.gather(k64, pc.bt, b, n), R.gather(v64, pc.bt, b, n)
        last = torch.tensor([n - T + 1 + t if causal else n for t in range(T) for _ in range(G)])
        seen = torch.arange(n)[None, :] < last[:, None]
        for h in range(pc.heads):
            at = slice(h * G, (h + 1) * G)
            assert_attention(out[b, :, at].reshape(T * G, D), lse[b, :, at].reshape(T * G),
                             q[b, :, at].double().reshape(T * G, D), kb[:, h], vb[:, h], seen, 1 / math.sqrt(D),
                             tolerance(pc.kind), (b, h))


def check_selected(pc, q, out, lse, blocks, causal):
    """Against the pages that `blocks` names."""
    B, T, Hq, _ = q.shape
    G = Hq // pc.heads
    out, lse, blocks = out.cpu().double(), lse.cpu().double(), blocks.cpu()
    k64, v64 = pc.values("k") * pc.ks, pc.values("v") * pc.vs
    for b, n in enumerate(pc.lens):
        for t in range(T):
            seen = max(0, n - T + 1 + t) if causal else n
            for h in range(pc.heads):
                at = blocks[b, t, h]
                at = at[at >= 0].long()
                m = len(at) * pc.page - (-(-seen // pc.page) * pc.page - seen)
                kk, vv = (x[pc.bt[b].long()[at]][:, :, h].flatten(0, 1)[:m] for x in (k64, v64))
                rows = slice(h * G, (h + 1) * G)
                assert_attention(out[b, t, rows], lse[b, t, rows], q[b, t, rows].double(), kk, vv,
                                 torch.ones(G, m, dtype=torch.bool), 1 / math.sqrt(D), tolerance(pc.kind), (b, t, h))


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("case", FP4_CASES, ids=lambda c: "g%d_t%d_%s_p%d" % (c[0], c[1], "causal" if c[2] else "full", c[3]))
def test_fp4(da, case, splits):
    G, T, causal, page, lens = case
    pc = Paged("fp4", lens, 2, page, 470 + G + T, std=1.5).gpu()
    q = bf16(gen(471), len(lens), T, 2 * G, D, std=2.0)
    out, lse = da.decode_attn(q.cuda(), pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=pc.max_len, causal=causal,
                              num_splits=splits, **nan_outputs(q), **pc.scales())
    check_dense(pc, q, out, lse, causal)


@pytest.mark.parametrize("heads", [4, 8])
@pytest.mark.parametrize("G,T,page", [(1, 1, 16), (16, 1, 16), (8, 4, 48), (8, 9, 32)])
def test_fp4_heads_that_share_boxes(da, heads, G, T, page):
    pc = longer(Paged("fp4", [700, 33, 0, 1500, 16], heads, page, 480 + heads, std=1.5), 65280).gpu()
    q = bf16(gen(481), 5, T, heads * G, D, std=2.0)
    out, lse = da.decode_attn(q.cuda(), pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=pc.max_len, causal=T > 1,
                              **nan_outputs(q), **pc.scales())
    check_dense(pc, q, out, lse, T > 1)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("case", [
    # page, lens, G, T, top_k, causal
    (16, [1, 100, 700, 0], 4, 1, 8, False), (16, [513, 2000], 1, 1, 33, False), (48, [1000, 47, 900], 8, 1, 4, True),
    (32, [600, 40, 1], 4, 3, 5, True), (16, [600, 333], 20, 1, 6, False), (16, [300, 17], 2, 5, 2, True),
    (64, [700, 90], 40, 1, 3, False), (16, [333], 100, 1, 9, False)], ids=lambda c: "p%d_g%d_t%d_k%d" % (c[0], c[2], c[3], c[4]))
def test_selected_pages(da, kind, case):
    page, lens, G, T, top_k, causal = case
    pc = Paged(kind, lens, 2, page, 490 + G).gpu()
    q = bf16(gen(491), len(lens), T, 2 * G, D, std=2.0)
    digest = da.block_digest(pc.dk, pc.dbt, pc.dlens, max_seq_len=pc.max_len, k_sf=pc.dk_sf)
    out, lse, blocks = da.decode_attn_sparse(q.cuda(), pc.dk, pc.dv, pc.dbt, pc.dlens, *digest, max_seq_len=pc.max_len,
                                             top_k=top_k, causal=causal, **nan_outputs(q), **pc.scales())
    check_selected(pc, q, out, lse, blocks, causal)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_replayed_graph(da, kind):
    """Dense and sparse attention captured once and replayed into outputs full of NaN."""
    pc = Paged(kind, [800, 90, 333], 2, 16, 500).gpu()
    q = bf16(gen(501), 3, 1, 8, D, std=2.0)
    dq = q.cuda()
    digest = da.block_digest(pc.dk, pc.dbt, pc.dlens, max_seq_len=pc.max_len, k_sf=pc.dk_sf)
    dense, sparse = nan_outputs(q), nan_outputs(q)
    res = {}

    def step():
        da.decode_attn(dq, pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=pc.max_len, **dense, **pc.scales())
        res["blocks"] = da.decode_attn_sparse(dq, pc.dk, pc.dv, pc.dbt, pc.dlens, *digest, max_seq_len=pc.max_len, top_k=7,
                                              **sparse, **pc.scales())[2]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([800, 90, 333], [1, 64, 0], [799, 17, 300]):
        pc.lens = lens
        pc.dlens.copy_(torch.tensor(lens, dtype=torch.int32))
        for t in (*dense.values(), *sparse.values()):
            t.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        check_dense(pc, q, dense["out"], dense["lse"], False)
        check_selected(pc, q, sparse["out"], sparse["lse"], res["blocks"], False)
