"""NaN and infinities in an attention call: a row whose query, or one of whose keys,
is not finite comes out as NaN, with a NaN LSE, however the call is cut into chunks
and whichever merge joins them; rows that see nothing stay 0 and -inf; all others
are what they would be without it."""
import math

import pytest

torch = pytest.importorskip("torch")
from tests import cache_ref as R
from tests.strict import assert_attention
from tests.test_gpu_cache_ops import Paged, bf16, gen

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


# how a call is cut and merged: chunks (0: the plan, on the device from two requests on), two launches
PLANS = {"one chunk": (1, False), "cluster": (4, False), "two launches": (4, True), "many chunks": (40, True),
         "planned": (0, False)}


def attend(da, pc, q, splits, two, **kw):
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    more = dict(k_sf=pc.dk_sf, v_sf=pc.dv_sf) if pc.kind == "fp4" else {}
    da.decode_attn(q.cuda(), pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=pc.max_len, num_splits=splits, two_pass=two,
                   out=out, lse=lse, k_scale=pc.ks, v_scale=pc.vs, **more, **kw)
    return out.cpu().double(), lse.cpu().double()


def check(pc, q, out, lse, bad, causal=False):
    """`bad` [B, T, Hq]: rows that have to be NaN; the others against 64 bits."""
    B, T, Hq, _ = q.shape
    G = Hq // pc.heads
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    k64, v64 = pc.values("k") * pc.ks, pc.values("v") * pc.vs
    tol = R.bf16_p_tolerance if pc.kind == "bf16" else R.out_tolerance
    for b, n in enumerate(pc.lens):
        kb, vb = R.gather(k64, pc.bt, b, n), R.gather(v64, pc.bt, b, n)
        for h in range(pc.heads):
            at = slice(h * G, (h + 1) * G)
            good = ~bad[b, :, at].reshape(T * G)
            if not bool(good.any()):
                continue
            last = torch.tensor([n - T + 1 + t if causal else n for t in range(T) for _ in range(G)])
            seen = torch.arange(n)[None, :] < last[:, None]
            assert_attention(out[b, :, at].reshape(T * G, D)[good], lse[b, :, at].reshape(T * G)[good],
                             q[b, :, at].double().reshape(T * G, D)[good], kb[:, h], vb[:, h], seen[good],
                             1 / math.sqrt(D), tol, (b, h))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf], ids=["nan", "inf", "minus_inf"])
@pytest.mark.parametrize("plan", list(PLANS))
@pytest.mark.parametrize("G", [4, 16, 24, 40, 100])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_query_row(da, kind, G, plan, value):
    pc = Paged(kind, [700, 333], 2, 16, 300 + G).gpu()
    q = bf16(gen(301), 2, 1, 2 * G, D)
    bad = torch.zeros(q.shape[:3], dtype=torch.bool)
    for b, h, d in ((0, 1, 3), (1, G, 127), (1, 2 * G - 1, 64)):
        q[b, 0, h, d] = value
        bad[b, 0, h] = True
    out, lse = attend(da, pc, q, *PLANS[plan])
    check(pc, q, out, lse, bad)


@pytest.mark.parametrize("plan", list(PLANS))
@pytest.mark.parametrize("G,T", [(4, 4), (8, 8)])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_query_row_beside_rows_that_see_nothing(da, kind, G, T, plan):
    """A request shorter than its new tokens: NaN in a row that sees nothing is not looked at."""
    pc = Paged(kind, [500, T - 2], 2, 16, 310 + G).gpu()
    q = bf16(gen(311), 2, T, 2 * G, D)
    bad = torch.zeros(q.shape[:3], dtype=torch.bool)
    q[1, 0, 2, 5] = math.nan                     # (token 0 of a request of T - 2: sees nothing)
    q[1, T - 1, 1, 5] = math.nan
    q[0, 0, 0, 0] = math.nan
    bad[1, T - 1, 1] = bad[0, 0, 0] = True
    out, lse = attend(da, pc, q, *PLANS[plan], causal=True)
    clean = q.clone()
    clean[1, 0, 2, 5] = 0.0
    check(pc, clean, out, lse, bad, causal=True)


@pytest.mark.parametrize("plan", list(PLANS))
@pytest.mark.parametrize("G", [4, 16, 40])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_one_key(da, kind, G, plan):
    """NaN in one seen key of one KV head: every row of that head, none of another's."""
    pc = Paged(kind, [700, 333], 2, 16, 320 + G)
    q = bf16(gen(321), 2, 1, 2 * G, D)
    page, slot = int(pc.bt[0, 37]), 9            # token 601 of request 0
    if kind == "bf16":
        pc.k[page, slot, 1, 20] = math.nan
    elif kind == "fp8":
        pc.k[page, slot, 1, 20] = 0x7F
    else:
        pc.k_sf[page, 1, slot, 2] = 0x7F
    pc.gpu()
    bad = torch.zeros(q.shape[:3], dtype=torch.bool)
    bad[0, :, G:] = True
    out, lse = attend(da, pc, q, *PLANS[plan])
    check(pc, q, out, lse, bad)


@pytest.mark.parametrize("plan", ["two launches", "planned"])
@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_query_row_among_many(da, kind, plan):
    """More rows than the merge with a CTA per row takes."""
    lens = [(97 * i) % 600 for i in range(70)]
    pc = Paged(kind, lens, 2, 16, 330).gpu()
    q = bf16(gen(331), 70, 1, 32, D)
    bad = torch.zeros(q.shape[:3], dtype=torch.bool)
    for b, h in ((1, 0), (33, 31), (69, 16)):
        q[b, 0, h, 77] = math.nan
        bad[b, 0, h] = True
    out, lse = attend(da, pc, q, *PLANS[plan])
    check(pc, q, out, lse, bad)


@pytest.mark.parametrize("G", [4, 24, 100])
@pytest.mark.parametrize("top_k", [3, 30])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_query_row_over_selected_pages(da, kind, top_k, G):
    pc = Paged(kind, [900, 333, 20], 2, 16, 340 + G).gpu()
    q = bf16(gen(341), 3, 1, 2 * G, D)
    bad = torch.zeros(q.shape[:3], dtype=torch.bool)
    for b, h, x in ((0, 1, math.nan), (1, G, math.inf), (2, 2 * G - 1, math.nan)):
        q[b, 0, h, 11] = x
        bad[b, 0, h] = True
    digest = da.block_digest(pc.dk, pc.dbt, pc.dlens, max_seq_len=pc.max_len, k_sf=pc.dk_sf)
    out, lse, blocks = da.decode_attn_sparse(q.cuda(), pc.dk, pc.dv, pc.dbt, pc.dlens, *digest, max_seq_len=pc.max_len,
                                             top_k=top_k, **pc.scales())
    out, lse, blocks = out.cpu().double(), lse.cpu().double(), blocks.cpu()
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    k64, v64 = pc.values("k") * pc.ks, pc.values("v") * pc.vs
    tol = R.bf16_p_tolerance if kind == "bf16" else R.out_tolerance
    for b, n in enumerate(pc.lens):
        for h in range(2):
            at = blocks[b, 0, h]
            at = at[at >= 0].long()
            m = len(at) * 16 - (-(-n // 16) * 16 - n)
            kk, vv = (x[pc.bt[b].long()[at]][:, :, h].flatten(0, 1)[:m] for x in (k64, v64))
            rows = slice(h * G, (h + 1) * G)
            good = ~bad[b, 0, rows]
            assert_attention(out[b, 0, rows][good], lse[b, 0, rows][good], q[b, 0, rows].double()[good], kk, vv,
                             torch.ones(int(good.sum()), m, dtype=torch.bool), 1 / math.sqrt(D), tol, (b, h))


@pytest.mark.parametrize("S", [3, 40])
def test_merge_alone(da, S):
    """Partials whose LSEs are NaN are not those of a row without keys."""
    chunk = 64
    lens = torch.tensor([S * chunk, 2 * chunk], dtype=torch.int32)
    p = da.decode_attn_params_init(2, 1, 4, 1, D, 0, 0, 0, S * chunk, False)
    p.flags = da.DA_FLAG_TWO_PASS
    g = gen(350)
    part_o = torch.randn(2, 1, 4, S, D, generator=g)
    part_l = torch.randn(2, 1, 4, S, generator=g)
    part_l[0, 0, 0], part_o[0, 0, 0] = -math.inf, 0.0     # no keys
    part_l[0, 0, 1] = math.nan                            # nothing but NaN
    part_l[0, 0, 2], part_l[0, 0, 2, S - 1] = -math.inf, math.nan
    part_l[0, 0, 3, 1] = math.nan
    part_l[1, 0, 0, :2] = math.nan
    part_l[1, 0, 1, 2:], part_o[1, 0, 1, 2:] = math.nan, math.nan  # (behind the request's chunks: stale)
    ws = torch.cat([part_o.flatten(), part_l.flatten()]).cuda()
    out = torch.full((2, 1, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, 1, 4), 7.0, device="cuda")
    da.decode_attn_combine(p, lens.cuda(), S, chunk, ws, out, lse)
    out, lse = out.cpu().double(), lse.cpu().double()
    assert not bool(out[0, 0, 0].any()) and float(lse[0, 0, 0]) == -math.inf
    for b, h in ((0, 1), (0, 2), (0, 3), (1, 0)):
        assert bool(out[b, 0, h].isnan().all()) and bool(lse[b, 0, h].isnan()), (b, h)
    for h in (1, 2, 3):
        w = torch.softmax(part_l[1, 0, h, :2].double(), 0)
        want = w @ part_o[1, 0, h, :2].double()
        # bf16 rounding 2^-8; weights and sums in fp32, exponentials to 2^-21
        assert bool(((out[1, 0, h] - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18).all())
        assert abs(float(lse[1, 0, h]) - float(torch.logsumexp(part_l[1, 0, h, :2].double(), 0))) <= 2.0 ** -18


@pytest.mark.parametrize("plan", list(PLANS))
@pytest.mark.parametrize("G", [4, 16, 24, 40])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_scores_that_are_all_minus_infinity(da, kind, G, plan):
    """They weigh nothing: 0 and -inf, as where there are no keys, in every merge."""
    pc = Paged(kind, [700, 333], 2, 16, 360 + G)
    if kind == "bf16":
        pc.k[..., 5] = -1.0
    elif kind == "fp8":
        pc.k[..., 5] = 0xB8                      # -1
    else:
        pc.k[..., 2] = (pc.k[..., 2] & 0x0F) | 0xA0
        pc.k_sf[..., 0] = 0x38
    pc.gpu()
    q = bf16(gen(361), 2, 1, 2 * G, D)
    q[0, 0, 1, 5] = q[1, 0, G, 5] = math.inf
    out, lse = attend(da, pc, q, *PLANS[plan])
    bad = torch.zeros(q.shape[:3], dtype=torch.bool)
    for b, h in ((0, 1), (1, G)):
        assert not bool(out[b, 0, h].any()) and float(lse[b, 0, h]) == -math.inf
        bad[b, 0, h] = True
        out[b, 0, h], lse[b, 0, h] = math.nan, math.nan      # (the others are checked as above)
    check(pc, q, out, lse, bad)
