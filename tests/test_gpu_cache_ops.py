"""GPU parity of the operators around the cache: rotary tables, the append into
caches of every type, page digests, attention over 4-bit caches and over selected
pages, and a decode step made of all of them.  References: tests/cache_ref.py."""
import math
from decimal import Decimal, getcontext

import pytest

torch = pytest.importorskip("torch")
from tests import cache_ref as R

pytestmark = pytest.mark.gpu
D = 128
SCALES = {"bf16": (1.0, 1.0), "fp8": (0.0625, 0.037), "fp4": (0.02, 0.015)}


@pytest.fixture(scope="module")
def da():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from split_kv_decode_attention_gb300 import binding as B
    from split_kv_decode_attention_gb300 import build as cuda_build
    cuda_build.build()
    B.lib()
    return B


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def bf16(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def as_cache(x, kind, scale):
    """bf16 values [G, S, H, 128] -> (cache, block scales [G, H, S, 8] or None)."""
    if kind == "bf16":
        return x.clone(), None
    if kind == "fp8":
        return R.to_e4m3(x.float() * (R.f32(1.0) / R.f32(scale))), None
    codes, sf = R.quant_fp4(x, scale)
    return codes, sf.permute(0, 2, 1, 3).contiguous()


class Paged:
    """Ragged requests over shuffled pages (or a contiguous cache), on the CPU and the GPU."""

    def __init__(self, kind, lens, heads, page, seed, std=1.0, extra_pages=2, width=None):
        g = gen(seed)
        self.kind, self.lens, self.page, self.heads = kind, list(lens), page, heads
        self.ks, self.vs = SCALES[kind]
        if page:
            need = [-(-n // page) for n in lens]
            groups = sum(need) + extra_pages
            ids = torch.randperm(groups, generator=g).to(torch.int32)
            self.bt = torch.zeros(len(lens), max(max(need), 1) if width is None else width, dtype=torch.int32)
            at = 0
            for b, n in enumerate(need):
                self.bt[b, :n] = ids[at:at + n]
                at += n
            tokens = page
        else:
            groups, tokens, self.bt = len(lens), -(-max(max(lens), 1) // 16) * 16, None
        self.k, self.k_sf = as_cache(bf16(g, groups, tokens, heads, D, std=std), kind, self.ks)
        self.v, self.v_sf = as_cache(bf16(g, groups, tokens, heads, D), kind, self.vs)
        self.max_len = max(max(lens), 1)

    def gpu(self):
        self.dk, self.dv, self.dk_sf, self.dv_sf, self.dbt = (
            None if t is None else t.cuda() for t in (self.k, self.v, self.k_sf, self.v_sf, self.bt))
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        return self

    def scales(self):
        return dict(k_scale=self.ks, v_scale=self.vs, k_sf=self.dk_sf, v_sf=self.dv_sf)

    def values(self, which):
        cache, sf = (self.k, self.k_sf) if which == "k" else (self.v, self.v_sf)
        return R.cache_values(self.kind, cache, sf)


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ rotary table
@pytest.mark.parametrize("n,count,first,amp", [(1, 1, 0, 1.0), (64, 4096, 0, 1.0), (5, 1000, 17, 1.25),
                                               (40, 333, 100000, 0.5), (64, 2000, 1 << 20, 1.0)])
def test_rope_table_matches_64_bits(da, n, count, first, amp):
    f, _ = da.rope_frequencies(2 * n, base=10000.0)
    out = da.rope_table(f.cuda(), count, amplitude=amp, first=first).cpu().double()
    a = (first + torch.arange(count, dtype=torch.float64))[:, None] * f
    want = torch.cat([a.cos(), a.sin()], dim=1) * amp
    # sincospif: 1 ulp (2^-23), its argument 2^-24 of at most pi / 4, the amplitude and
    # the product 2^-24 each; the reference's angle: 2^-53 of itself, twice
    tol = amp * (2.0 ** -23 + 3 * 2.0 ** -24) + amp * (first + count) * 2.0 ** -52
    assert float((out - want).abs().max()) <= tol


def test_rope_table_far_positions_against_decimal(da):
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    f = torch.tensor([1.0, 0.7310585786300049, 3.0e-5, 2.5, 1e-9], dtype=torch.float64)
    first = (1 << 31) - 3
    out = da.rope_table(f.cuda(), 3, first=first).cpu().double()
    for r in range(3):
        for i, x in enumerate(f.tolist()):
            a = float((Decimal(first + r) * Decimal(x)) % two_pi)  # exact product, one rounding
            # F is off by under 2^-63 turns (two fp64 roundings), times the position
            tol = 2.0 ** -23 + 3 * 2.0 ** -24 + 2 * math.pi * first * 2.0 ** -63 + 2.0 ** -50
            assert abs(float(out[r, i]) - math.cos(a)) <= tol
            assert abs(float(out[r, 5 + i]) - math.sin(a)) <= tol


def test_rope_table_frequency_not_finite_gives_nan(da):
    f = torch.tensor([1.0, math.inf, math.nan], dtype=torch.float64).cuda()
    out = da.rope_table(f, 4).cpu()
    assert bool(out[:, [1, 2, 4, 5]].isnan().all()) and not bool(out[:, [0, 3]].isnan().any())


# ------------------------------------------------------------------ append
def append_reference(pc, q, k, v, table, T, new_lens, positions, interleaved):
    """The caches and q_out (fp64, None where left alone) that a call should give."""
    rot = 0 if table is None else table.shape[1]
    want = {"k": pc.k.clone(), "v": pc.v.clone(),
            "k_sf": None if pc.k_sf is None else pc.k_sf.clone(),
            "v_sf": None if pc.v_sf is None else pc.v_sf.clone()}
    rows = {}
    for b, L in enumerate(pc.lens):
        n = T if new_lens is None else new_lens[b]
        for t in range(n):
            at = L - n + t
            if at < 0:
                continue
            pos = at if positions is None else int(positions[b, t])
            if rot and not 0 <= pos < table.shape[0]:
                continue
            group, slot = (b, at) if pc.bt is None else (int(pc.bt[b, at // pc.page]), at % pc.page)
            c, s = (table[pos, :rot // 2], table[pos, rot // 2:]) if rot else (torch.zeros(0), torch.zeros(0))
            if q is not None:
                rows[b, t] = (R.rotate(q[b, t], c, s, rot, interleaved, torch.float64),
                              R.rotate(q[b, t].abs(), c.abs(), -s.abs(), rot, interleaved, torch.float64).abs()
                              + 2 * q[b, t].double().abs())
            if k is not None:
                new_k = R.rotate(k[b, t], c, s, rot, interleaved, torch.float32).to(torch.bfloat16)
                for name, x, scale in (("k", new_k, pc.ks), ("v", v[b, t], pc.vs)):
                    cc, sf = as_cache(x[None, None], pc.kind, scale)
                    want[name][group, slot] = cc[0, 0]
                    if sf is not None:
                        want[name + "_sf"][group, :, slot] = sf[0, :, 0]
    return want, rows


def check_append(da, kind, page, lens, T, hq, hkv, rot, interleaved, seed, new_lens=None, positions=None,
                 in_place=False, fused=True, table_rows=None):
    pc = Paged(kind, lens, hkv, page, seed).gpu()
    g = gen(seed + 1)
    B = len(lens)
    qkv = bf16(g, B, T, hq + 2 * hkv, D, std=2.0)
    dqkv = qkv.cuda()
    parts = (qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:])
    dparts = [dqkv[:, :, :hq], dqkv[:, :, hq:hq + hkv], dqkv[:, :, hq + hkv:]]
    if not fused:
        dparts = [x.contiguous() for x in dparts]
    table = None
    if rot:
        f, _ = da.rope_frequencies(rot)
        table = da.rope_table(f.cuda(), table_rows or max(lens) + 1)
    q_out = dparts[0] if in_place else torch.full((B, T, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    st = status_word()
    dpos = None if positions is None else torch.tensor(positions, dtype=torch.int32).cuda()
    dnew = None if new_lens is None else torch.tensor(new_lens, dtype=torch.int32).cuda()
    da.rope_append(*dparts, table, pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=pc.max_len,
                   interleaved=interleaved, positions=dpos, new_lens=dnew, q_out=q_out, status=st, **pc.scales())
    want, rows = append_reference(pc, *parts, None if table is None else table.cpu(), T, new_lens,
                                  None if positions is None else torch.tensor(positions), interleaved)
    for name, got in (("k", pc.dk), ("v", pc.dv), ("k_sf", pc.dk_sf), ("v_sf", pc.dv_sf)):
        if got is not None:
            a, w = got.cpu(), want[name]
            assert torch.equal(a.view(torch.uint8) if a.dtype != torch.bfloat16 else a.view(torch.int16),
                               w.view(torch.uint8) if w.dtype != torch.bfloat16 else w.view(torch.int16)), name
    got = q_out.cpu()
    for b in range(B):
        for t in range(T):
            if (b, t) in rows:
                ref, mag = rows[b, t]
                # bf16 half a step, and three fp32 roundings of the two products
                tol = 2.0 ** -8 * ref.abs() + 3 * 2.0 ** -24 * mag
                assert bool(((got[b, t].double() - ref).abs() <= tol).all()), (b, t)
            else:
                assert torch.equal(got[b, t], parts[0][b, t] if in_place else torch.full_like(got[b, t], 7.0))
    return int(st.item())


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("rot", [0, 2, 8, 16, 20, 24, 72, 96, 120, 126, 128])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_append_one_token(da, kind, rot, interleaved):
    assert check_append(da, kind, 16, [1, 17, 40, 16], 1, 4, 2, rot, interleaved, 5) == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("page,hq,hkv,T,lens", [
    (0, 3, 1, 5, [5, 9, 33]), (48, 5, 5, 7, [7, 60, 100]), (16, 8, 1, 40, [40, 41, 56]),
    (64, 12, 3, 2, [2, 64, 65, 66, 129]), (16, 1, 1, 1, [1])])
def test_append_shapes(da, kind, page, hq, hkv, T, lens):
    assert check_append(da, kind, page, lens, T, hq, hkv, 64, False, 11 + T) == 0
    assert check_append(da, kind, page, lens, T, hq, hkv, 128, True, 12 + T, fused=False) == 0


@pytest.mark.parametrize("rot", [20, 24, 128])
@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_append_in_place(da, kind, rot):
    assert check_append(da, kind, 16, [20, 33], 3, 6, 2, rot, False, 21, in_place=True) == 0


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_append_padded_rows_positions_and_short_requests(da, kind):
    # right-padded new tokens; angles of their own
    assert check_append(da, kind, 16, [20, 33, 6], 4, 4, 2, 64, False, 31, new_lens=[4, 0, 2]) == 0
    pos = [[0, 5, 9, 1], [40, 41, 42, 43], [7, 7, 7, 7]]
    assert check_append(da, kind, 16, [20, 33, 6], 4, 4, 2, 64, True, 32, positions=pos, table_rows=50) == 0
    # fewer tokens than new ones: the first rows have no place
    assert check_append(da, kind, 16, [2, 33, 0], 4, 4, 2, 64, False, 33) == da.DA_STATUS_SHORT_CAUSAL
    # a position without a row in the table, on both sides
    pos[1][2], pos[2][0] = 50, -1
    assert check_append(da, kind, 16, [20, 33, 6], 4, 4, 2, 64, False, 34, positions=pos,
                        table_rows=50) == da.DA_STATUS_POSITION


def test_append_special_values(da):
    """Zeros, NaN, infinities, ties and tiny blocks in every cache type."""
    x = torch.zeros(1, 1, 2, D)
    x[0, 0, 0, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5,
                                    -3.5, -5.0, -6.0])
    x[0, 0, 0, 16:32] = math.nan
    x[0, 0, 0, 32] = math.inf
    x[0, 0, 0, 33] = -3.0
    x[0, 0, 0, 48:64] = 1e-6
    x[0, 0, 0, 64] = -math.nan
    x[0, 0, 0, 65:70] = torch.tensor([1.0, -1.0, -0.0, 0.0, 0.1])
    x[0, 0, 1] = torch.linspace(-448 * 7, 448 * 7, D)
    x = x.to(torch.bfloat16)
    for kind in ("bf16", "fp8", "fp4"):
        pc = Paged(kind, [3], 2, 16, 3).gpu()
        pc.ks = pc.vs = 1.0
        da.rope_append(None, x.cuda(), x.cuda(), None, pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=3, **pc.scales())
        want, sf = as_cache(x, kind, 1.0)
        page = int(pc.bt[0, 0])
        for got, got_sf in ((pc.dk, pc.dk_sf), (pc.dv, pc.dv_sf)):
            a, w = got.cpu()[page, 2], want[0, 0]
            if kind == "fp4":
                assert torch.equal(a, w) and torch.equal(got_sf.cpu()[page, :, 2], sf[0, :, 0])
            else:  # (any NaN for a NaN)
                a, w = (t.view(R.E4M3).float() if kind == "fp8" else t.float() for t in (a, w))
                assert torch.equal(a.isnan(), w.isnan()) and torch.equal(a.nan_to_num(9.0, 8.0, 7.0), w.nan_to_num(9.0, 8.0, 7.0))


def test_append_bad_page_is_not_written(da):
    pc = Paged("bf16", [20, 33], 2, 16, 41).gpu()
    pc.dbt[0, 1] = pc.dk.shape[0]
    pc.dbt[1, 2] = -1
    before = pc.dk.clone(), pc.dv.clone()
    g = gen(42)
    q, k, v = (bf16(g, 2, 1, h, D).cuda() for h in (4, 2, 2))
    st = status_word()
    out = da.rope_append(q, k, v, None, pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=33, status=st)
    assert int(st.item()) == da.DA_STATUS_BAD_PAGE
    assert torch.equal(pc.dk, before[0]) and torch.equal(pc.dv, before[1]) and torch.equal(out, q)


def test_append_rotation_is_undone_by_its_gradient(da):
    """The transposed rotation (the table's sines negated) is the gradient of the
    rotation; applied to a rotated vector it gives the vector back."""
    f, _ = da.rope_frequencies(96)
    table = da.rope_table(f.cuda(), 600)
    back = torch.cat([table[:, :48], -table[:, 48:]], dim=1).contiguous()
    g = gen(8)
    q = bf16(g, 2, 300, 4, D).cuda()
    cache = torch.zeros(2, 512, 4, D, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([300, 512], dtype=torch.int32, device="cuda")
    kw = dict(max_seq_len=512)
    y = da.rope_append(q, None, None, table, cache, cache, None, lens, **kw)
    x = da.rope_append(y, None, None, back, cache, cache, None, lens, **kw)
    # y is off by 2^-8 of itself; turned back, both values of a pair mix, and x rounds again
    pair = (y.double()[..., :48].square() + y.double()[..., 48:96].square()).sqrt()
    tol = torch.cat([pair, pair, y.double()[..., 96:].abs()], dim=-1) * (2 * 2.0 ** -8 + 2.0 ** -8 + 2.0 ** -20)
    assert bool(((x.double() - q.double()).abs() <= tol).all())
    assert not bool(cache.any())


# ------------------------------------------------------------------ digests
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("page,heads,lens,max_new", [
    (16, 2, [1, 16, 17, 0, 250], 0), (48, 3, [47, 48, 49, 200], 0), (64, 1, [640], 0), (16, 8, [5, 16, 33, 0], 1),
    (16, 2, [40, 100, 3], 17), (128, 5, [1000, 129], 2)])
def test_digest(da, kind, page, heads, lens, max_new):
    pc = Paged(kind, lens, heads, page, 50 + page).gpu()
    P = pc.k.shape[0]
    dg = torch.full((P, heads, 2, D), 3, dtype=torch.int8, device="cuda")
    ds = torch.full((P, heads), -1.0, device="cuda")
    st = status_word()
    da.block_digest(pc.dk, pc.dbt, pc.dlens, dg, ds, max_seq_len=pc.max_len, max_new=max_new, k_sf=pc.dk_sf, status=st)
    assert int(st.item()) == 0
    want_d, want_s = torch.full((P, heads, 2, D), 3, dtype=torch.int8), torch.full((P, heads), -1.0)
    x = pc.values("k").float()
    for b, n in enumerate(lens):
        lo = max(0, n - max_new) // page if max_new else 0
        for c in range(lo, -(-n // page)):
            pg = int(pc.bt[b, c])
            for h in range(heads):
                want_d[pg, h], want_s[pg, h] = R.digest_page(x[pg, :min(page, n - c * page), h])
    assert torch.equal(dg.cpu(), want_d) and torch.equal(ds.cpu(), want_s)


def test_digest_special_values(da):
    k = torch.zeros(4, 16, 1, D)
    k[1, :, 0, 0] = math.nan                 # a channel of NaN only
    k[1, 3, 0, 1] = math.nan
    k[1, :, 0, 2] = torch.linspace(-2, 5, 16)
    k[2, 5, 0, 7] = math.inf
    k[2, 6, 0, 8] = -math.inf
    k[2, 6, 0, 9] = 3.0
    k[3, 9:] = math.nan                      # behind the sequence: not read
    k[3, :9, 0] = torch.randn(9, D, generator=gen(1))
    k = k.to(torch.bfloat16)
    bt = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32)
    dg, ds = da.block_digest(k.cuda(), bt.cuda(), torch.tensor([57], dtype=torch.int32).cuda(), max_seq_len=64)
    for p in range(4):
        d, s = R.digest_page(k[p, :9 if p == 3 else 16, 0].float())
        assert torch.equal(dg.cpu()[p, 0], d) and float(ds[p, 0]) == float(s), p


def test_digest_bad_pages_and_lengths(da):
    pc = Paged("bf16", [40, 20], 2, 16, 61).gpu()
    pc.dbt[0, 1] = 99
    pc.dlens[1] = 1000
    st = status_word()
    dg, ds = da.block_digest(pc.dk, pc.dbt, pc.dlens, max_seq_len=40, status=st)
    assert int(st.item()) == da.DA_STATUS_BAD_PAGE | da.DA_STATUS_SEQ_LEN


# ------------------------------------------------------------------ attention over 4-bit caches
def check_attention(pc, q, out, lse, causal, scale, tolerance=R.out_tolerance):
    B, T, Hq, _ = q.shape
    G = Hq // pc.heads
    k64, v64 = pc.values("k") * pc.ks, pc.values("v") * pc.vs
    out, lse = out.cpu().double(), lse.cpu().double()
    for b, n in enumerate(pc.lens):
        kb, vb = R.gather(k64, pc.bt, b, n), R.gather(v64, pc.bt, b, n)
        for h in range(pc.heads):
            rows = q[b, :, h * G:(h + 1) * G].double().reshape(T * G, D)
            last = torch.tensor([n - T + 1 + t if causal else n for t in range(T) for _ in range(G)])
            seen = torch.arange(n)[None, :] < last[:, None]
            o, l, wabs, mag = R.attention_rows(rows, kb[:, h], vb[:, h], seen, scale)
            got = out[b, :, h * G:(h + 1) * G].reshape(T * G, D)
            gl = lse[b, :, h * G:(h + 1) * G].reshape(T * G)
            assert torch.equal(gl.isinf(), l.isinf()), (b, h)
            f = ~l.isinf()
            assert bool(((gl - l).abs() <= R.lse_tolerance(l, mag))[f].all()), (b, h, float((gl - l)[f].abs().max()))
            bad = (got - o).abs() > tolerance(o, wabs, mag)
            assert not bool(bad.any()), (b, h, float((got - o).abs().max()))
            assert not bool(got[~f].any())


FP4_CASES = [
    # heads per KV head, q_len, causal, page, lens
    (1, 1, False, 16, [1, 15, 16, 17, 31, 32, 33, 700]), (4, 1, False, 0, [512, 1, 333]),
    (8, 1, False, 48, [129, 48, 1000]), (7, 1, False, 16, [0, 5, 300, 0]), (4, 4, True, 16, [4, 100, 777]),
    (2, 3, False, 32, [3, 64, 65]), (16, 1, False, 64, [1, 900]), (5, 7, True, 16, [7, 200]),
    (8, 4, True, 16, [4, 33, 500]), (8, 8, True, 128, [8, 129, 600]), (16, 8, True, 16, [8, 300]),
    (33, 1, False, 32, [0, 1, 64, 65, 400]), (10, 4, True, 0, [4, 70, 511]), (64, 2, True, 48, [2, 1, 1000]),
    (4, 4, True, 16, [2, 1, 40]),  # causal requests shorter than q_len: rows that see nothing
]


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("case", FP4_CASES, ids=lambda c: "g%d_t%d_%s_p%d" % (c[0], c[1], "causal" if c[2] else "full", c[3]))
def test_fp4_attention(da, case, splits):
    G, T, causal, page, lens = case
    pc = Paged("fp4", lens, 2, page, 70 + G + T, std=1.5).gpu()
    q = bf16(gen(71), len(lens), T, 2 * G, D, std=2.0)
    st = status_word()
    out, lse = da.decode_attn(q.cuda(), pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=pc.max_len, causal=causal,
                              num_splits=splits, status=st, **pc.scales())
    assert int(st.item()) == (da.DA_STATUS_SHORT_CAUSAL if causal and min(lens) < T else 0)
    check_attention(pc, q, out, lse, causal, 1 / math.sqrt(D))


@pytest.mark.parametrize("G", [4, 40, 80])
@pytest.mark.parametrize("factor", [2.0 ** 60, 2.0 ** -60, 3.0e5, 1e-5])
def test_fp4_attention_query_range(da, factor, G):
    """q far outside f16's range gives what the scale makes of it."""
    pc = Paged("fp4", [200, 31], 2, 16, 75).gpu()
    q = (bf16(gen(76), 2, 1, 2 * G, D, std=2.0).float() * factor).to(torch.bfloat16)
    out, lse = da.decode_attn(q.cuda(), pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=pc.max_len,
                              scale=1 / math.sqrt(D) / factor, **pc.scales())
    check_attention(pc, q, out, lse, False, float(R.f32(1 / math.sqrt(D) / factor)))


@pytest.mark.parametrize("G", [1, 36, 128])
def test_fp4_attention_long_tail_of_small_weights(da, G):
    """One key far above 60000 others whose weights are each below f16's smallest
    number of one: together they still count."""
    n = 60000
    pc = Paged("fp4", [n], 1, 64, 77)
    pc.k_sf[:] = 0
    pc.v[:] = 0x22                                # code 2 = 1.0 everywhere
    pc.v_sf[:] = 0x38                             # E4M3 1.0
    first = int(pc.bt[0, 0])
    pc.k[first, 0] = 0x77                         # 6.0 along all of d
    pc.k_sf[first, :, 0] = 0x38
    pc.v[first, 0] = 0xAA                         # -1.0
    pc.ks, pc.vs = 1.0, 1.0
    pc.gpu()
    q = torch.zeros(1, 1, G, D)
    q[..., 0] = 18.5 * math.log(2) * math.sqrt(D) / 6   # weight of the others: 2^-18.5
    q = q.to(torch.bfloat16)
    out, lse = da.decode_attn(q.cuda(), pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=n, **pc.scales())
    check_attention(pc, q, out, lse, False, 1 / math.sqrt(D))
    assert float(out[..., 0].min()) > -0.75       # (-1 + 0.15) / 1.15, not -1


@pytest.mark.parametrize("splits", [0, 2])
def test_fp4_attention_poisoned_slots(da, splits):
    """Nothing behind a sequence, in its last page or in other pages, is read:
    NaN block scales there leave the bits as they were."""
    lens = [1, 17, 40, 0, 63]
    for page, G in ((16, 4), (48, 4), (0, 4), (16, 20), (64, 40), (0, 40)):
        pc = Paged("fp4", lens, 2, page, 80).gpu()
        q = bf16(gen(81), 5, 2, 2 * G, D).cuda()
        kw = dict(max_seq_len=pc.max_len, num_splits=splits)
        clean = da.decode_attn(q, pc.dk, pc.dv, pc.dbt, pc.dlens, **kw, **pc.scales())
        live = torch.zeros(pc.k.shape[:2], dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(n):
                live[(int(pc.bt[b, j // page]), j % page) if page else (b, j)] = True
        dead = (~live).cuda()
        for c, sf in ((pc.dk, pc.dk_sf), (pc.dv, pc.dv_sf)):
            c[dead] = 0xFF
            sf.permute(0, 2, 1, 3)[dead] = 0x7F
        out, lse = da.decode_attn(q, pc.dk, pc.dv, pc.dbt, pc.dlens, **kw, **pc.scales())
        assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


def longer(pc, max_len):
    """The same requests under a larger max_seq_len: a wider block table, -1 behind
    the pages that exist."""
    wide = torch.full((len(pc.lens), -(-max_len // pc.page)), -1, dtype=torch.int32)
    for b, n in enumerate(pc.lens):
        wide[b, :-(-n // pc.page)] = pc.bt[b, :-(-n // pc.page)]
    pc.bt, pc.max_len = wide, max_len
    return pc


@pytest.mark.parametrize("splits", [0, 128])
@pytest.mark.parametrize("heads", [2, 4, 8, 12])
@pytest.mark.parametrize("G,T,page", [(1, 1, 16), (8, 1, 64), (16, 1, 16), (8, 4, 48), (8, 9, 32)])
def test_fp4_attention_heads_that_share_boxes(da, heads, G, T, page, splits):
    """Calls with work enough for CTAs of two, four and eight KV heads."""
    pc = longer(Paged("fp4", [700, 33, 0, 1500, 16], heads, page, 170 + heads, std=1.5), 65280).gpu()
    q = bf16(gen(171), 5, T, heads * G, D, std=2.0)
    out, lse = da.decode_attn(q.cuda(), pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=pc.max_len, causal=T > 1,
                              num_splits=splits, **pc.scales())
    check_attention(pc, q, out, lse, T > 1, 1 / math.sqrt(D))


@pytest.mark.parametrize("splits", [0, 1])
def test_fp4_attention_many_requests_in_a_contiguous_cache(da, splits):
    lens = [(37 * i) % 257 for i in range(320)]
    pc = Paged("fp4", lens, 2, 0, 172).gpu()
    q = bf16(gen(173), 320, 1, 8, D, std=2.0)
    out, lse = da.decode_attn(q.cuda(), pc.dk, pc.dv, None, pc.dlens, max_seq_len=pc.max_len, num_splits=splits,
                              **pc.scales())
    check_attention(pc, q, out, lse, False, 1 / math.sqrt(D))


@pytest.mark.parametrize("G", [1, 20, 48])
def test_fp4_attention_more_requests_than_a_planner_holds(da, G):
    lens = [(13 * i) % 41 for i in range(1100)]
    pc = Paged("fp4", lens, 1, 16, 174).gpu()
    q = bf16(gen(175), 1100, 1, G, D, std=2.0)
    out, lse = da.decode_attn(q.cuda(), pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=pc.max_len, **pc.scales())
    check_attention(pc, q, out, lse, False, 1 / math.sqrt(D))


def test_fp4_attention_poisoned_slots_of_shared_boxes(da):
    pc = longer(Paged("fp4", [1, 17, 140, 0, 63], 8, 48, 176), 65280).gpu()
    q = bf16(gen(177), 5, 1, 16, D).cuda()
    clean = da.decode_attn(q, pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=pc.max_len, **pc.scales())
    live = torch.zeros(pc.k.shape[:2], dtype=torch.bool)
    for b, n in enumerate(pc.lens):
        for j in range(n):
            live[int(pc.bt[b, j // 48]), j % 48] = True
    dead = (~live).cuda()
    for c, sf in ((pc.dk, pc.dk_sf), (pc.dv, pc.dv_sf)):
        c[dead] = 0xFF
        sf.permute(0, 2, 1, 3)[dead] = 0x7F
    out, lse = da.decode_attn(q, pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=pc.max_len, **pc.scales())
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


def test_fp4_attention_one_launch_and_two(da):
    """The cluster merge and the merge of partials agree with the reference, into
    tensors that the caller gives."""
    pc = Paged("fp4", [2000, 1111], 2, 16, 178).gpu()
    q = bf16(gen(179), 2, 1, 8, D, std=2.0)
    out = torch.full((2, 1, 8, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, 1, 8), 7.0, device="cuda")
    for two in (False, True):
        ws = torch.full((1 << 22,), 0xFF, dtype=torch.uint8, device="cuda")
        got = da.decode_attn(q.cuda(), pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=2000, num_splits=4, out=out, lse=lse,
                             workspace=ws, two_pass=two, **pc.scales())
        assert got[0].data_ptr() == out.data_ptr() and got[1].data_ptr() == lse.data_ptr()
        assert bool((ws != 0xFF).any()) == two
        check_attention(pc, q, out, lse, False, 1 / math.sqrt(D))
        out.fill_(7.0)
        lse.fill_(7.0)


def test_fp4_attention_bad_pages_and_lengths(da):
    pc = Paged("fp4", [40, 20], 2, 16, 82).gpu()
    q = bf16(gen(83), 2, 1, 4, D).cuda()
    pc.dbt[0, 1] = 1000
    pc.dlens[1] = -5
    for splits in (0, 1):
        st = status_word()
        out, lse = da.decode_attn(q, pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=40, status=st, num_splits=splits,
                                  **pc.scales())
        assert int(st.item()) == da.DA_STATUS_BAD_PAGE | da.DA_STATUS_SEQ_LEN
        assert not bool(out[1].any()) and bool(lse[1].isinf().all())
    pc.bt[0, 1] = 0                               # (page 0 is read instead)
    pc.lens = [40, 0]
    check_attention(pc, q.cpu(), out, lse, False, 1 / math.sqrt(D))


def test_fp4_attention_nan_scale_in_a_seen_key_spreads(da):
    pc = Paged("fp4", [40], 1, 16, 84).gpu()
    pc.dv_sf[int(pc.bt[0, 0]), 0, 3, 1] = 0x7F
    q = bf16(gen(85), 1, 1, 2, D).cuda()
    out, _ = da.decode_attn(q, pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=40, **pc.scales())
    assert bool(out[..., 16:32].isnan().all()) and not bool(out[..., :16].isnan().any()) and not bool(out[..., 32:].isnan().any())


def test_fp4_attention_strides(da):
    """Caches as views: heads outermost, q and out inside larger tensors."""
    pc = Paged("fp4", [70, 33, 16], 3, 16, 86).gpu()
    q = bf16(gen(87), 3, 2, 9, D)
    big = torch.zeros(3, 2, 20, D, dtype=torch.bfloat16, device="cuda")
    big[:, :, 5:14] = q.cuda()
    out = torch.zeros(3, 4, 9, D, dtype=torch.bfloat16, device="cuda")
    dk, dv = (t.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3) for t in (pc.dk, pc.dv))
    dk_sf, dv_sf = (t.permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3) for t in (pc.dk_sf, pc.dv_sf))
    _, lse = da.decode_attn(big[:, :, 5:14], dk, dv, pc.dbt, pc.dlens, max_seq_len=70, out=out[:, ::2], k_scale=pc.ks,
                            v_scale=pc.vs, k_sf=dk_sf, v_sf=dv_sf)
    check_attention(pc, q, out[:, ::2], lse, False, 1 / math.sqrt(D))
    assert not bool(out[:, 1::2].any())


def test_fp4_attention_offsets_past_32_bits(da):
    """Pages whose byte offsets exceed 2^32."""
    heads, page = 8, 128
    groups = (1 << 32) // (page * heads * 64) + 40
    k = torch.zeros(groups, page, heads, 64, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    k_sf = torch.zeros(groups, heads, page, 8, dtype=torch.uint8, device="cuda")
    v_sf = torch.zeros_like(k_sf)
    pc = Paged("fp4", [300, 200], heads, page, 88, extra_pages=0)
    n = pc.k.shape[0]
    for big, small in ((k, pc.k), (v, pc.v), (k_sf, pc.k_sf), (v_sf, pc.v_sf)):
        big[groups - n:] = small.cuda()
    bt = (pc.bt + (groups - n)).cuda()
    lens = torch.tensor(pc.lens, dtype=torch.int32, device="cuda")
    q = bf16(gen(89), 2, 1, 16, D)
    out, lse = da.decode_attn(q.cuda(), k, v, bt, lens, max_seq_len=300, k_scale=pc.ks, v_scale=pc.vs, k_sf=k_sf, v_sf=v_sf)
    check_attention(pc, q, out, lse, False, 1 / math.sqrt(D))
    # and the append writes there
    new = bf16(gen(90), 2, 1, heads, D)
    da.rope_append(None, new.cuda(), new.cuda(), None, k, v, bt, lens, max_seq_len=300, k_scale=pc.ks, v_scale=pc.vs,
                   k_sf=k_sf, v_sf=v_sf)
    want, sf = as_cache(new, "fp4", pc.ks)
    pg = int(bt[0, 299 // page])
    assert torch.equal(k[pg, 299 % page].cpu(), want[0, 0]) and torch.equal(k_sf[pg, :, 299 % page].cpu(), sf[0, :, 0])


# ------------------------------------------------------------------ selected pages
def reference_blocks(pc, q, digest, dscale, top_k, sink, local, causal):
    B, T, Hq, _ = q.shape
    G = Hq // pc.heads
    blocks = torch.full((B, T, pc.heads, top_k), -1, dtype=torch.int32)
    for b, n in enumerate(pc.lens):
        for t in range(T):
            seen = max(0, n - T + 1 + t) if causal else n
            count = -(-seen // pc.page)
            at = pc.bt[b, :count].long()
            for h in range(pc.heads):
                s = R.page_scores(q[b, t, h * G:(h + 1) * G], digest[at, h], dscale[at, h])
                p = R.pick(s, top_k, sink, local)
                blocks[b, t, h, :len(p)] = p.to(torch.int32)
    return blocks


def check_sparse(da, kind, page, lens, G, T, top_k, causal, seed, sink=1, local=1, heads=2, tie=False):
    pc = Paged(kind, lens, heads, page, seed).gpu()
    q = bf16(gen(seed + 1), len(lens), T, heads * G, D, std=2.0)
    dg, ds = da.block_digest(pc.dk, pc.dbt, pc.dlens, max_seq_len=pc.max_len, k_sf=pc.dk_sf)
    if tie:  # all pages score alike
        dg[:] = 5
        ds[:] = 0.25
    st = status_word()
    kw = dict(max_seq_len=pc.max_len, top_k=top_k, sink=sink, local=local, causal=causal)
    out, lse, blocks = da.decode_attn_sparse(q.cuda(), pc.dk, pc.dv, pc.dbt, pc.dlens, dg, ds, status=st, **kw, **pc.scales())
    short = causal and any(0 < n < T for n in lens)
    assert int(st.item()) == (da.DA_STATUS_SHORT_CAUSAL if short else 0)
    want = reference_blocks(pc, q, dg.cpu(), ds.cpu(), top_k, sink, local, causal)
    assert torch.equal(blocks.cpu(), want)
    b2, ids, tokens = da.block_select(q.cuda(), dg, ds, pc.dbt, pc.dlens, page_size=page, **kw)
    assert torch.equal(b2, blocks)
    k64, v64 = pc.values("k") * pc.ks, pc.values("v") * pc.vs
    for b, n in enumerate(lens):
        for t in range(T):
            seen = max(0, n - T + 1 + t) if causal else n
            for h in range(heads):
                at = want[b, t, h]
                at = at[at >= 0].long()
                pages = pc.bt[b].long()[at]
                assert torch.equal(ids[b, t, h, :len(at)].cpu().long(), pages)
                m = len(at) * page - (-(-seen // page) * page - seen)
                assert int(tokens[b, t, h]) == m
                kk, vv = (x[pages][:, :, h].flatten(0, 1)[:m] for x in (k64, v64))
                rows = q[b, t, h * G:(h + 1) * G].double()
                o, l, wabs, mag = R.attention_rows(rows, kk, vv, torch.ones(G, m, dtype=torch.bool), 1 / math.sqrt(D))
                got, gl = out[b, t, h * G:(h + 1) * G].cpu().double(), lse[b, t, h * G:(h + 1) * G].cpu().double()
                f = ~l.isinf()
                assert torch.equal(gl.isinf(), l.isinf())
                assert bool(((gl - l).abs() <= R.lse_tolerance(l, mag))[f].all())
                tol = R.bf16_p_tolerance if kind == "bf16" or G > 16 else R.out_tolerance
                assert not bool(((got - o).abs() > tol(o, wabs, mag)).any()), (b, t, h)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("case", [
    # page, lens, G, T, top_k, causal
    (16, [1, 100, 700, 0], 4, 1, 8, False), (16, [513, 2000], 1, 1, 33, False), (48, [1000, 47, 900], 8, 1, 4, True),
    (32, [600, 40, 1], 4, 3, 5, True), (64, [3000], 7, 2, 16, False), (16, [600, 333], 20, 1, 6, False),
    (16, [300, 17], 2, 5, 2, True), (64, [700, 90], 40, 1, 3, False), (16, [333], 100, 1, 9, False)], ids=lambda c: "p%d_g%d_t%d_k%d" % (c[0], c[2], c[3], c[4]))
def test_sparse(da, kind, case):
    check_sparse(da, kind, *case, seed=100 + case[0] + case[2])


def test_sparse_ties_take_the_lower_page(da):
    check_sparse(da, "bf16", 16, [1000, 333], 4, 1, 9, False, 120, tie=True)
    check_sparse(da, "bf16", 16, [1000, 333], 4, 1, 9, False, 121, sink=3, local=4, tie=True)


def test_sparse_forced_pages(da):
    check_sparse(da, "fp4", 16, [1000, 160, 170], 4, 2, 10, True, 122, sink=0, local=10)
    check_sparse(da, "fp4", 16, [1000, 160, 170], 4, 2, 10, True, 123, sink=9, local=1)
    check_sparse(da, "bf16", 16, [40, 17], 4, 1, 1, False, 124, sink=0, local=1)


@pytest.mark.parametrize("pages,top_k", [(2047, 64), (2049, 700), (8192, 1), (8193, 64), (20011, 4096)])
def test_select_many_pages(da, pages, top_k):
    """The selection alone, over counts on both sides of its kernels' limits; repeated
    digests give many equal scores."""
    g = gen(pages)
    heads, G, T = 2, 3, 2
    kinds = 37
    dg = torch.randint(-127, 128, (kinds, heads, 2, D), generator=g).to(torch.int8)
    ds = torch.rand(kinds, heads, generator=g)
    bt = torch.randint(0, kinds, (2, pages), generator=g).to(torch.int32)
    q = bf16(g, 2, T, heads * G, D)
    lens = [pages * 16 - 3, pages * 8]
    class Fake:
        pass
    pc = Fake()
    pc.lens, pc.page, pc.bt, pc.heads = lens, 16, bt, heads
    want = reference_blocks(pc, q, dg, ds, top_k, 1 if top_k > 1 else 0, 1, True)
    blocks, ids, tokens = da.block_select(q.cuda(), dg.cuda(), ds.cuda(), bt.cuda(),
                                          torch.tensor(lens, dtype=torch.int32).cuda(), page_size=16,
                                          max_seq_len=pages * 16, top_k=top_k, sink=1 if top_k > 1 else 0, causal=True)
    assert torch.equal(blocks.cpu(), want)


def test_select_special_queries(da):
    """NaN, infinities, zeros and huge scales in q and digests."""
    g = gen(9)
    pages, heads = 300, 1
    dg = torch.randint(-127, 128, (pages, heads, 2, D), generator=g).to(torch.int8)
    ds = torch.rand(pages, heads, generator=g)
    ds[5], ds[6], ds[7] = 2.6e36, 0.0, 1e-40
    q = bf16(g, 6, 1, 2, D)
    q[1, 0, 0, 3] = math.nan
    q[2, 0, 1, 3] = math.inf
    q[2, 0, 1, 4] = -math.inf
    q[3] = 0
    q[4] = math.nan
    q[5] = q[5] * 1e-38
    class Fake:
        pass
    pc = Fake()
    pc.lens, pc.page, pc.heads = [pages * 16] * 6, 16, heads
    pc.bt = torch.stack([torch.randperm(pages, generator=g) for _ in range(6)]).to(torch.int32)
    want = reference_blocks(pc, q, dg, ds, 20, 1, 1, False)
    blocks, _, _ = da.block_select(q.cuda(), dg.cuda(), ds.cuda(), pc.bt.cuda(),
                                   torch.tensor(pc.lens, dtype=torch.int32).cuda(), page_size=16, max_seq_len=pages * 16,
                                   top_k=20)
    assert torch.equal(blocks.cpu(), want)


def test_select_bad_pages_and_lengths(da):
    pc = Paged("bf16", [400, 300], 2, 16, 130).gpu()
    q = bf16(gen(131), 2, 1, 4, D).cuda()
    dg, ds = da.block_digest(pc.dk, pc.dbt, pc.dlens, max_seq_len=400)
    pc.dbt[0, :] = 10 ** 6
    pc.dlens[1] = 500
    st = status_word()
    out, lse, blocks = da.decode_attn_sparse(q, pc.dk, pc.dv, pc.dbt, pc.dlens, dg, ds, max_seq_len=400, top_k=5, status=st)
    assert int(st.item()) == da.DA_STATUS_BAD_PAGE | da.DA_STATUS_SEQ_LEN
    assert not bool(out.isnan().any())


def test_sparse_of_all_pages_is_dense_attention(da):
    for kind in ("bf16", "fp8", "fp4"):
        pc = Paged(kind, [300, 77, 160], 2, 16, 140).gpu()
        q = bf16(gen(141), 3, 1, 8, D).cuda()
        dg, ds = da.block_digest(pc.dk, pc.dbt, pc.dlens, max_seq_len=300, k_sf=pc.dk_sf)
        out, lse, blocks = da.decode_attn_sparse(q, pc.dk, pc.dv, pc.dbt, pc.dlens, dg, ds, max_seq_len=300, top_k=19,
                                                 **pc.scales())
        check_attention(pc, q.cpu(), out, lse, False, 1 / math.sqrt(D),
                        R.bf16_p_tolerance if kind == "bf16" else R.out_tolerance)


# ------------------------------------------------------------------ a decode step of all of them
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_decode_steps_captured_in_a_graph(da, kind):
    """Append, digest, dense and sparse attention, captured once and replayed over
    steps whose lengths grow in device memory; every step against the reference."""
    page, heads, G, start = 16, 2, 4, [30, 100, 15]
    steps = 4
    pc = Paged(kind, [n + steps for n in start], heads, page, 150).gpu()
    f, amp = da.rope_frequencies(64, base=50000.0, scaling="by_parts", factor=4.0, original_positions=64)
    table = da.rope_table(f.cuda(), 200, amplitude=amp)
    g = gen(151)
    new = [bf16(g, 3, 1, heads * (G + 2), D, std=1.5) for _ in range(steps)]
    qkv = new[0].cuda()
    q_in, k_in, v_in = qkv[:, :, :heads * G], qkv[:, :, heads * G:heads * (G + 1)], qkv[:, :, heads * (G + 1):]
    lens = torch.tensor(start, dtype=torch.int32, device="cuda")
    dg, ds = da.block_digest(pc.dk, pc.dbt, lens, max_seq_len=pc.max_len, k_sf=pc.dk_sf)
    q = torch.zeros(3, 1, heads * G, D, dtype=torch.bfloat16, device="cuda")
    res = {}

    def step():
        lens.add_(1)
        da.rope_append(q_in, k_in, v_in, table, pc.dk, pc.dv, pc.dbt, lens, max_seq_len=pc.max_len, q_out=q, **pc.scales())
        da.block_digest(pc.dk, pc.dbt, lens, dg, ds, max_seq_len=pc.max_len, max_new=1, k_sf=pc.dk_sf)
        res["dense"] = da.decode_attn(q, pc.dk, pc.dv, pc.dbt, lens, max_seq_len=pc.max_len, **pc.scales())
        res["sparse"] = da.decode_attn_sparse(q, pc.dk, pc.dv, pc.dbt, lens, dg, ds, max_seq_len=pc.max_len, top_k=4,
                                              **pc.scales())

    saved = [t.clone() for t in (pc.dk, pc.dv, lens, dg, ds)] + [None if t is None else t.clone() for t in (pc.dk_sf, pc.dv_sf)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()  # (the first call sets kernel attributes)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, s in zip((pc.dk, pc.dv, lens, dg, ds, pc.dk_sf, pc.dv_sf), saved):
        if t is not None:
            t.copy_(s)
    tab = table.cpu()
    for i in range(steps):
        qkv.copy_(new[i])
        graph.replay()
        torch.cuda.synchronize()
        pc.lens = [n + i + 1 for n in start]
        assert lens.tolist() == pc.lens
        want, _ = append_reference(pc, None, new[i][:, :, heads * G:heads * (G + 1)], new[i][:, :, heads * (G + 1):], tab,
                                   1, None, None, False)
        for name, got in (("k", pc.dk), ("v", pc.dv), ("k_sf", pc.dk_sf), ("v_sf", pc.dv_sf)):
            if got is not None:
                assert torch.equal(got.cpu(), want[name]), name
                setattr(pc, name, want[name])
        x = pc.values("k").float()
        for b, n in enumerate(pc.lens):
            for c in range(-(-n // page)):
                pg = int(pc.bt[b, c])
                for h in range(heads):
                    d, s = R.digest_page(x[pg, :min(page, n - c * page), h])
                    assert torch.equal(dg[pg, h].cpu(), d) and float(ds[pg, h]) == float(s)
        tol = R.bf16_p_tolerance if kind == "bf16" else R.out_tolerance
        check_attention(pc, q.cpu(), *res["dense"], False, 1 / math.sqrt(D), tol)
        blocks = reference_blocks(pc, q.cpu(), dg.cpu(), ds.cpu(), 4, 1, 1, False)
        assert torch.equal(res["sparse"][2].cpu(), blocks)


def test_two_streams_and_repeats_give_the_same_bits(da):
    pc = Paged("fp4", [3000, 1500, 700], 4, 16, 160).gpu()
    q = bf16(gen(161), 3, 1, 16, D).cuda()
    dg, ds = da.block_digest(pc.dk, pc.dbt, pc.dlens, max_seq_len=3000, k_sf=pc.dk_sf)
    want = da.decode_attn(q, pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=3000, **pc.scales())
    want_s = da.decode_attn_sparse(q, pc.dk, pc.dv, pc.dbt, pc.dlens, dg, ds, max_seq_len=3000, top_k=20, **pc.scales())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(da.decode_attn(q, pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=3000, **pc.scales()))
                got.append(da.decode_attn_sparse(q, pc.dk, pc.dv, pc.dbt, pc.dlens, dg, ds, max_seq_len=3000, top_k=20,
                                                 **pc.scales()))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want if len(g) == 2 else want_s):
            assert torch.equal(a, b)


def test_empty_batches(da):
    k = torch.zeros(4, 16, 2, 64, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(4, 2, 16, 8, dtype=torch.uint8, device="cuda")
    bt = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    lens = torch.zeros(0, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 1, 4, D, dtype=torch.bfloat16, device="cuda")
    out, lse = da.decode_attn(q, k, k, bt, lens, max_seq_len=32, k_sf=sf, v_sf=sf)
    assert out.shape == q.shape
    new = torch.zeros(0, 1, 2, D, dtype=torch.bfloat16, device="cuda")
    da.rope_append(q, new, new, None, k, k.clone(), bt, lens, max_seq_len=32, k_sf=sf, v_sf=sf.clone())
    dg, ds = da.block_digest(k, bt, lens, max_seq_len=32, k_sf=sf)
    out, lse, blocks = da.decode_attn_sparse(q, k, k, bt, lens, dg, ds, max_seq_len=32, top_k=2, k_sf=sf, v_sf=sf)
    assert blocks.shape == (0, 1, 2, 2)


def test_calls_on_a_stream_that_is_not_the_current_one(da):
    """What a call allocates and clears is ordered with the call's stream, however
    busy the current one is."""
    pc = Paged("fp4", [900, 450, 33], 4, 16, 162).gpu()
    q, new = bf16(gen(163), 3, 1, 16, D).cuda(), bf16(gen(164), 3, 1, 4, D).cuda()
    f = da.rope_frequencies(D)[0].cuda()
    kw = dict(max_seq_len=900)

    def run(stream):
        tab = da.rope_table(f, 1000, stream=stream)
        turned = da.rope_append(q, new, new, tab, pc.dk, pc.dv, pc.dbt, pc.dlens, stream=stream, **kw, **pc.scales())
        dg, ds = da.block_digest(pc.dk, pc.dbt, pc.dlens, k_sf=pc.dk_sf, stream=stream, **kw)
        dense = da.decode_attn(turned, pc.dk, pc.dv, pc.dbt, pc.dlens, stream=stream, **kw, **pc.scales())
        some = da.decode_attn_sparse(turned, pc.dk, pc.dv, pc.dbt, pc.dlens, dg, ds, top_k=5, stream=stream, **kw,
                                     **pc.scales())
        picked = da.block_select(turned, dg, ds, pc.dbt, pc.dlens, page_size=16, top_k=5, stream=stream, **kw)
        return [tab, turned, dg, ds, *dense, *some, picked[0], picked[2]]

    want = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        before = torch.cuda.current_stream()
        torch.cuda._sleep(100_000_000)
        got = run(stream)
        assert torch.cuda.current_stream() == before
        side.synchronize()
        with torch.cuda.stream(side):
            copies = [t.clone() for t in got]
        side.synchronize()
        torch.cuda.synchronize()
        for a, b, c in zip(want, copies, got):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_two_graphs_that_share_a_workspace(da):
    """Captured calls leave nothing in a workspace that another call needs."""
    pc = longer(Paged("fp4", [3000, 1500, 700], 4, 16, 165), 8192).gpu()
    q = bf16(gen(166), 3, 1, 16, D).cuda()
    dg, ds = da.block_digest(pc.dk, pc.dbt, pc.dlens, max_seq_len=8192, k_sf=pc.dk_sf)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    kw = dict(max_seq_len=8192, workspace=ws)

    def dense():
        return da.decode_attn(q, pc.dk, pc.dv, pc.dbt, pc.dlens, **kw, **pc.scales())

    def some():
        return da.decode_attn_sparse(q, pc.dk, pc.dv, pc.dbt, pc.dlens, dg, ds, top_k=20, **kw, **pc.scales())

    want = [[t.clone() for t in f()] for f in (dense, some)]
    graphs, outs = [], []
    for f in (dense, some):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for t in (*outs[0], *outs[1]):
            t.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in order:
            for a, b in zip(outs[i], want[i]):
                assert torch.equal(a, b)
    # lengths that change between replays
    pc.lens = [2999, 1, 0]
    pc.dlens.copy_(torch.tensor(pc.lens, dtype=torch.int32))
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    check_attention(pc, q.cpu(), *outs[0], False, 1 / math.sqrt(D))
    assert torch.equal(outs[1][2].cpu(), reference_blocks(pc, q.cpu(), dg.cpu(), ds.cpu(), 20, 1, 1, False))


def test_sparse_into_given_tensors(da):
    pc = Paged("bf16", [900, 450], 2, 16, 167).gpu()
    q = bf16(gen(168), 2, 2, 8, D).cuda()
    dg, ds = da.block_digest(pc.dk, pc.dbt, pc.dlens, max_seq_len=900)
    kw = dict(max_seq_len=900, top_k=7, causal=True)
    want = da.decode_attn_sparse(q, pc.dk, pc.dv, pc.dbt, pc.dlens, dg, ds, **kw)
    wide = torch.zeros(2, 2, 12, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(2, 2, 8, device="cuda")
    blocks = torch.zeros(2, 2, 2, 7, dtype=torch.int32, device="cuda")
    ws = torch.full((1 << 22,), 0xFF, dtype=torch.uint8, device="cuda")
    got = da.decode_attn_sparse(q, pc.dk, pc.dv, pc.dbt, pc.dlens, dg, ds, out=wide[:, :, 2:10], lse=lse, blocks=blocks,
                                workspace=ws, **kw)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert got[2].data_ptr() == blocks.data_ptr() and bool((ws != 0xFF).any())
    assert not bool(wide[:, :, :2].any()) and not bool(wide[:, :, 10:].any())
