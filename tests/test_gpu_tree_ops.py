"""GPU parity of trees of drafted tokens (masks, attention, kept tokens), cross
attention, and reading a cache back, against plain 64-bit references on the CPU."""
import math
import random

import pytest

torch = pytest.importorskip("torch")
from tests import cache_ref as R
from tests.strict import assert_attention, assert_within
from tests.test_gpu_cache_ops import D, SCALES, Paged, as_cache, bf16, gen, status_word

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


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def random_parents(T, seed):
    r = random.Random(seed)
    return [-1] + [-1 if r.random() < 0.05 else r.randint(max(0, t - 8), t - 1) for t in range(1, T)]


def ways(parents):
    """bool [T, T]: token i is t or on its path."""
    T = len(parents)
    out = torch.zeros(T, T, dtype=torch.bool)
    for t, p in enumerate(parents):
        if p >= 0:
            out[t] = out[p]
        out[t, t] = True
    return out


def pack(seen):
    """bool [.., T, T] -> int32 [.., T, ceil(T / 32)]."""
    T = seen.shape[-1]
    x = torch.nn.functional.pad(seen, (0, -T % 32)).unflatten(-1, (-1, 32)).long()
    w = (x << torch.arange(32)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def tolerance_for(kind, G, T):
    """P is rounded to bf16 over bf16 caches, and over others that are read back first (from 3 pairs of tiles of 128 // G
    tokens on, 4-bit ones from 2); to f16 over the others."""
    pairs = -(-T // (2 * (128 // G))) if G * T > 128 else 0
    return R.bf16_p_tolerance if kind == "bf16" or pairs >= (2 if kind == "fp4" else 3) else R.out_tolerance


def check_rows(c, q, out, lse, own, seen_new, scale=SCALE, lost=0.0):
    """Every request's rows of out / lse against 64 bits; seen_new[b] bool [own, own] or None.  lost: an absolute error
    that outputs may have besides."""
    B, T, Hq, _ = q.shape
    G = Hq // c.heads
    base = tolerance_for(c.kind, G, T)
    tol = (lambda o, wabs, mag: base(o, wabs, mag) + lost) if lost else base
    kv, vv = (c.values(w) * s for w, s in (("k", c.ks), ("v", c.vs)))
    out, lse = out.double().cpu(), lse.double().cpu()
    for b, n in enumerate(c.lens):
        m = own[b]
        if m < T:
            assert bool((out[b, m:] == 0).all()) and bool((lse[b, m:] == -math.inf).all())
        k, v = R.gather(kv, c.bt, b, n), R.gather(vv, c.bt, b, n)
        seen = torch.ones(m, n, dtype=torch.bool)
        if seen_new is not None and m > 0:
            new = seen_new[b][:m, :m]
            have = min(m, n)                       # new tokens that have a key
            seen[:, n - have:] = new[:, m - have:]
        for h in range(c.heads):
            rows = q[b, :m, h * G:(h + 1) * G].double().reshape(-1, D)
            assert_attention(out[b, :m, h * G:(h + 1) * G].reshape(-1, D), lse[b, :m, h * G:(h + 1) * G].reshape(-1), rows,
                             k[:, h], v[:, h], seen.repeat_interleave(G, 0), scale, tol, (b, h))


# ------------------------------------------------------------------ masks
@pytest.mark.parametrize("batch,T", [(1, 1), (1, 2), (3, 16), (2, 31), (2, 32), (5, 33), (2, 63), (300, 64), (1, 127),
                                     (2, 128), (3, 129), (1, 1023), (2, 1024)])
def test_tree_masks(da, batch, T):
    r = random.Random(T)
    own = [r.randint(0, T) for _ in range(batch)]
    own[0] = T
    parents = [random_parents(T, 7 * T + b) for b in range(batch)]
    if T == 1024:
        parents[1] = list(range(-1, T - 1))  # one chain
        own[1] = T
    lens = [n + r.randint(0, 5000) for n in own]
    status = status_word()
    mask, pos = da.tree_mask(ints(parents), ints(lens), max_seq_len=10000, new_lens=ints(own), status=status)
    assert mask.shape == (batch, T, -(-T // 32)) and mask.dtype == torch.int32
    for b in range(batch):
        w = ways(parents[b])
        w[own[b]:] = False
        assert torch.equal(mask[b].cpu(), pack(w))
        want = torch.where(torch.arange(T) < own[b], lens[b] - own[b] + w.sum(1) - 1, 0).to(torch.int32)
        assert torch.equal(pos[b].cpu(), want)
    assert int(status) == 0
    if own == [T] * batch:
        other, _ = da.tree_mask(ints(parents), ints(lens), max_seq_len=10000)
        assert torch.equal(other, mask)


def test_tree_mask_of_bad_parents_and_lengths(da):
    """A parent that is no earlier token counts as -1; lengths are clamped; each sets its bit."""
    for parents, lens, own, bits in [([[-1, 1, 0, 1]], [9], [4], 32), ([[-1, -2, 0, 7]], [9], [4], 32),
                                     ([[0, 0, 1, 2]], [9], [4], 32), ([[-1, 0, 1, 2]], [11], [4], 2),
                                     ([[-1, 0, 1, 2]], [9], [5], 2), ([[-1, 0, 1, 2]], [9], [-1], 2),
                                     ([[-1, 0, 1, 2]], [3], [4], 4), ([[-1, 0, 9, 9]], [9], [2], 0)]:
        status = status_word()
        mask, pos = da.tree_mask(ints(parents), ints(lens), max_seq_len=10, new_lens=ints(own), status=status)
        assert int(status) == bits, (parents, lens, own)
        n, L = min(max(own[0], 0), 4), min(lens[0], 10)
        good = [p if -1 <= p < t else -1 for t, p in enumerate(parents[0])]
        w = ways(good)
        w[n:] = False
        assert torch.equal(mask[0].cpu(), pack(w))
        want = torch.where(torch.arange(4) < n, L - n + w.sum(1) - 1, 0).to(torch.int32)
        assert torch.equal(pos[0].cpu(), want)


# ------------------------------------------------------------------ attention of trees
TREES = [
    # lens, heads, group, T, page, own (None: all T)
    ([40], 1, 1, 1, 16, None),
    ([1], 2, 4, 1, 16, None),
    ([5, 300], 2, 1, 5, 0, None),
    ([4, 17, 100, 611], 2, 4, 4, 16, [4, 1, 0, 3]),
    ([129, 16, 33], 1, 5, 3, 48, [2, 3, 1]),
    ([700, 65, 7], 2, 4, 7, 16, [7, 5, 7]),             # 28 rows
    ([900, 0, 64, 250], 2, 4, 16, 32, [16, 0, 9, 16]),  # 64 rows
    ([333, 36], 1, 1, 33, 16, [33, 20]),                # 33 rows, two words
    ([500, 128, 2000], 2, 4, 32, 16, [32, 17, 32]),     # 128 rows
    ([400, 70], 1, 2, 64, 64, None),                    # 128 rows, two words
    ([300, 129], 1, 1, 128, 0, [128, 100]),             # four words
    ([260, 33], 2, 4, 33, 16, [33, 20]),                # 132 rows
    ([1300, 64, 700], 2, 8, 32, 48, [32, 9, 20]),       # 256 rows
    ([900, 400], 1, 5, 63, 128, [63, 40]),              # 315 rows
    ([700], 1, 7, 100, 0, None),                        # 700 rows
    ([1100, 1050], 1, 1, 1024, 16, [1024, 333]),
]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("case", range(len(TREES)))
def test_tree_attention(da, kind, case):
    lens, heads, G, T, page, own = TREES[case]
    c = Paged(kind, lens, heads, page, 100 + case).gpu()
    q = bf16(gen(case), len(lens), T, heads * G, D, std=2.0)
    seen = [ways(random_parents(T, 31 * case + b)) for b in range(len(lens))]
    mask = pack(torch.stack(seen)).cuda()
    status = status_word()
    n = own if own is not None else [T] * len(lens)
    for splits in (0, 1, 3):
        out, lse = da.decode_attn_tree(q.cuda(), c.dk, c.dv, c.dbt, c.dlens, mask, max_seq_len=c.max_len, num_splits=splits,
                                       new_lens=None if own is None else ints(own), status=status, **c.scales())
        check_rows(c, q, out, lse, n, seen)
    assert int(status) == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("heads,G,T", [(2, 4, 4), (1, 4, 8), (1, 1, 40), (1, 4, 32), (1, 4, 50)])
def test_any_bits_and_one_mask_for_all(da, kind, heads, G, T):
    """Rows of arbitrary bits, some empty, the same rows for all requests; requests without a key before the tree."""
    g = gen(T)
    lens = [T + 400, T, T + 1, T + 130]
    c = Paged(kind, lens, heads, 16, 9 + T).gpu()
    q = bf16(g, len(lens), T, heads * G, D, std=2.0)
    seen = torch.rand(T, T, generator=g) < 0.3
    seen[::3] = False
    out, lse = da.decode_attn_tree(q.cuda(), c.dk, c.dv, c.dbt, c.dlens, pack(seen)[None].cuda(), max_seq_len=c.max_len, **c.scales())
    check_rows(c, q, out, lse, [T] * 4, [seen] * 4)
    every = pack(seen).expand(4, -1, -1).contiguous().cuda()
    again, lse2 = da.decode_attn_tree(q.cuda(), c.dk, c.dv, c.dbt, c.dlens, every, max_seq_len=c.max_len, **c.scales())
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    assert bool((lse[1, ::3] == -math.inf).all())  # (nothing before the tree, no bit set)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("G,T", [(4, 4), (4, 16), (4, 32), (4, 40)])
def test_a_chain_is_the_causal_mask(da, kind, G, T):
    """A tree with one path gives what the causal mask gives (up to 128 rows: the same bits)."""
    lens = [500, T, 77 + T]
    c = Paged(kind, lens, 2, 16, 5).gpu()
    q = bf16(gen(T), 3, T, 2 * G, D, std=2.0).cuda()
    mask, _ = da.tree_mask(ints([list(range(-1, T - 1))] * 3), c.dlens, max_seq_len=c.max_len)
    out, lse = da.decode_attn_tree(q, c.dk, c.dv, c.dbt, c.dlens, mask, max_seq_len=c.max_len, num_splits=2, **c.scales())
    if G * T <= 128:
        want, wlse = da.decode_attn(q, c.dk, c.dv, c.dbt, c.dlens, max_seq_len=c.max_len, causal=True, num_splits=2, **c.scales())
        assert torch.equal(out, want) and torch.equal(lse, wlse)
    else:
        check_rows(c, q.cpu(), out, lse, [T] * 3, [torch.ones(T, T).tril().bool()] * 3)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("G,T", [(4, 4), (4, 16), (4, 32), (4, 40)])
def test_hidden_keys_padding_and_stale_slots_may_hold_nan(da, kind, G, T):
    """NaN in hidden keys, in slots behind the sequence and in padding rows of q reaches no other row."""
    lens, own = [300, 133, T], [T, T - 2, T - 1]
    c = Paged(kind, lens, 2, 16, 3).gpu()
    q = bf16(gen(1), 3, T, 2 * G, D, std=2.0)
    seen = torch.zeros(T, T, dtype=torch.bool)
    seen[:, 0] = True
    seen[:, 1] = True                              # token 2, which holds NaN, is seen by token 2 alone
    seen[2, 2] = True
    mask = pack(seen)[None].cuda()
    nan = 0x7f if kind == "fp8" else float("nan")
    for b in range(3):
        for x in (c.k, c.dk):
            j = lens[b] - own[b] + 2
            x[int(c.bt[b, j // 16]), j % 16] = nan
        for j in range(lens[b], -(-lens[b] // 16) * 16):
            for x in (c.dk, c.dv):
                x[int(c.bt[b, j // 16]), j % 16] = nan
    q[1, own[1]:] = float("nan")
    q[2, own[2]:] = float("inf")
    out, lse = da.decode_attn_tree(q.cuda(), c.dk, c.dv, c.dbt, c.dlens, mask, max_seq_len=c.max_len, new_lens=ints(own), **c.scales())
    for b in range(3):
        if own[b] > 2:
            assert bool(out[b, 2].isnan().all()) and bool(lse[b, 2].isnan().all())
    keep = [t for t in range(T) if t != 2]
    c.k = torch.where(c.k == nan, 0, c.k) if kind == "fp8" else torch.nan_to_num(c.k, nan=0.0)
    G_rows = q[:, keep]
    out, lse = out[:, keep], lse[:, keep]
    kv, vv = (c.values(w) * s for w, s in (("k", c.ks), ("v", c.vs)))
    for b, n in enumerate(lens):
        m = own[b] - 1 if own[b] > 2 else own[b]
        assert bool((out[b, m:] == 0).all()) and bool((lse[b, m:] == -math.inf).all())
        k, v = R.gather(kv, c.bt, b, n), R.gather(vv, c.bt, b, n)
        see = torch.ones(m, n, dtype=torch.bool)
        see[:, n - own[b]:] = seen[keep][:m, :own[b]]
        for h in range(2):
            rows = G_rows[b, :m, h * G:(h + 1) * G].double().reshape(-1, D)
            assert_attention(out[b, :m, h * G:(h + 1) * G].double().cpu().reshape(-1, D),
                             lse[b, :m, h * G:(h + 1) * G].double().cpu().reshape(-1), rows, k[:, h], v[:, h],
                             see.repeat_interleave(G, 0), SCALE, tolerance_for(kind, G, T), (b, h))


@pytest.mark.parametrize("G,T", [(4, 4), (2, 16), (4, 40)])
@pytest.mark.parametrize("scale", [0.0, -0.07, 1.0])
def test_scales_of_any_sign(da, G, T, scale):
    c = Paged("bf16", [300, 200], 1, 16, 4).gpu()
    q = bf16(gen(2), 2, T, G, D, std=0.5)
    seen = [ways(random_parents(T, b)) for b in range(2)]
    out, lse = da.decode_attn_tree(q.cuda(), c.dk, c.dv, c.dbt, c.dlens, pack(torch.stack(seen)).cuda(), max_seq_len=c.max_len, scale=scale)
    check_rows(c, q, out, lse, [T, T], seen, scale=scale)


@pytest.mark.parametrize("G,T", [(4, 4), (4, 16), (4, 40)])
def test_tree_status_bits(da, G, T):
    """Out-of-range lengths and pages are clamped and reported; a tree longer than its sequence sees what there is."""
    c = Paged("bf16", [100, 50, T - 2], 1, 16, 8).gpu()
    q = bf16(gen(3), 3, T, G, D)
    seen = [ways(random_parents(T, b)) for b in range(3)]
    mask = pack(torch.stack(seen)).cuda()

    def run(**kw):
        status = status_word()
        a = dict(lens=c.dlens, own=None, bt=c.dbt)
        a.update(kw)
        out, lse = da.decode_attn_tree(q.cuda(), c.dk, c.dv, a["bt"], a["lens"], mask, max_seq_len=c.max_len, new_lens=a["own"], status=status)
        return out, lse, int(status)

    out, lse, bits = run()
    assert bits == 4
    check_rows(c, q, out, lse, [T] * 3, seen)
    assert run(own=ints([T, T + 1, 0]))[2] == 2
    assert run(own=ints([T, -1, 0]))[2] == 2
    assert run(own=ints([T, T, 0]), lens=ints([101, 50, 0]))[2] == 2
    bad = c.dbt.clone()
    bad[0, 1] = 1000
    assert run(own=ints([T, T, 0]), bt=bad)[2] == 1


# ------------------------------------------------------------------ cross attention
CROSS = [
    # lens, heads, group, T, page, own
    ([1500, 30, 1], 2, 1, 1, 0, None),
    ([200, 0, 77], 2, 8, 1, 16, None),
    ([17, 300], 1, 4, 4, 16, [4, 2]),
    ([90, 130, 16], 2, 2, 20, 32, [20, 0, 13]),
    ([128, 129, 127, 1], 1, 1, 129, 16, [129, 128, 0, 1]),
    ([300, 5], 2, 1, 257, 0, [257, 100]),
    ([1000, 640, 0], 1, 3, 100, 48, [100, 43, 100]),
    ([513, 64], 1, 8, 70, 128, [70, 33]),
    ([2100], 1, 1, 1000, 64, None),
    ([40, 400], 5, 4, 64, 16, None),
]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("case", range(len(CROSS)))
def test_cross_attention(da, kind, case):
    lens, heads, G, T, page, own = CROSS[case]
    c = Paged(kind, lens, heads, page, 200 + case).gpu()
    q = bf16(gen(50 + case), len(lens), T, heads * G, D, std=2.0)
    status = status_word()
    for splits in (0, 1, 4):
        out, lse = da.cross_attn(q.cuda(), c.dk, c.dv, c.dbt, c.dlens, max_seq_len=c.max_len, num_splits=splits,
                                 q_lens=None if own is None else ints(own), status=status, **c.scales())
        check_rows(c, q, out, lse, own if own is not None else [T] * len(lens), None)
    assert int(status) == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("T", [1, 9, 150])
def test_cross_attention_into_strided_outputs_on_another_stream(da, kind, T):
    """q and out are views of wider tensors; what lies between stays; a stream of one's own; a workspace full of NaN."""
    lens = [300, 40]
    c = Paged(kind, lens, 2, 16, 6).gpu()
    q = bf16(gen(7), 2, T, 3, 4, D, std=2.0)
    wide = torch.full((2, T, 3, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((1 << 22,), float("nan"), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse = da.cross_attn(q.cuda()[:, :, 1], c.dk, c.dv, c.dbt, c.dlens, max_seq_len=c.max_len, out=wide[:, :, 1], workspace=ws, **c.scales())
    again, lse2 = da.cross_attn(q.cuda()[:, :, 1], c.dk, c.dv, c.dbt, c.dlens, max_seq_len=c.max_len, stream=s, **c.scales())
    torch.cuda.synchronize()
    assert bool((wide[:, :, 0] == 7).all()) and bool((wide[:, :, 2] == 7).all())
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    check_rows(c, q[:, :, 1], out, lse, [T] * 2, None)


def test_many_rows_without_a_key(da):
    """max_seq_len 0, and caches with no token at all."""
    k = torch.zeros(2, 16, 1, D, dtype=torch.bfloat16, device="cuda")
    for T in (3, 200):
        q = bf16(gen(1), 2, T, 1, D).cuda()
        out, lse = da.cross_attn(q, k, k, None, ints([0, 0]), max_seq_len=0)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())
        out, lse = da.cross_attn(q, k, k, None, ints([0, 0]), max_seq_len=16)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_one_value_dominates(da):
    """A row whose weight lies on one key returns that key's value, whatever the rows around it (300 rows)."""
    T = 300
    c = Paged("bf16", [260], 1, 16, 2).gpu()
    at = [(7 * t) % 260 for t in range(T)]
    k = R.gather(c.k, c.bt, 0, 260)[:, 0]
    q = (k[at].float() * 40).to(torch.bfloat16)[None, :, None]
    out, _ = da.cross_attn(q.cuda(), c.dk, c.dv, c.dbt, c.dlens, max_seq_len=c.max_len)
    v = R.gather(c.v, c.bt, 0, 260)[:, 0]
    assert torch.equal(out[0, :, 0].cpu(), v[at])


# ------------------------------------------------------------------ kept tokens
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("page", [0, 16, 48])
@pytest.mark.parametrize("heads,T", [(1, 1), (2, 8), (8, 32), (3, 100), (1, 1024)])
def test_kept_tokens(da, kind, page, heads, T):
    r = random.Random(heads * T + page)
    own = [T, max(1, T // 2), T, T, 0]
    lens = [T, T + 17, T + 100, T + 31, 5]
    c = Paged(kind, lens, heads, page, 11).gpu()
    M = max(1, T - T // 4)
    keep, counts = [], []
    for n in own:
        m = r.randint(0, min(n, M)) if keep else min(n, M)
        path = sorted(r.sample(range(n), m))
        keep.append(path + [r.randint(-5, 2000) for _ in range(M - m)])
        counts.append(m)
    before = {w: getattr(c, w).clone() for w in ("k", "v", "k_sf", "v_sf") if getattr(c, w) is not None}
    status = status_word()
    got = da.cache_keep(c.dk, c.dv, c.dbt, c.dlens, ints(keep), ints(counts), new_tokens=T, max_seq_len=c.max_len,
                        new_lens=ints(own), k_sf=c.dk_sf, v_sf=c.dv_sf, status=status)
    assert got.tolist() == [n - o + m for n, o, m in zip(lens, own, counts)]
    for w, x in before.items():
        want = x.clone()
        for b, path in enumerate(keep):
            for i, p in enumerate(path[:counts[b]]):
                at = []
                for j in (lens[b] - own[b] + i, lens[b] - own[b] + p):
                    at.append((int(c.bt[b, j // page]), j % page) if page else (b, j))
                (gd, sd), (gs, ss) = at
                if w.endswith("sf"):
                    want[gd, :, sd] = x[gs, :, ss]
                else:
                    want[gd, sd] = x[gs, ss]
        assert torch.equal(getattr(c, "d" + w).cpu().view(torch.uint8), want.view(torch.uint8)), w
    assert int(status) == 0


def test_kept_tokens_that_do_not_rise_are_dropped(da):
    c = Paged("bf16", [40], 1, 16, 1).gpu()

    def run(keep, count, lens=40, own=8, bt=None):
        k = c.k.cuda()
        v = c.v.cuda()
        status = status_word()
        got = da.cache_keep(k, v, c.dbt if bt is None else bt, ints([lens]), ints([keep]), ints([count]), new_tokens=8,
                            max_seq_len=c.max_len, new_lens=ints([own]), status=status)
        moved = R.gather(k.cpu(), c.bt, 0, 40)[32:40, 0]
        return int(got), int(status), moved

    old = R.gather(c.k, c.bt, 0, 40)[32:40, 0]
    for keep, count, m, bits in [([1, 3, 3, 5], 4, 2, 32), ([1, 0, 2, 3], 4, 1, 32), ([8, 9, 9, 9], 4, 0, 32), ([-1, 2, 3, 4], 3, 0, 32),
                                 ([2, 3, 4, 5], 5, 4, 32), ([2, 3, 4, 5], -1, 0, 32), ([2, 5, 6, 7], 3, 3, 0)]:
        n, status, moved = run(keep, count)
        assert (n, status) == (32 + m, bits), keep
        want = old.clone()
        want[:m] = old[keep[:m]]
        assert torch.equal(moved, want)
    bad = c.dbt.clone()
    bad[0, 2] = -1
    n, status, moved = run([1, 2, 3, 4], 4, bt=bad)  # (all new tokens lie in the bad page)
    assert (n, status) == (36, 1) and torch.equal(moved, old)
    assert run([0, 1, 2, 3], 2, lens=41)[1] == 2
    assert run([0, 1, 2, 3], 2, own=9)[1] == 2
    n, status, moved = run([1, 2, 3, 4], 4, lens=3, own=8)  # tokens before position 0
    assert (n, status) == (0, 4)


# ------------------------------------------------------------------ read back
def read_reference(c, b, n, start):
    """fp32 products with the cache's scale, rounded to bf16: [n - start, heads, 128]."""
    got = []
    for w, s in (("k", c.ks), ("v", c.vs)):
        x = R.gather(c.values(w), c.bt, b, n)[start:]
        got.append((x.float() * R.f32(s)).to(torch.bfloat16))
    return got


def same_bits(x, y):
    return torch.equal(x.cpu().contiguous().view(torch.int16), y.cpu().contiguous().view(torch.int16))


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("lens,heads,page", [([1], 1, 16), ([100, 0, 33, 500], 2, 16), ([257, 64], 3, 0), ([70, 200], 8, 48),
                                             ([40, 31], 20, 128), ([129], 1, 64)])
def test_read_back(da, kind, lens, heads, page):
    c = Paged(kind, lens, heads, page, 21).gpu()
    status = status_word()
    k, v = da.cache_read(c.dk, c.dv, c.dbt, c.dlens, max_seq_len=c.max_len, status=status, **c.scales())
    assert k.shape == (len(lens), c.max_len, heads, D)
    starts = [n // 3 for n in lens]
    kept = [n - s for n, s in zip(lens, starts)]
    offsets = [sum(kept[:b]) + b for b in range(len(lens))]  # (a row between two requests)
    kp, vp = (torch.full((sum(kept) + len(lens), heads, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    da.cache_read(c.dk, c.dv, c.dbt, c.dlens, max_seq_len=c.max_len, starts=ints(starts), offsets=ints(offsets), k_out=kp, v_out=vp,
                  status=status, **c.scales())
    short = [torch.full((len(lens), 17, heads, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    da.cache_read(c.dk, c.dv, c.dbt, c.dlens, max_seq_len=c.max_len, starts=ints(starts), k_out=short[0], v_out=short[1],
                  status=status, **c.scales())
    for b, n in enumerate(lens):
        for full, packed, cut, whole, part in zip((k, v), (kp, vp), short, read_reference(c, b, n, 0), read_reference(c, b, n, starts[b])):
            assert same_bits(full[b, :n], whole) and bool((full[b, n:] == 0).all())
            assert same_bits(packed[offsets[b]:offsets[b] + kept[b]], part)
            assert bool((packed[offsets[b] + kept[b]] == 9).all())
            m = min(17, kept[b])
            assert same_bits(cut[b, :m], part[:m]) and bool((cut[b, m:] == 9).all())
    assert int(status) == 0


def test_read_back_status_and_bounds(da):
    c = Paged("fp8", [40, 20], 1, 16, 3).gpu()

    def run(lens=(40, 20), starts=(0, 0), offsets=(0, 40), rows=60, bt=None):
        k, v = (torch.full((rows + 8, 1, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        status = status_word()
        da.cache_read(c.dk, c.dv, c.dbt if bt is None else bt, ints(list(lens)), max_seq_len=c.max_len, starts=ints(list(starts)),
                      offsets=ints(list(offsets)), k_out=k[:rows], v_out=v[:rows], status=status, **c.scales())
        assert bool((k[rows:] == 9).all()) and bool((v[rows:] == 9).all())
        return k[:rows], int(status)

    assert run()[1] == 0
    assert run(lens=(41, 20))[1] == 2
    assert run(starts=(0, 21))[1] == 2
    assert run(starts=(-1, 0))[1] == 2
    k, bits = run(offsets=(0, 45))
    assert bits == 2 and same_bits(k[45:], read_reference(c, 1, 20, 0)[0][:15])
    k, bits = run(offsets=(-3, 40))
    assert bits == 2 and bool((k[:40] == 9).all())
    k, bits = run(offsets=(0, 1 << 30))
    assert bits == 2 and bool((k[40:] == 9).all())
    bad = c.dbt.clone()
    bad[0, 0] = 77
    assert run(bt=bad)[1] == 1


def test_append_and_read_back_between_cache_types(da):
    """A 4-bit cache read back and appended to another 4-bit cache of the same scale holds the same bytes."""
    c = Paged("fp4", [100, 37], 2, 16, 5).gpu()
    k, v = da.cache_read(c.dk, c.dv, c.dbt, c.dlens, max_seq_len=112, k_scale=1.0, v_scale=1.0, k_sf=c.dk_sf, v_sf=c.dv_sf)
    new = [torch.zeros_like(x) for x in (c.dk, c.dv, c.dk_sf, c.dv_sf)]
    da.rope_append(None, k, v, None, new[0], new[1], c.dbt, c.dlens, max_seq_len=112, new_lens=c.dlens, k_sf=new[2], v_sf=new[3])
    k2, v2 = da.cache_read(new[0], new[1], c.dbt, c.dlens, max_seq_len=112, k_sf=new[2], v_sf=new[3])
    assert same_bits(k, k2) and same_bits(v, v2)


# ------------------------------------------------------------------ a step of all of them
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("T,G", [(6, 2), (12, 8), (40, 4)])
def test_speculative_steps_captured_in_a_graph(da, kind, T, G):
    """mask -> append at the tree's positions -> attention -> keep, captured and replayed: the cache then holds, byte for
    byte, what appending the accepted tokens alone would have left, and the attention is right at every step."""
    heads, page, B, steps = 2, 16, 3, 4
    ks, vs = SCALES[kind]
    first = [70, 0, 33]
    width = 16
    g = gen(T)
    r = random.Random(T)
    bt = torch.randperm(B * width, generator=g).to(torch.int32).reshape(B, width)
    max_len = width * page

    def empty():
        k, sf = as_cache(torch.zeros(B * width, page, heads, D, dtype=torch.bfloat16), kind, ks)
        return [x.cuda() for x in (k, k, *(() if sf is None else (sf, sf)))]

    caches, plain = [x.clone() for x in empty()], [x.clone() for x in empty()]

    def kw(c):
        return dict(k_sf=c[2], v_sf=c[3]) if kind == "fp4" else {}

    scales = dict(k_scale=ks, v_scale=vs)
    freqs, amp = da.rope_frequencies(D)
    table = da.rope_table(freqs.cuda(), max_len, amplitude=amp)
    pre = [bf16(g, B, max(first), heads, D) for _ in range(2)]
    for c in (caches, plain):
        da.rope_append(None, pre[0].cuda(), pre[1].cuda(), table, c[0], c[1], bt.cuda(), ints(first), max_seq_len=max_len,
                       new_lens=ints(first), **scales, **kw(c))
    status = status_word()
    dbt = bt.cuda()
    q, k, v = (torch.zeros(B, T, h, D, dtype=torch.bfloat16, device="cuda") for h in (heads * G, heads, heads))
    parents, own, keep, counts, lens = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B, T), B, (B, T), B, B))
    mask = torch.zeros(B, T, -(-T // 32), dtype=torch.int32, device="cuda")
    pos = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    out = torch.zeros(B, T, heads * G, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(B, T, heads * G, device="cuda")
    q_rot, new_lens = torch.zeros_like(q), torch.zeros_like(lens)
    seen_cache = [x.clone() for x in caches]

    def step():
        da.tree_mask(parents, lens, max_seq_len=max_len, new_lens=own, mask=mask, positions=pos, status=status)
        da.rope_append(q, k, v, table, caches[0], caches[1], dbt, lens, max_seq_len=max_len, positions=pos, new_lens=own, q_out=q_rot,
                       status=status, **scales, **kw(caches))
        da.decode_attn_tree(q_rot, caches[0], caches[1], dbt, lens, mask, max_seq_len=max_len, new_lens=own, out=out, lse=lse,
                            status=status, **scales, **kw(caches))
        for a, b in zip(seen_cache, caches):
            a.copy_(b)
        da.cache_keep(caches[0], caches[1], dbt, lens, keep, counts, new_tokens=T, max_seq_len=max_len, new_lens=own, out_lens=new_lens,
                      status=status, **kw(caches))

    def fill(now):
        sizes = [T, r.randint(1, T), r.randint(1, T)]
        trees = [random_parents(n, r.random()) + [-1] * (T - n) for n in sizes]
        paths = []
        for b, n in enumerate(sizes):
            t, path = r.randrange(n), []
            while t >= 0:
                path.append(t)
                t = trees[b][t]
            paths.append(path[::-1])
        for x, h in ((q, heads * G), (k, heads), (v, heads)):
            x.copy_(bf16(g, B, T, h, D, std=1.5))
        parents.copy_(ints(trees))
        own.copy_(ints(sizes))
        keep.copy_(ints([p + [0] * (T - len(p)) for p in paths]))
        counts.copy_(ints([len(p) for p in paths]))
        lens.copy_(ints([a + n for a, n in zip(now, sizes)]))
        return sizes, trees, paths

    now = list(first)
    graph = None
    for i in range(steps):
        sizes, trees, paths = fill(now)
        if i == 0:
            step()
        elif graph is None:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            graph.replay()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert int(status) == 0
        c = Paged.__new__(Paged)
        c.kind, c.heads, c.ks, c.vs, c.bt, c.lens = kind, heads, ks, vs, bt, [a + n for a, n in zip(now, sizes)]
        host = [x.cpu() for x in seen_cache]
        c.k, c.v, c.k_sf, c.v_sf = host[0], host[1], *(host[2:] if kind == "fp4" else (None, None))
        check_rows(c, q_rot.cpu(), out, lse, sizes, [ways(p[:n]) for p, n in zip(trees, sizes)])
        # the accepted tokens alone
        accepted = [torch.zeros(B, T, heads, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        for b, p in enumerate(paths):
            for x, y in zip(accepted, (k, v)):
                x[b, :len(p)] = y[b, p]
        now = [a + len(p) for a, p in zip(now, paths)]
        assert new_lens.tolist() == now
        da.rope_append(None, accepted[0], accepted[1], table, plain[0], plain[1], dbt, ints(now), max_seq_len=max_len,
                       new_lens=ints([len(p) for p in paths]), **scales, **kw(plain))
        for x, y in zip(caches, plain):
            x, y = x.cpu(), y.cpu()
            for b, n in enumerate(now):
                for j in range(n):
                    at = (int(bt[b, j // page]), j % page) if x.shape[1] == page else (int(bt[b, j // page]), slice(None), j % page)
                    assert torch.equal(x[at], y[at]), (i, b, j)


# ------------------------------------------------------------------ many rows, in calls of every shape
def cross_call(da, c, q, **kw):
    return da.cross_attn(q, c.dk, c.dv, c.dbt, c.dlens, max_seq_len=c.max_len, **c.scales(), **kw)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("seed", range(10))
@pytest.mark.parametrize("splits", [0, 1])
def test_many_rows_of_any_shape(da, kind, seed, splits):
    """Lengths on both sides of a step's 128 keys and of the cuts, empty requests and padding, odd groups."""
    r = random.Random(seed)
    G = [1, 5, 7, 100, 3, 16, 4, 1, 8, 11][seed]
    heads, B = r.randint(1, 3), [70, 9, 5, 3, 2, 40, 40, 35, 6, 17][seed]
    T = r.randint(128 // G + 1, 128 // G + [60, 40, 150, 3, 600, 9, 5, 140, 100, 30][seed])
    most = [200, 700, 1500, 600, 5000, 300, 2000, 900, 3500, 1100][seed]
    lens = [r.choice([0, 1, 128 * r.randint(1, most // 128 + 1) + r.randint(-1, 1), r.randint(1, most)]) for _ in range(B)]
    own = [r.choice([0, 1, T, r.randint(0, T)]) for _ in range(B)]
    lens[-1], own[-1] = most, T
    c = Paged(kind, lens, heads, r.choice([0, 16, 64, 128]), 400 + seed).gpu()
    q = bf16(gen(seed), B, T, heads * G, D, std=2.0)
    status = status_word()
    out, lse = cross_call(da, c, q.cuda(), q_lens=ints(own), status=status, num_splits=splits)
    check_rows(c, q, out, lse, own, None)
    assert int(status) == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("lens,T,G", [([40000], 130, 1), ([20000, 1, 3], 65, 4)])
def test_few_rows_over_long_keys_in_many_pieces(da, kind, lens, T, G):
    c = Paged(kind, lens, 1, 64, 12).gpu()
    q = bf16(gen(9), len(lens), T, G, D, std=2.0)
    out, lse = cross_call(da, c, q.cuda())
    check_rows(c, q, out, lse, [T] * len(lens), None)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_many_rows_of_more_heads_than_ctas(da, kind):
    """Several whole items to a CTA."""
    heads = 330
    c = Paged(kind, [150, 20], heads, 16, 13).gpu()
    q = bf16(gen(10), 2, 140, heads, D, std=2.0)
    out, lse = cross_call(da, c, q.cuda(), q_lens=ints([140, 77]))
    check_rows(c, q, out, lse, [140, 77], None)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("T", [40, 300])
@pytest.mark.parametrize("splits", [0, 1])
def test_many_rows_of_nothing_but_padding(da, kind, T, splits):
    c = Paged(kind, [100, 30], 2, 16, 14).gpu()
    q = torch.full((2, T, 8, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    out, lse = cross_call(da, c, q, q_lens=ints([0, 0]), num_splits=splits)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("T", [40, 100, 250])
@pytest.mark.parametrize("splits", [0, 1])
def test_status_bits_of_many_rows(da, kind, T, splits):
    """As for few rows, also where the cache is read back first."""
    c = Paged(kind, [100, 50], 1, 16, 15).gpu()
    q = bf16(gen(3), 2, T, 4, D).cuda()

    def bits(lens=c.dlens, bt=c.dbt, own=None):
        status = status_word()
        da.cross_attn(q, c.dk, c.dv, bt, lens, max_seq_len=c.max_len, q_lens=own, status=status, num_splits=splits, **c.scales())
        return int(status)

    bad = c.dbt.clone()
    bad[0, 1] = 1000
    assert bits() == 0 and bits(bt=bad) == 1 and bits(lens=ints([101, -1])) == 2 and bits(own=ints([T, T + 1])) == 2
    assert bits(own=ints([-1, 0])) == 2


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("splits", [0, 1])
def test_many_rows_on_two_streams_and_in_one_workspace(da, kind, splits):
    """Calls that overlap on two streams, and calls of different shapes that follow one another in one workspace, give
    the bits of calls alone."""
    shapes = [([700, 90], 2, 4, 50), ([300, 1200, 5], 1, 5, 90), ([90] * 6, 3, 1, 140), ([2500], 1, 8, 17)]
    cases = []
    for i, (lens, heads, G, T) in enumerate(shapes):
        c = Paged(kind, lens, heads, 16, 20 + i).gpu()
        q = bf16(gen(i), len(lens), T, heads * G, D, std=2.0).cuda()
        cases.append((c, q, cross_call(da, c, q, num_splits=splits)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for rep in range(6):
        for i, (c, q, _) in enumerate(cases):
            got.append((i, cross_call(da, c, q, num_splits=splits, stream=streams[(i + rep) % 2])))
    torch.cuda.synchronize()
    ws = torch.full((1 << 24,), float("nan"), device="cuda")
    for rep in range(3):
        for i, (c, q, _) in enumerate(cases):
            got.append((i, cross_call(da, c, q, num_splits=splits, workspace=ws)))
    torch.cuda.synchronize()
    for i, (out, lse) in got:
        assert torch.equal(out, cases[i][2][0]) and torch.equal(lse, cases[i][2][1]), i


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("splits", [0, 1])
def test_many_rows_replayed_with_other_lengths(da, kind, splits):
    """The plan is made on the device: a captured call follows the lengths, the pages and the rows."""
    c = Paged(kind, [900, 333, 64], 2, 16, 21).gpu()
    T = 60
    q = bf16(gen(11), 3, T, 8, D, std=2.0)
    lens, own, dq = c.dlens.clone(), ints([T, T, T]), q.cuda()
    out = torch.empty(3, T, 8, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, T, 8, device="cuda")

    def call():
        da.cross_attn(dq, c.dk, c.dv, c.dbt, lens, max_seq_len=900, q_lens=own, out=out, lse=lse, num_splits=splits,
                      **c.scales())

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for now, rows in (([900, 333, 64], [60, 60, 60]), ([1, 0, 17], [60, 3, 0]), ([0, 0, 0], [60, 60, 60]), ([890, 129, 64], [1, 60, 33])):
        lens.copy_(ints(now))
        own.copy_(ints(rows))
        out.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        c.lens = now
        check_rows(c, q, out, lse, rows, None)


@pytest.mark.parametrize("T,splits", [(4, 0), (50, 0), (50, 1)])
def test_infinite_keys_weigh_nothing_or_everything(da, T, splits):
    """A key whose score is -inf is as if it were not there; one of +inf makes its rows NaN, and those alone."""
    c = Paged("bf16", [300], 1, 16, 22).gpu()
    q = bf16(gen(12), 1, T, 4, D)
    q[..., 0] = q[..., 0].abs() + 0.5
    q[0, 1, :, 0] = -1.0
    at = (int(c.bt[0, 77 // 16]), 77 % 16)
    c.dk[at[0], at[1], 0, 0] = -math.inf
    out, lse = cross_call(da, c, q.cuda(), num_splits=splits)
    assert bool(out[0, 1].isnan().all()) and bool(lse[0, 1].isnan().all())
    k, v = (R.gather(c.values(w) * 1.0, c.bt, 0, 300)[:, 0] for w in "kv")
    seen = torch.ones(4 * (T - 1), 300, dtype=torch.bool)
    seen[:, 77] = False
    rest = [t for t in range(T) if t != 1]
    assert_attention(out[0, rest].double().cpu().reshape(-1, D), lse[0, rest].double().cpu().reshape(-1),
                     q[0, rest].double().reshape(-1, D), k, v, seen, SCALE, tolerance_for("bf16", 4, T))


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_rows_of_any_magnitude(da, kind):
    """Rows of q as large and as small as bf16 goes: with 16-bit operands each is scaled by itself."""
    T = 150
    c = Paged(kind, [200], 1, 16, 23).gpu()
    q = bf16(gen(13), 1, T, 1, D)
    for t in range(T):
        q[0, t] = (q[0, t].float() * 2.0 ** (-120 + 1.6 * t)).to(torch.bfloat16)
    q[0, 7] = 0
    scale = 2.0 ** -100
    out, lse = cross_call(da, c, q.cuda(), scale=scale, num_splits=1)
    # Weights of at most 2^-30 of the largest are subnormal in f16, which holds them to 2^-25 (half its last step) of 2^6:
    # 200 of them can be off by 2^-31 each.  (With one key of all the weight that is more than the relative tolerance.)
    lost = 0.0 if kind == "bf16" else 200 * 2.0 ** -31 * float((c.values("v") * c.vs).abs().max())
    check_rows(c, q, out, lse, [T], None, scale=scale, lost=lost)


def test_far_pages_and_tokens(da):
    """Pages and tokens behind 2^32 bytes of a cache: attention of few and of many rows, kept tokens, reading back."""
    page, heads, lens = 16, 2, [200, 75]
    near = Paged("bf16", lens, heads, page, 24).gpu()
    per_page = page * heads * D * 2
    first = (1 << 32) // per_page + 5
    pages = first + near.k.shape[0]
    k, v = (torch.empty(pages, page, heads, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    k[first:], v[first:] = near.dk, near.dv
    bt = near.dbt + first
    for T, splits in ((3, 0), (60, 0), (60, 1)):
        q = bf16(gen(14), 2, T, 4 * heads, D, std=2.0).cuda()
        want = cross_call(da, near, q, num_splits=splits)
        got = da.cross_attn(q, k, v, bt, near.dlens, max_seq_len=200, num_splits=splits)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = da.cache_read(k, v, bt, near.dlens, max_seq_len=200)
    want = da.cache_read(near.dk, near.dv, near.dbt, near.dlens, max_seq_len=200)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for kc, vc, b in ((k, v, bt), (near.dk, near.dv, near.dbt)):
        da.cache_keep(kc, vc, b, near.dlens, ints([[1, 4, 7], [0, 3, 5]]), ints([3, 3]), new_tokens=8, max_seq_len=200)
    assert torch.equal(k[first:], near.dk) and torch.equal(v[first:], near.dv)


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_kept_tokens_of_a_cache_whose_values_are_its_keys(da, kind):
    T = 600
    c = Paged(kind, [T + 9], 2, 16, 25).gpu()
    other = [None if x is None else x.clone() for x in (c.dk, c.dk_sf)]
    keep = ints([list(range(1, T, 2))])
    counts = ints([T // 2])
    da.cache_keep(c.dk, c.dk, c.dbt, c.dlens, keep, counts, new_tokens=T, max_seq_len=c.max_len, k_sf=c.dk_sf, v_sf=c.dk_sf)
    v, v_sf = (None if x is None else x.clone() for x in (c.dv, c.dv_sf))
    da.cache_keep(other[0], v, c.dbt, c.dlens, keep, counts, new_tokens=T, max_seq_len=c.max_len, k_sf=other[1], v_sf=v_sf)
    assert torch.equal(c.dk, other[0]) and (c.dk_sf is None or torch.equal(c.dk_sf, other[1]))
