"""Trees of drafted tokens and cross attention over a KV cache: what is measured, and their plain forms.

  mask    of a tree of drafted tokens (each one's parent): per token the tokens on its way to the root, as bits, and its position
  tree    decode attention of the tree's tokens: each sees the cache's earlier tokens and those on its way to the root
  keep    the tokens of the accepted path, scattered over the cache's end, moved together (keys and values, any cache type)
  read    keys and values of a cache of any type as bf16 tensors, padded or one request behind the other
  cross   attention of every token of a prompt (or of one new token) over an encoder's states, of another length

Formats.  Caches are those of operators.py: bf16, E4M3 bytes with one scale, or 4-bit values (value 2i in the low and 2i + 1 in
the high nibble of byte i) with an E4M3 scale for each 16 of them, [pages, heads, page, 8], and one for the cache.
Request b's n new tokens are the last n of its `lens` tokens.  Bit i % 32 of word i / 32 of row t of a mask says that new token t
sees new token i.  Rows of q behind a request's own are padding: zeros, and a log-sum-exp of -inf.
"""
import math
import random

import torch

own = False

D = 128
DEV = "cuda" if torch.cuda.is_available() else "cpu"
E4M3 = torch.float8_e4m3fn
K_SCALE = {"bf16": 1.0, "fp8": 0.0625, "fp4": 0.02}
V_SCALE = {"bf16": 1.0, "fp8": 0.03125, "fp4": 0.015}


# ------------------------------------------------------------------ the cases
def _mask(name, batch, nodes, ragged):
    return dict(name=name, op="mask", batch=batch, nodes=nodes, ragged=ragged, lo=64, hi=8192)


def _tree(name, batch, nodes, ragged, hq, hkv, page, lo, hi, cache):
    return dict(name=name, op="tree", batch=batch, nodes=nodes, ragged=ragged, hq=hq, hkv=hkv, page=page, lo=lo, hi=hi, cache=cache)


def _keep(name, batch, nodes, most, hkv, page, cache, hi):
    return dict(name=name, op="keep", batch=batch, nodes=nodes, most=most, ragged=False, hkv=hkv, page=page, cache=cache, lo=nodes, hi=hi)


def _read(name, batch, hkv, page, lo, hi, cache, packed, skip):
    return dict(name=name, op="read", batch=batch, hkv=hkv, page=page, lo=lo, hi=hi, cache=cache, packed=packed, skip=skip)


def _cross(name, batch, tokens, ragged, hq, hkv, page, lo, hi, cache):
    return dict(name=name, op="cross", batch=batch, nodes=tokens, ragged=ragged, hq=hq, hkv=hkv, page=page, lo=lo, hi=hi, cache=cache)


def listed():
    return [
        # one request's tree of 16 drafts, before every speculative step: all latency
        _mask("mask 1 x 16", 1, 16, False),
        # a serving batch, trees of different sizes
        _mask("mask 128 x 63 ragged", 128, 63, True),
        # one chat of 4K tokens that verifies 16 drafts: 64 query rows per KV head, latency
        _tree("tree 1 x 16, 4K bf16", 1, 16, False, 32, 8, 0, 4096, 4096, "bf16"),
        # ragged serving of small trees over an FP8 cache: 16 query rows per KV head, bandwidth
        _tree("tree 32 x 4 ragged fp8", 32, 4, True, 32, 8, 16, 1024, 16384, "fp8"),
        # large trees over long paged contexts: 256 query rows per KV head
        _tree("tree 16 x 32, 64/8 heads, bf16", 16, 32, True, 64, 8, 16, 4096, 16384, "bf16"),
        # after a step of one request: 5 of 16 drafts were accepted
        _keep("keep 1 of 16 bf16", 1, 16, 5, 8, 16, "bf16", 4096),
        # after a step of a large batch over 4-bit pages
        _keep("keep 256 of 32 fp4", 256, 32, 8, 8, 16, "fp4", 2048),
        # a prefix of an FP8 cache read back for one request's next prompt chunk
        _read("read 1 x 4K fp8", 1, 8, 16, 4096, 4096, "fp8", False, 0),
        # contexts moved out of 4-bit pages, packed: all bandwidth
        _read("read 32 ragged fp4", 32, 8, 16, 512, 16381, "fp4", True, 300),
        # one decoder step of 32 requests over 1500 states each, one query head per KV head
        _cross("cross 32 x 1, 1500 states", 32, 1, False, 16, 16, 0, 1500, 1500, "bf16"),
        # ragged decoder prompts over ragged states in FP8 pages
        _cross("cross 8 x 448 ragged fp8", 8, 448, True, 20, 20, 16, 100, 1500, "fp8"),
        # long inputs, grouped heads: all tensor cores, the largest case
        _cross("cross 4 x 2048, 4096 states", 4, 2048, False, 32, 8, 0, 4096, 4096, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mask", "tree", "tree", "tree", "keep", "read", "read", "cross", "cross", "cross"])
    hkv = rng.choice([1, 2, 4, 8, 8])
    page = rng.choice([16, 16, 32, 48, 64, 128])
    cache = rng.choice(["bf16", "bf16", "fp8", "fp4"])
    if op == "mask":
        c = _mask("", _log(rng, 1, 256), _log(rng, 2, 128), rng.random() < 0.6)
    elif op == "tree":
        batch, group, nodes = _log(rng, 1, 64), rng.choice([1, 2, 4, 4, 5, 8, 8]), _log(rng, 2, 64)
        hi = _log(rng, 256, min(32768, 262144 // batch, 268435456 // (batch * nodes * group * hkv)))
        c = _tree("", batch, nodes, rng.random() < 0.6, hkv * group, hkv, rng.choice([0, page, page]), rng.randint(nodes, max(nodes, hi)), max(nodes, hi), cache)
    elif op == "keep":
        nodes = _log(rng, 4, 64)
        c = _keep("", _log(rng, 1, 256), nodes, rng.randint(1, nodes // 2), hkv, page, cache, nodes + _log(rng, 16, 2048))
    elif op == "read":
        batch = _log(rng, 1, 64)
        hi = _log(rng, 32, min(32768, 262144 // batch))
        c = _read("", batch, hkv, rng.choice([0, page, page]), rng.randint(1, hi), hi, cache, rng.random() < 0.5, rng.choice([0, 0, rng.randint(1, hi - 1)]))
    else:
        batch, group, tokens = _log(rng, 1, 32), rng.choice([1, 1, 1, 2, 4, 5, 8]), rng.choice([1, _log(rng, 2, 2048), _log(rng, 2, 2048)])
        hi = _log(rng, 16, min(8192, max(17, 536870912 // (batch * tokens * group * hkv))))
        c = _cross("", batch, tokens, rng.random() < 0.5, hkv * group, hkv, rng.choice([0, 0, page]), rng.randint(1, hi), hi, cache)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _ragged(lo, hi, n, seed):
    """n sizes of lo .. hi, hi among them: the same set for every seed (so the same number of pages), in the seed's order."""
    r = random.Random(lo * 65536 + hi)
    v = [hi] + [r.randint(lo, hi) for _ in range(n - 1)]
    random.Random(seed).shuffle(v)
    return v


def _lengths(c, seed):
    return _ragged(c["lo"], c["hi"], c["batch"], seed)


def _own_tokens(c, seed):
    """New tokens (or prompt tokens) of each request; the other rows of q are padding."""
    return _ragged(max(1, c["nodes"] // 4), c["nodes"], c["batch"], seed + 1) if c["ragged"] else [c["nodes"]] * c["batch"]


def _randn(g, *shape, dtype=torch.bfloat16, std=1.0):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=g)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pages(c, lens, g):
    """A block table over shuffled pages; entries behind a request's last page are 0."""
    need = [-(-n // c["page"]) for n in lens]
    width = max(max(need), 1)
    ids = torch.randperm(sum(need) + 3, generator=g, device=DEV).to(torch.int32)
    at = torch.zeros(len(lens), width, dtype=torch.int64)
    first = 0
    for b, n in enumerate(need):
        at[b, :n] = torch.arange(first, first + n)
        first += n
    held = torch.arange(width)[None, :] < torch.tensor(need)[:, None]
    return torch.where(held.to(DEV), ids[at.to(DEV)], 0).to(torch.int32).contiguous(), sum(need) + 3


def _to_cache(x, kind, scale):
    """Values [groups, tokens, heads, 128] as a cache of `kind`: (bytes or bf16, block scales or None)."""
    if kind == "bf16":
        return x, None
    y = x.float() / scale
    if kind == "fp8":
        return y.clamp(-448, 448).to(E4M3).view(torch.uint8), None
    y = y.unflatten(-1, (8, 16))
    sf = (y.abs().amax(-1) / 6).clamp(max=448).to(E4M3)
    t = torch.where(sf.float()[..., None] > 0, y / sf.float()[..., None], 0.0).flatten(-2)
    code = (t.abs()[..., None] > torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)).sum(-1).to(torch.uint8)
    code |= torch.signbit(t).to(torch.uint8) << 3
    return code[..., 0::2] | (code[..., 1::2] << 4), sf.view(torch.uint8).permute(0, 2, 1, 3).contiguous()


def _caches(c, groups, tokens, g):
    st = {}
    for n, scale in (("k", K_SCALE), ("v", V_SCALE)):
        x, sf = zip(*(_to_cache(_randn(g, min(256, groups - i), tokens, c["hkv"], D), c["cache"], scale[c["cache"]]) for i in range(0, groups, 256)))
        st[n], st[n + "_sf"] = torch.cat(x), None if sf[0] is None else torch.cat(sf)
    return st


def _trees(c, sizes, seed):
    """Parents [B, nodes]: a token's parent is a root's follower or a few places before it; -1 for roots and padding."""
    r = random.Random(seed)
    rows = [[-1] + [-1 if r.random() < 0.03 else r.randint(max(0, t - 9), t - 1) for t in range(1, n)] for n in sizes]
    return [v + [-1] * (c["nodes"] - len(v)) for v in rows]


def _bits(seen):
    """Truth values [..., T, T] as words of 32 bits [..., T, ceil(T / 32)]."""
    x = torch.nn.functional.pad(seen, (0, -seen.shape[-1] % 32)).unflatten(-1, (-1, 32)).long()
    w = (x << torch.arange(32, device=seen.device)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _seen_of(parents, sizes):
    """Truth values [B, T, T] on the CPU: token i is on token t's way to its root (itself among them)."""
    out = torch.zeros(len(parents), len(parents[0]), len(parents[0]), dtype=torch.bool)
    for b, v in enumerate(parents):
        for t in range(sizes[b]):
            if v[t] >= 0:
                out[b, t] = out[b, v[t]]
            out[b, t, t] = True
    return out


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    lens = _lengths(c, seed)
    st = dict(case=c, max_len=max(lens))
    if c["op"] in ("mask", "tree", "keep", "cross"):
        sizes = _own_tokens(c, seed)
        if c["op"] != "cross":
            lens = [max(a, b) for a, b in zip(lens, sizes)]
        st["sizes"] = _ints(sizes) if c["ragged"] else None
    st["lens"] = _ints(lens)
    if c["op"] == "mask":
        st["parents"] = _ints(_trees(c, sizes, seed))
        return st
    if c["page"]:
        st["block_table"], pages = _pages(c, lens, g)
        st.update(_caches(c, pages, c["page"], g))
    else:
        st["block_table"] = None
        st.update(_caches(c, c["batch"], -(-max(lens) // 16) * 16, g))
    if c["op"] in ("tree", "cross"):
        st["q"] = _randn(g, c["batch"], c["nodes"], c["hq"], D, std=2.0)
    if c["op"] == "tree":
        st["mask"] = _bits(_seen_of(_trees(c, sizes, seed), sizes).to(DEV))
    if c["op"] == "keep":
        # The accepted tokens: the first few as they lie, then a path whose tokens lie behind all the places that it moves to, so
        # that a pass over its own result moves the same tokens again.
        r = random.Random(seed)
        keep, counts = [], []
        for _ in range(c["batch"]):
            m = r.randint(1, c["most"])
            stay = r.randint(1, m)
            path = list(range(stay)) + sorted(r.sample(range(m, c["nodes"]), m - stay))
            keep.append(path + [0] * (c["most"] - m))
            counts.append(m)
        st["keep"], st["counts"] = _ints(keep), _ints(counts)
        st["new_lens"] = torch.empty_like(st["lens"])
    if c["op"] == "read":
        starts = [min(c["skip"], n) for n in lens]
        held = [n - s for n, s in zip(lens, starts)]
        st["starts"] = _ints(starts) if c["skip"] else None
        st["width"] = max(held)
        shape = (sum(held), c["hkv"], D) if c["packed"] else (c["batch"], max(held), c["hkv"], D)
        st["offsets"] = _ints([sum(held[:b]) for b in range(c["batch"])]) if c["packed"] else None
        st["k_out"], st["v_out"] = (torch.zeros(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    return st


# ------------------------------------------------------------------ the plain forms
def _pairs():
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    v = torch.cat([v, -v])
    byte = torch.arange(256, device=DEV)
    return torch.stack([v[byte % 16], v[byte // 16]], dim=1)


def _values(x, sf, scale):
    """Rows of a cache [..., heads, width], their block scales [..., heads, 8] or None, as the 32-bit values they stand for."""
    if sf is not None:
        x = _pairs()[x.int()].flatten(-2).unflatten(-1, (8, 16))
        return ((x * sf.contiguous().view(E4M3).float()[..., None]) * scale).flatten(-2)
    return (x.view(E4M3).float() if x.dtype == torch.uint8 else x.float()) * scale


def _tokens(st, c):
    """The caches by request: K and V [B, tokens, heads, 128] in 32 bits."""
    got = []
    for n, scale in (("k", K_SCALE), ("v", V_SCALE)):
        x, sf = st[n], st[n + "_sf"]
        sf = None if sf is None else sf.permute(0, 2, 1, 3)
        if st["block_table"] is not None:
            at = st["block_table"].long()
            x, sf = x[at].flatten(1, 2), None if sf is None else sf[at].flatten(1, 2)
        got.append(_values(x, sf, scale[c["cache"]]))
    return got


def _sizes(st, c):
    return st["sizes"].long() if st["sizes"] is not None else torch.full((c["batch"],), c["nodes"], device=DEV)


def _plain_mask(st, c):
    t = torch.arange(c["nodes"], device=DEV)
    n, parents = _sizes(st, c), st["parents"].long()
    way = (t == parents[:, :, None]) | (t == t[:, None])  # one step towards the root, or none
    for _ in range(max(1, (c["nodes"] - 1).bit_length())):  # each product doubles the steps
        way = torch.matmul(way.float(), way.float()) > 0
    way &= (t < n[:, None])[:, :, None]
    positions = torch.where(t < n[:, None], st["lens"].long()[:, None] - n[:, None] + way.sum(-1) - 1, 0)
    return _bits(way), positions.to(torch.int32)


def _plain_attention(st, c, seen):
    """q's rows over the tokens `seen` [B, nodes, tokens] says."""
    b, t, hkv = c["batch"], c["nodes"], c["hkv"]
    k, v = (x.transpose(1, 2) for x in _tokens(st, c))
    q = st["q"].float().view(b, t, hkv, -1, D).permute(0, 2, 3, 1, 4)
    s = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, (-1, t)) * (1.0 / math.sqrt(D))
    s = torch.where(seen[:, None, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    del s
    n = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (-1, t)) / torch.where(n > 0, n, 1.0)
    lse = (m + torch.log(n))[..., 0]
    return o.permute(0, 3, 1, 2, 4).reshape(b, t, c["hq"], D).to(torch.bfloat16), lse.permute(0, 3, 1, 2).reshape(b, t, c["hq"])


def _own_rows(st, c):
    return torch.arange(c["nodes"], device=DEV) < _sizes(st, c)[:, None]


def _width(st, c):
    return st["block_table"].shape[1] * c["page"] if st["block_table"] is not None else st["k"].shape[1]


def _plain_tree(st, c):
    t, j = torch.arange(c["nodes"], device=DEV), torch.arange(_width(st, c), device=DEV)
    lens, n = st["lens"].long(), _sizes(st, c)
    way = (st["mask"][:, :, t // 32] >> (t % 32)) & 1 != 0
    place = (j - (lens - n)[:, None])[:, None].expand(-1, c["nodes"], -1)  # of a key among the new tokens
    seen = (place < 0) | torch.gather(way, 2, place.clamp(0, c["nodes"] - 1))
    return _plain_attention(st, c, seen & (j < lens[:, None])[:, None] & _own_rows(st, c)[:, :, None])


def _plain_cross(st, c):
    j = torch.arange(_width(st, c), device=DEV)
    return _plain_attention(st, c, (j < st["lens"].long()[:, None])[:, None] & _own_rows(st, c)[:, :, None])


def _plain_keep(st, c):
    base = st["lens"].long() - c["nodes"]
    i = torch.arange(c["most"], device=DEV)
    use = i < st["counts"][:, None]
    src, dst = (base[:, None] + st["keep"])[use], (base[:, None] + i)[use]
    row = torch.arange(c["batch"], device=DEV)[:, None].expand(-1, c["most"])[use]
    table = st["block_table"].long()
    ps, pd = table[row, src // c["page"]], table[row, dst // c["page"]]
    for n in ("k", "v"):
        st[n][pd, dst % c["page"]] = st[n][ps, src % c["page"]]
        if st[n + "_sf"] is not None:
            sf = st[n + "_sf"].permute(0, 2, 1, 3)
            sf[pd, dst % c["page"]] = sf[ps, src % c["page"]]
    st["new_lens"].copy_(base + st["counts"])


def _plain_read(st, c):
    lens = st["lens"].long()
    starts = st["starts"].long() if st["starts"] is not None else torch.zeros_like(lens)
    j = torch.arange(st["width"], device=DEV)
    use = j < (lens - starts)[:, None]
    tok = (starts[:, None] + j)[use]
    row = torch.arange(c["batch"], device=DEV)[:, None].expand(-1, st["width"])[use]
    place = tok
    if c["page"]:
        row, place = st["block_table"].long()[row, tok // c["page"]], tok % c["page"]
    for n, scale in (("k", K_SCALE), ("v", V_SCALE)):
        sf = None if st[n + "_sf"] is None else st[n + "_sf"].permute(0, 2, 1, 3)[row, place]
        x = _values(st[n][row, place], sf, scale[c["cache"]]).to(torch.bfloat16)
        if c["packed"]:
            st[n + "_out"].copy_(x)
        else:
            st[n + "_out"][use] = x


# ------------------------------------------------------------------ one pass
def _own(st, c):
    from split_kv_decode_attention_gb300 import binding as da
    if c["op"] == "mask":
        return da.tree_mask(st["parents"], st["lens"], max_seq_len=st["max_len"], new_lens=st["sizes"])
    kind = c["cache"]
    sf = dict(k_sf=st["k_sf"], v_sf=st["v_sf"])
    scales = dict(k_scale=K_SCALE[kind], v_scale=V_SCALE[kind], **sf)
    if c["op"] == "tree":
        return da.decode_attn_tree(st["q"], st["k"], st["v"], st["block_table"], st["lens"], st["mask"], max_seq_len=st["max_len"],
                                   new_lens=st["sizes"], **scales)
    if c["op"] == "cross":
        return da.cross_attn(st["q"], st["k"], st["v"], st["block_table"], st["lens"], max_seq_len=st["max_len"], q_lens=st["sizes"], **scales)
    if c["op"] == "keep":
        da.cache_keep(st["k"], st["v"], st["block_table"], st["lens"], st["keep"], st["counts"], new_tokens=c["nodes"],
                      max_seq_len=st["max_len"], out_lens=st["new_lens"], **sf)
    else:
        da.cache_read(st["k"], st["v"], st["block_table"], st["lens"], max_seq_len=st["max_len"], starts=st["starts"],
                      offsets=st["offsets"], k_out=st["k_out"], v_out=st["v_out"], **scales)


def run(state):
    c = state["case"]
    if own:
        r = _own(state, c)
    else:
        r = {"mask": _plain_mask, "tree": _plain_tree, "keep": _plain_keep, "read": _plain_read, "cross": _plain_cross}[c["op"]](state, c)
    if c["op"] == "mask":
        return dict(mask=r[0], positions=r[1])
    if c["op"] == "keep":
        # the cache's own bytes: they have to be equal, which is more than the values they stand for
        return {n: state[n] for n in ("k", "v", "k_sf", "v_sf", "new_lens") if state[n] is not None}
    if c["op"] == "read":
        return dict(k=state["k_out"], v=state["v_out"])
    return dict(out=r[0], lse=r[1])


# ------------------------------------------------------------------ 64 bits, from the definitions
def _row_64(codes, sf, kind, scale):
    """Tokens [n, heads, width] of a cache (block scales [heads, n, 8]) as 64-bit values."""
    if kind == "bf16":
        return codes.double()
    if kind == "fp8":
        return codes.view(E4M3).double() * scale
    nib = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).double()
    mag = nib % 8
    e = (mag / 2).floor()
    val = torch.where(e == 0, mag / 2, (1 + (mag % 2) / 2) * torch.exp2(e - 1)) * torch.where(nib >= 8, -1.0, 1.0)
    return val * sf.contiguous().view(E4M3).double().transpose(0, 1).repeat_interleave(16, dim=-1) * scale


def _request_64(st, c, b, n):
    """K and V of request b's first n tokens: [n, heads, 128]."""
    got = []
    for name, scale in (("k", K_SCALE), ("v", V_SCALE)):
        x, sf = st[name], st[name + "_sf"]
        if st["block_table"] is not None:
            at = st["block_table"][b, :-(-n // c["page"])].long()
            x = x[at].flatten(0, 1)
            sf = None if sf is None else sf[at].transpose(0, 1).flatten(1, 2)
        else:
            x, sf = x[b], None if sf is None else sf[b]
        got.append(_row_64(x[:n], None if sf is None else sf[:, :n], c["cache"], scale[c["cache"]]))
    return got


def exact(case, seed):
    c = case
    if c["op"] == "mask" or (c["op"] == "keep" and c["cache"] != "bf16"):
        return None  # whole numbers and bytes: no value in 64 bits
    st = prepare(c, seed)
    lens = st["lens"].tolist()
    if c["op"] == "keep":
        k, v = st["k"].double(), st["v"].double()
        for b, n in enumerate(lens):
            for i, w in enumerate(st["keep"][b, :int(st["counts"][b])].tolist()):
                at = [(int(st["block_table"][b, p // c["page"]]), p % c["page"]) for p in (n - c["nodes"] + i, n - c["nodes"] + w)]
                for x, y in ((k, st["k"]), (v, st["v"])):
                    x[at[0]] = y[at[1]].double()
        return dict(k=k, v=v, new_lens=None)
    if c["op"] == "read":
        out = [torch.zeros(st["k_out"].shape, dtype=torch.float64, device=DEV) for _ in range(2)]
        for b, n in enumerate(lens):
            s = int(st["starts"][b]) if st["starts"] is not None else 0
            if s == n:
                continue
            for o, x in zip(out, _request_64(st, c, b, n)):
                if c["packed"]:
                    o[int(st["offsets"][b]):int(st["offsets"][b]) + n - s] = x[s:]
                else:
                    o[b, :n - s] = x[s:]
        return dict(k=out[0], v=out[1])
    group = c["hq"] // c["hkv"]
    out = torch.zeros(c["batch"], c["nodes"], c["hq"], D, dtype=torch.float64, device=DEV)
    lse = torch.full((c["batch"], c["nodes"], c["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    sizes = st["sizes"].tolist() if st["sizes"] is not None else [c["nodes"]] * c["batch"]
    parents = _trees(c, sizes, seed) if c["op"] == "tree" else None
    seen = _seen_of(parents, sizes).to(DEV) if parents else None
    for b, n in enumerate(lens):
        m = sizes[b]
        k, v = _request_64(st, c, b, n)
        for h in range(c["hq"]):
            s = (st["q"][b, :m, h].double() @ k[:, h // group].T) / math.sqrt(D)
            if seen is not None:
                s[:, n - m:].masked_fill_(~seen[b, :m, :m], -math.inf)
            lse[b, :m, h] = torch.logsumexp(s, 1)
            out[b, :m, h] = torch.exp(s - lse[b, :m, h, None]) @ v[:, h // group]
    return dict(out=out, lse=lse)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    lens = _lengths(c, 0)
    if c["op"] == "mask":
        n = sum(_own_tokens(c, 0))
        words = -(-c["nodes"] // 32)
        return dict(bytes=4 * n + 8 * c["batch"] + 4 * c["batch"] * c["nodes"] * (words + 1), flops=4 * n)
    row = {"bf16": 2 * D, "fp8": D, "fp4": D // 2 + D // 16}[c["cache"]] * c["hkv"]
    if c["op"] == "keep":
        moved = c["batch"] * (1 + c["most"]) / 4  # of the m kept, half lie where they were
        return dict(bytes=4 * row * moved + 16 * c["batch"] + 4 * c["batch"] * c["most"], flops=0)
    if c["op"] == "read":
        n = sum(max(0, x - c["skip"]) for x in lens)
        return dict(bytes=2 * n * (row + 2 * D * c["hkv"]), flops=2 * n * D * c["hkv"])
    sizes = _own_tokens(c, 0)
    rows = sum(sizes) * c["hq"]
    if c["op"] == "tree":
        lens = [max(a, b) for a, b in zip(lens, sizes)]
    pairs = sum(a * b for a, b in zip(lens, sizes)) * c["hq"]
    return dict(bytes=2 * sum(lens) * row + rows * (4 * D + 4), flops=4 * D * pairs)
