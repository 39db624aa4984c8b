"""The operators around a decode step's KV cache: what is measured, and their plain forms.

  table    cos / sin of every position for rotary embeddings, frequencies scaled for long contexts
  append   rotary positions on the new tokens' q and k, and k / v written into the cache (bf16, FP8 E4M3, or 4 bits)
  digest   per page and KV head: the channel-wise minimum and maximum of its keys in 8 bits, for block selection
  attend4  decode attention over a cache held in 4 bits (E2M1 values, one E4M3 scale per 16 of them)
  sparse   decode attention over the top_k pages that the digests score highest for each query

Formats.  A 4-bit cache holds value 2i of a (token, head) in the low and 2i + 1 in the high nibble of byte i; the value is
scale * block scale * E2M1 (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign), its block scales are [pages, heads, page, 8] E4M3.
New keys are rotated in 32 bits (each product and sum rounded), rounded to bf16, and from there (times 1 / scale, in 32
bits) to the cache's type; a block's scale is its largest magnitude / 6.
A digest holds rint(x * 127 / amax) of the page's minimum and maximum per channel, and amax / 127.  The score of a page is
the largest over the group's heads of  (sum_d max(q_d * min_d, q_d * max_d) of 8-bit q and digest) * digest scale * q's scale.
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
def _table(name, max_pos, rot, base_lo, factor):
    return dict(name=name, op="table", max_pos=max_pos, rot=rot, base_lo=base_lo, factor=factor)


def _append(name, batch, q_len, hq, hkv, page, cache, rot, interleaved, past):
    return dict(name=name, op="append", batch=batch, q_len=q_len, hq=hq, hkv=hkv, page=page, cache=cache, rot=rot,
                interleaved=interleaved, past=past)


def _digest(name, batch, lo, hi, hkv, page, cache, new):
    return dict(name=name, op="digest", batch=batch, lo=lo, hi=hi, hkv=hkv, page=page, cache=cache, new=new)


def _attend4(name, batch, q_len, causal, hq, hkv, page, lo, hi):
    return dict(name=name, op="attend4", batch=batch, q_len=q_len, causal=causal, hq=hq, hkv=hkv, page=page, lo=lo, hi=hi)


def _sparse(name, batch, q_len, hq, hkv, page, lo, hi, top_k, cache):
    return dict(name=name, op="sparse", batch=batch, q_len=q_len, hq=hq, hkv=hkv, page=page, lo=lo, hi=hi, top_k=top_k,
                cache=cache)


def listed():
    return [
        # a short context's table with half of each head rotated: the smallest call
        _table("table 4K x 64", 4096, 64, 10000.0, 1.0),
        # a long context's table, made when a model is loaded or its scaling changes
        _table("table 128K x 128", 131072, 128, 500000.0, 8.0),
        # one request's next token: all latency
        _append("append 1 token bf16", 1, 1, 32, 8, 16, "bf16", 128, False, 4096),
        # a decode step of many requests into a 4-bit cache, interleaved pairs over half the head
        _append("append 256 tokens fp4", 256, 1, 64, 8, 16, "fp4", 64, True, 2048),
        # four prompts of an odd length into an FP8 cache
        _append("append 4 x 2039 fp8", 4, 2039, 32, 8, 64, "fp8", 128, False, 0),
        # digests of prompts that have just been read
        _digest("digest 16 ragged bf16", 16, 512, 32768, 8, 16, "bf16", 0),
        # one decode step's digests: one page of each request
        _digest("digest step 64 fp4", 64, 512, 8192, 8, 64, "fp4", 1),
        # one request, 4K tokens, contiguous: all latency
        _attend4("attend4 1 x 4K", 1, 1, False, 32, 8, 0, 4096, 4096),
        # ragged serving, paged: all bandwidth, the largest case
        _attend4("attend4 64 ragged", 64, 1, False, 32, 8, 16, 512, 32768),
        # speculative tokens under the causal mask, 16 query rows per KV head
        _attend4("attend4 32 x 4 causal", 32, 4, True, 32, 8, 16, 1024, 16384),
        # one long request over 64 of its 4096 pages
        _sparse("sparse 1 x 128K bf16", 1, 1, 32, 8, 32, 131072, 131072, 64, "bf16"),
        # long ragged requests over FP8 pages
        _sparse("sparse 32 ragged fp8", 32, 1, 32, 8, 32, 4096, 65536, 64, "fp8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "append", "append", "digest", "attend4", "attend4", "sparse", "sparse"])
    hkv = rng.choice([1, 2, 4, 8, 8])
    page = rng.choice([16, 16, 32, 48, 64, 128])
    if op == "table":
        rot = rng.choice([16, 32, 64, 80, 96, 112, 128])
        c = _table("", _log(rng, 512, 131072), rot, rng.choice([10000.0, 100000.0, 500000.0]), rng.choice([1.0, 2.0, 4.0, 8.0, 32.0]))
    elif op == "append":
        tokens = _log(rng, 1, 8192)
        q_len = rng.choice([1, 1, min(tokens, rng.randint(2, 8)), tokens])
        c = _append("", max(1, tokens // q_len), q_len, hkv * rng.choice([1, 2, 4, 5, 8]), hkv, page,
                    rng.choice(["bf16", "fp8", "fp4"]), rng.choice([16, 32, 64, 72, 96, 128, 128]), rng.random() < 0.4, _log(rng, 1, 4096))
    elif op == "digest":
        batch, hi = _log(rng, 1, 64), _log(rng, 64, 16384)
        c = _digest("", batch, rng.randint(1, hi), hi, hkv, page, rng.choice(["bf16", "fp8", "fp4"]), rng.choice([0, 0, 1, rng.randint(2, 9)]))
    elif op == "attend4":
        group, q_len = rng.choice([(1, 1), (4, 1), (8, 1), (4, 4), (2, 3), (7, 1), (16, 1), (8, 4), (8, 8), (5, 7), (16, 8)])
        batch = _log(rng, 1, 64)
        hi = _log(rng, 64, 524288 // batch if batch > 4 else 131072)
        c = _attend4("", batch, q_len, q_len > 1 and rng.random() < 0.7, hkv * group, hkv, rng.choice([0, page, page]),
                     rng.randint(q_len, max(q_len, hi)), hi)
    else:
        group, q_len = rng.choice([(1, 1), (4, 1), (4, 1), (8, 1), (4, 3), (7, 1), (2, 2), (16, 2)])
        batch = _log(rng, 1, 32)
        hi = _log(rng, 1024, 1048576 // batch if batch > 8 else 131072)
        c = _sparse("", batch, q_len, hkv * group, hkv, page, rng.randint(q_len + 100, hi), hi, rng.randint(4, 96), rng.choice(["bf16", "fp8", "fp4"]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _lengths(c, seed):
    """Tokens held by each request: the same set for every seed (so the same number of pages), in the seed's order."""
    lo, hi = (c["q_len"], c["q_len"] + c["past"]) if c["op"] == "append" else (c["lo"], c["hi"])
    r = random.Random(lo * 65536 + hi)
    n = [hi] + [r.randint(lo, hi) for _ in range(c["batch"] - 1)]
    random.Random(seed).shuffle(n)
    return n


def _randn(g, *shape, dtype=torch.bfloat16, std=1.0):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=g)


def _pages(c, lens, g):
    """A block table over shuffled pages; entries behind a request's last page are 0."""
    page = c["page"]
    need = [-(-n // page) for n in lens]
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
    """Values [pages, page, heads, 128] as a cache of `kind`: (bytes or bf16, block scales or None)."""
    if kind == "bf16":
        return x, None
    if kind == "fp8":
        return _scaled(x.float(), scale).clamp(-448, 448).to(E4M3).view(torch.uint8), None
    codes, sf = _fp4(x.float(), scale)
    return codes, sf.permute(0, 2, 1, 3).contiguous()


def _caches(c, kind, groups, tokens, g, want_v=True):
    """K and V of `groups` pages (or requests) of `tokens` each; the keys of a page lean its own way."""
    k = _randn(g, groups, tokens, c["hkv"], D, std=0.8)
    k += _randn(g, groups, 1, c["hkv"], D, std=0.6)
    st = {}
    st["k"], st["k_sf"] = _to_cache(k, kind, K_SCALE[kind])
    del k
    if want_v:
        st["v"], st["v_sf"] = _to_cache(_randn(g, groups, tokens, c["hkv"], D), kind, V_SCALE[kind])
    return st


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = dict(case=c)
    if c["op"] == "table":
        # by-parts scaling: slow pairs turn `factor` times slower, fast ones are left, a ramp between
        n = c["rot"] // 2
        base = c["base_lo"] * (1.0 + random.Random(seed).random())
        f = base ** (-torch.arange(n, dtype=torch.float64) / n)
        keep = ((8192.0 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        st["inv_freq"] = (f * (keep + (1 - keep) / c["factor"])).to(DEV)
        st["amplitude"] = 0.1 * math.log(c["factor"]) + 1.0
        return st
    kind = c.get("cache", "fp4")
    if c["op"] == "append":
        lens = _lengths(c, seed)
        st["block_table"], pages = _pages(c, lens, g)
        st.update(_caches(c, kind, pages, c["page"], g))
        heads = c["hq"] + 2 * c["hkv"]
        qkv = _randn(g, c["batch"], c["q_len"], heads, D)
        st["q"], st["k_new"], st["v_new"] = qkv[:, :, :c["hq"]], qkv[:, :, c["hq"]:c["hq"] + c["hkv"]], qkv[:, :, c["hq"] + c["hkv"]:]
        st["q_out"] = torch.empty_like(st["q"], memory_format=torch.contiguous_format)
        n = c["rot"] // 2
        ang = torch.arange(max(lens), dtype=torch.float64, device=DEV)[:, None] * 10000.0 ** (-torch.arange(n, dtype=torch.float64, device=DEV) / n)
        st["table"] = torch.cat([ang.cos(), ang.sin()], dim=1).float()
    else:
        lens = _lengths(c, seed)
        if c["page"]:
            st["block_table"], pages = _pages(c, lens, g)
            st.update(_caches(c, kind, pages, c["page"], g, want_v=c["op"] != "digest"))
        else:
            st["block_table"] = None
            st.update(_caches(c, kind, c["batch"], -(-max(lens) // 16) * 16, g))
        if c["op"] == "digest":
            st["digest"] = torch.zeros(pages, c["hkv"], 2, D, dtype=torch.int8, device=DEV)
            st["digest_scale"] = torch.zeros(pages, c["hkv"], dtype=torch.float32, device=DEV)
        else:
            st["q"] = _randn(g, c["batch"], c["q_len"], c["hq"], D, std=2.0)
        if c["op"] == "sparse":
            every = _values(st["k"], st["k_sf"], 1.0)
            st["digest"], st["digest_scale"] = _digest_of(every.amin(1), every.amax(1))
            del every
    st["max_len"] = max(lens)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    return st


# ------------------------------------------------------------------ the plain forms
def _num(x):
    return torch.full((), float(x), dtype=torch.float32, device=DEV)


def _scaled(x, scale):
    """x times the 32-bit reciprocal of the cache's scale."""
    return x * (_num(1.0) / _num(scale))


def _fp4(x, scale):
    """[..., 128] in 32 bits as (bytes [..., 64], block scales [..., 8]); ties to the even code."""
    y = _scaled(x, scale).unflatten(-1, (8, 16))
    sf = (y.abs().amax(-1) / _num(6)).clamp(max=448).to(E4M3)
    s = sf.float()[..., None]
    t = torch.where(s > 0, y / s, 0.0)
    a = t.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)) | (torch.signbit(t).to(torch.uint8) << 3)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), sf.view(torch.uint8)


def _pairs():
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    v = torch.cat([v, -v])
    byte = torch.arange(256, device=DEV)
    return torch.stack([v[byte % 16], v[byte // 16]], dim=1)


def _values(cache, sf, scale):
    """A cache [groups, tokens, heads, ...] as the 32-bit values it stands for."""
    if sf is not None:
        x = _pairs()[cache.int()].flatten(-2).unflatten(-1, (8, 16))
        return (x * (sf.permute(0, 2, 1, 3).contiguous().view(E4M3).float()[..., None] * scale)).flatten(-2)
    return (cache.view(E4M3).float() if cache.dtype == torch.uint8 else cache.float()) * scale


def _digest_of(lo, hi):
    """Minimum and maximum [pages, heads, 128] in 8 bits, and their scale."""
    amax = torch.maximum(lo.abs(), hi.abs()).amax(-1, keepdim=True)
    inv = torch.where(amax > 0, _num(127) / amax, 0.0)
    code = torch.stack([lo * inv, hi * inv], dim=2 if lo.dim() == 3 else -2).round().clamp(-127, 127).to(torch.int8)
    return code, (amax / _num(127))[..., 0]


def _rotate(x, cos, sin, rot, interleaved):
    y = x.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([torch.stack([u, v], dim=-1).flatten(-2) if interleaved else torch.cat([u, v], dim=-1), y[..., rot:]], dim=-1)
    return y.to(torch.bfloat16)


def _write(cache, sf, new, page, slot, kind, scale):
    if kind == "fp4":
        codes, s = _fp4(new.float(), scale)
        cache[page, slot] = codes
        sf.permute(0, 2, 1, 3)[page, slot] = s
    elif kind == "fp8":
        cache[page, slot] = _scaled(new.float(), scale).clamp(-448, 448).to(E4M3).view(torch.uint8)
    else:
        cache[page, slot] = new


def _softmax_rows(q, k, v, seen, scale):
    """Rows [..., R, 128] over keys [..., S, 128] where `seen` [..., R, S]: (out, log-sum-exp)."""
    s = torch.where(seen, torch.matmul(q, k.transpose(-1, -2)) * scale, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    n = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(n > 0, n, 1.0)
    return o, (m + torch.log(n))[..., 0]


def _gathered(cache, sf, table):
    """The pages of `table` [B, N] one behind the other: [B, N * page, heads, ...]."""
    at = table.long()
    return cache[at].flatten(1, 2), None if sf is None else sf[at].permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_table(st, c):
    ang = torch.arange(c["max_pos"], dtype=torch.float64, device=DEV)[:, None] * st["inv_freq"]
    return (torch.cat([ang.cos(), ang.sin()], dim=1) * st["amplitude"]).float()


def _plain_append(st, c):
    pos = st["lens"].long()[:, None] - c["q_len"] + torch.arange(c["q_len"], device=DEV)
    cos, sin = st["table"][pos][:, :, None].chunk(2, dim=-1)
    st["q_out"].copy_(_rotate(st["q"], cos, sin, c["rot"], c["interleaved"]))
    page, slot = torch.gather(st["block_table"].long(), 1, pos // c["page"]), pos % c["page"]
    _write(st["k"], st["k_sf"], _rotate(st["k_new"], cos, sin, c["rot"], c["interleaved"]), page, slot, c["cache"], K_SCALE[c["cache"]])
    _write(st["v"], st["v_sf"], st["v_new"], page, slot, c["cache"], V_SCALE[c["cache"]])


def _plain_digest(st, c):
    table, lens = st["block_table"].long(), st["lens"].long()[:, None]
    held = torch.arange(table.shape[1], device=DEV) * c["page"]
    first = (lens - c["new"]).clamp(min=0) if c["new"] else torch.zeros_like(lens)
    here = (held < lens) & (held + c["page"] > first)
    row = here.nonzero()
    page = table[here]
    x = _values(st["k"][page], None if st["k_sf"] is None else st["k_sf"][page], 1.0)
    seen = (held[row[:, 1]][:, None] + torch.arange(c["page"], device=DEV) < lens[row[:, 0]])[:, :, None, None]
    lo, hi = torch.where(seen, x, math.inf).amin(1), torch.where(seen, x, -math.inf).amax(1)
    st["digest"][page], st["digest_scale"][page] = _digest_of(lo, hi)


def _plain_attend4(st, c):
    b, t, hkv = c["batch"], c["q_len"], c["hkv"]
    k, v, k_sf, v_sf = st["k"], st["v"], st["k_sf"], st["v_sf"]
    if st["block_table"] is not None:
        k, k_sf = _gathered(k, k_sf, st["block_table"])
        v, v_sf = _gathered(v, v_sf, st["block_table"])
    k, v = _values(k, k_sf, K_SCALE["fp4"]).transpose(1, 2), _values(v, v_sf, V_SCALE["fp4"]).transpose(1, 2)
    q = st["q"].float().view(b, t, hkv, -1, D).permute(0, 2, 1, 3, 4)
    at = torch.arange(k.shape[2], device=DEV)
    last = st["lens"].long()[:, None] - (t - 1 - torch.arange(t, device=DEV) if c["causal"] else 0 * torch.arange(t, device=DEV))
    seen = (at < last[:, :, None])[:, None, :, None].expand(b, 1, t, q.shape[3], k.shape[2]).flatten(2, 3)
    o, lse = _softmax_rows(q.flatten(2, 3), k, v, seen, 1.0 / math.sqrt(D))
    o = o.unflatten(2, (t, -1)).permute(0, 2, 1, 3, 4).reshape(b, t, c["hq"], D)
    return o.to(torch.bfloat16), lse.unflatten(2, (t, -1)).permute(0, 2, 1, 3).reshape(b, t, c["hq"])


def _plain_sparse(st, c):
    b, t, hkv, page, kind = c["batch"], c["q_len"], c["hkv"], c["page"], c["cache"]
    q = st["q"].float().view(b, t, hkv, -1, D)
    table = st["block_table"].long()
    nb = table.shape[1]
    # scores: whole numbers below 2^24 until the two scales come in, so exact in 32 bits
    amax = q.abs().amax(-1, keepdim=True)
    qi = (q * torch.where(amax > 0, _num(127) / amax, 0.0)).round()
    dg = st["digest"][table].float()
    dot = torch.einsum("btkgd,bnkd->btkgn", qi.clamp(max=0), dg[:, :, :, 0]) + torch.einsum("btkgd,bnkd->btkgn", qi.clamp(min=0), dg[:, :, :, 1])
    score = ((dot * st["digest_scale"][table].permute(0, 2, 1)[:, None, :, None]) * (amax / _num(127))).amax(3)
    # the first page and the last always, then the best; ties to the lowest page
    seen_len = st["lens"].long()[:, None] - (t - 1) + torch.arange(t, device=DEV)
    count = ((seen_len + page - 1) // page)[:, :, None, None]
    at = torch.arange(nb, device=DEV)
    score = torch.where((at == 0) | (at == count - 1), math.inf, torch.where(at < count, score, -math.inf))
    n = min(c["top_k"], nb)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :n]
    order = torch.where(torch.arange(n, device=DEV) < count, order, nb).sort(-1).values
    held = order < nb
    idx = torch.where(held, order, 0)
    # the chosen pages' keys and values
    phys = torch.gather(table[:, None, None].expand(b, t, hkv, nb), 3, idx)
    head = torch.arange(hkv, device=DEV)[None, None, :, None]
    k, v = st["k"][phys, :, head], st["v"][phys, :, head]
    k_sf = v_sf = None
    if kind == "fp4":
        k_sf, v_sf = st["k_sf"][phys, head].flatten(3, 4), st["v_sf"][phys, head].flatten(3, 4)
    k, v = (_sparse_values(x.flatten(3, 4), s, w[kind]) for x, s, w in ((k, k_sf, K_SCALE), (v, v_sf, V_SCALE)))
    pos = (idx[..., None] * page + torch.arange(page, device=DEV))
    seen = (held[..., None] & (pos < seen_len[:, :, None, None, None])).flatten(3, 4)[:, :, :, None]
    o, lse = _softmax_rows(q, k, v, seen, 1.0 / math.sqrt(D))
    blocks = torch.full((b, t, hkv, c["top_k"]), -1, dtype=torch.int32, device=DEV)
    blocks[..., :n] = torch.where(held, order, -1).to(torch.int32)
    return o.reshape(b, t, c["hq"], D).to(torch.bfloat16), lse.reshape(b, t, c["hq"]), blocks


def _sparse_values(x, sf, scale):
    if sf is not None:
        x = _pairs()[x.int()].flatten(-2).unflatten(-1, (8, 16))
        return (x * (sf.view(E4M3).float()[..., None] * scale)).flatten(-2)
    return (x.view(E4M3).float() if x.dtype == torch.uint8 else x.float()) * scale


# ------------------------------------------------------------------ one pass
def _own(st, c):
    from split_kv_decode_attention_gb300 import binding as da
    if c["op"] == "table":
        return da.rope_table(st["inv_freq"], c["max_pos"], amplitude=st["amplitude"])
    kind = c.get("cache", "fp4")
    scales = dict(k_scale=K_SCALE[kind], v_scale=V_SCALE[kind], k_sf=st["k_sf"], v_sf=st.get("v_sf"))
    if c["op"] == "append":
        da.rope_append(st["q"], st["k_new"], st["v_new"], st["table"], st["k"], st["v"], st["block_table"], st["lens"],
                       max_seq_len=st["max_len"], interleaved=c["interleaved"], q_out=st["q_out"], **scales)
    elif c["op"] == "digest":
        da.block_digest(st["k"], st["block_table"], st["lens"], st["digest"], st["digest_scale"], max_seq_len=st["max_len"],
                        max_new=c["new"], k_sf=st["k_sf"])
    elif c["op"] == "attend4":
        return da.decode_attn(st["q"], st["k"], st["v"], st["block_table"], st["lens"], max_seq_len=st["max_len"],
                              causal=c["causal"], **scales)
    else:
        return da.decode_attn_sparse(st["q"], st["k"], st["v"], st["block_table"], st["lens"], st["digest"], st["digest_scale"],
                                     max_seq_len=st["max_len"], top_k=c["top_k"], causal=True, **scales)


def run(state):
    c = state["case"]
    if own:
        r = _own(state, c)
    else:
        r = {"table": _plain_table, "append": _plain_append, "digest": _plain_digest, "attend4": _plain_attend4,
             "sparse": _plain_sparse}[c["op"]](state, c)
    if c["op"] == "append":
        # the cache's own bytes: they have to be equal, which is more than the values they stand for
        held = {n: state[n] for n in ("k", "v", "k_sf", "v_sf") if state[n] is not None}
        return dict(held, q=state["q_out"])
    if c["op"] == "digest":
        return dict(digest=state["digest"], scale=state["digest_scale"])
    return dict(table=r) if c["op"] == "table" else dict(zip(("out", "lse", "blocks"), r))


# ------------------------------------------------------------------ 64 bits, from the definitions
def _fp4_64(codes, sf):
    """Bytes [T, 64] and block scales [T, 8] as 64-bit values [T, 128]."""
    nib = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(codes.shape[0], D).to(torch.float64)
    sign, mag = torch.where(nib >= 8, -1.0, 1.0).to(torch.float64), nib % 8
    e, m = (mag / 2).floor(), mag % 2
    val = torch.where(e == 0, m * 0.5, (1 + m / 2) * torch.pow(torch.full_like(e, 2.0), e - 1)) * sign
    return val * sf.view(E4M3).to(torch.float64).repeat_interleave(16, dim=1)


def _head_64(st, which, kind, scale, b, h, n, pick=None):
    """The first n tokens (or those of the pages `pick`) of request b, head h, in 64 bits."""
    cache, sf = st[which], st[which + "_sf"]
    if st["block_table"] is None:
        x, s = cache[b, :, h], None if sf is None else sf[b, h]
    else:
        at = st["block_table"][b].long() if pick is None else st["block_table"][b].long()[pick]
        x, s = cache[at, :, h].flatten(0, 1), None if sf is None else sf[at, h].flatten(0, 1)
    x, s = x[:n], None if s is None else s[:n]
    v = _fp4_64(x, s) if kind == "fp4" else x.view(E4M3).double() if kind == "fp8" else x.double()
    return v * scale


def _row_64(q, k, v):
    """One query over its keys: out and log-sum-exp."""
    s = (k @ q) / math.sqrt(D)
    lse = torch.logsumexp(s, 0)
    return torch.exp(s - lse) @ v, lse


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    if c["op"] == "table":
        out = torch.empty(c["max_pos"], c["rot"], dtype=torch.float64, device=DEV)
        for i, f in enumerate(st["inv_freq"].tolist()):
            a = torch.arange(c["max_pos"], dtype=torch.float64, device=DEV) * f
            out[:, i], out[:, i + c["rot"] // 2] = torch.cos(a) * st["amplitude"], torch.sin(a) * st["amplitude"]
        return dict(table=out)
    lens = st["lens"].tolist()
    if c["op"] == "append":
        rot, T = c["rot"], c["q_len"]
        first = (torch.arange(rot // 2, device=DEV) * 2) if c["interleaved"] else torch.arange(rot // 2, device=DEV)
        second = first + (1 if c["interleaved"] else rot // 2)
        q, kn = st["q"].double().clone(), st["k_new"].double().clone()
        for b, n in enumerate(lens):
            z = torch.complex(st["table"][n - T:n, :rot // 2].double(), st["table"][n - T:n, rot // 2:].double())[:, None]
            for x in (q[b], kn[b]):
                w = torch.complex(x[..., first].clone(), x[..., second].clone()) * z
                x[..., first], x[..., second] = w.real, w.imag
        k = v = None
        if c["cache"] == "bf16":
            k, v = st["k"].double(), st["v"].double()
            for b, n in enumerate(lens):
                p = torch.arange(n - T, n, device=DEV)
                at = st["block_table"][b].long()[p // c["page"]]
                k[at, p % c["page"]], v[at, p % c["page"]] = kn[b], st["v_new"][b].double()
        return dict(k=k, v=v, q=q, **({"k_sf": None, "v_sf": None} if c["cache"] == "fp4" else {}))
    if c["op"] == "digest":
        scale = st["digest_scale"].double()
        for b, n in enumerate(lens):
            for h in range(c["hkv"]):
                x = _head_64(st, "k", c["cache"], 1.0, b, h, n).abs().amax(1)
                pages = -(-n // c["page"])
                x = torch.nn.functional.pad(x, (0, pages * c["page"] - n)).view(pages, c["page"]).amax(1) / 127
                lo = max(0, n - c["new"]) // c["page"] if c["new"] else 0
                scale[st["block_table"][b].long()[lo:pages], h] = x[lo:]
        return dict(digest=None, scale=scale)
    group, T, kind = c["hq"] // c["hkv"], c["q_len"], c.get("cache", "fp4")
    if c["batch"] * c["hkv"] * (T * group if c["op"] == "attend4" else T * group * 4) > 12000:
        return None
    out = torch.zeros(c["batch"], T, c["hq"], D, dtype=torch.float64, device=DEV)
    lse = torch.full((c["batch"], T, c["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    q = st["q"].double()
    for b, n in enumerate(lens):
        for h in range(c["hkv"]):
            if c["op"] == "attend4":
                k, v = (_head_64(st, x, kind, w[kind], b, h, n) for x, w in (("k", K_SCALE), ("v", V_SCALE)))
            for t in range(T):
                m = n - T + 1 + t if c["op"] == "sparse" or c["causal"] else n
                if m < 1:
                    continue
                if c["op"] == "sparse":
                    pick, m = _picked_64(st, c, b, h, t, m)
                    k, v = (_head_64(st, x, kind, w[kind], b, h, m, pick) for x, w in (("k", K_SCALE), ("v", V_SCALE)))
                for j in range(h * group, (h + 1) * group):
                    out[b, t, j], lse[b, t, j] = _row_64(q[b, t, j], k[:m], v[:m])
    return dict(out=out, lse=lse, **({"blocks": None} if c["op"] == "sparse" else {}))


def _picked_64(st, c, b, h, t, m):
    """The pages of token t of request b, head h (m tokens seen), in order; and how many tokens they hold."""
    count = -(-m // c["page"])
    at = st["block_table"][b, :count].long()
    lo, hi = st["digest"][at, h, 0].double(), st["digest"][at, h, 1].double()
    best = None
    group = c["hq"] // c["hkv"]
    for j in range(h * group, (h + 1) * group):
        q = st["q"][b, t, j].float()
        top = q.abs().max()
        qi = torch.round(q * (_num(127) / top)).double()  # 8 bits, in 32-bit steps as the definition has it
        dot = torch.maximum(qi * lo, qi * hi).sum(1).float()
        s = (dot * st["digest_scale"][at, h]) * (top / _num(127))
        best = s if best is None else torch.maximum(best, s)
    best[0] = best[-1] = math.inf
    n = min(c["top_k"], count)
    pick = torch.sort(best, descending=True, stable=True).indices[:n].sort().values
    return pick, n * c["page"] - (count * c["page"] - m)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "table":
        n = c["max_pos"] * c["rot"]
        return dict(bytes=4 * n + 4 * c["rot"], flops=2 * n)
    row = {"bf16": 2 * D, "fp8": D, "fp4": D // 2 + D // 16}[c.get("cache", "fp4")]
    if c["op"] == "append":
        t = c["batch"] * c["q_len"]
        return dict(bytes=t * (4 * D * (c["hq"] + c["hkv"]) + 2 * c["hkv"] * row + 4 * c["rot"] + 4), flops=t * (c["hq"] + c["hkv"]) * c["rot"] * 3)
    lens = _lengths(c, 0)
    tokens = sum(lens)
    if c["op"] == "digest":
        first = [max(0, n - c["new"]) // c["page"] if c["new"] else 0 for n in lens]
        tokens = sum(n - f * c["page"] for n, f in zip(lens, first))
        pages = sum(-(-n // c["page"]) - f for n, f in zip(lens, first))
        return dict(bytes=c["hkv"] * (tokens * row + pages * (2 * D + 4)) + 4 * pages, flops=2 * tokens * c["hkv"] * D)
    rows = c["batch"] * c["q_len"] * c["hq"]
    if c["op"] == "attend4":
        return dict(bytes=2 * tokens * c["hkv"] * row + rows * (4 * D + 4), flops=4 * D * tokens * c["q_len"] * c["hq"])
    pages = sum(-(-n // c["page"]) for n in lens)
    seen = sum(min(n, c["top_k"] * c["page"]) for n in lens) * c["q_len"]
    return dict(bytes=pages * (c["hkv"] * (2 * D + 4) + 4) + 2 * min(seen, tokens) * c["hkv"] * row + rows * (4 * D + 4) + 4 * rows * c["hkv"] / c["hq"] * c["top_k"],
                flops=4 * D * pages * c["q_len"] * c["hq"] + 4 * D * seen * c["hq"])
