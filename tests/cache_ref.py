"""Plain CPU references of the operators around the cache (torch, 64 bits, or
32 bits where the definition says how each step rounds)."""
import math

import torch

D = 128
E4M3 = torch.float8_e4m3fn
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def f32(x):
    return torch.tensor(float(x), dtype=torch.float32)


def to_e4m3(x):
    """fp32 -> E4M3 bytes, saturating (NaN stays NaN)."""
    return torch.where(x.isnan(), x, x.clamp(-448.0, 448.0)).to(E4M3).view(torch.uint8)


def quant_fp4(x, scale):
    """bf16 [..., 128] -> (bytes [..., 64], block scales [..., 8]): the definition."""
    z = (x.float() * (f32(1.0) / f32(scale))).unflatten(-1, (8, 16))
    z = torch.where(z.isnan(), 0.0, z)
    sf = to_e4m3(z.abs().amax(-1) / f32(6.0))
    s = sf.view(E4M3).float()[..., None]
    t = torch.where(s > 0, z / s, 0.0)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    a = t.abs()[..., None]
    # ties to even: below or at the midpoints before codes 1, 3, 5, 7
    past = torch.where(torch.arange(7) % 2 == 0, a > mids, a >= mids)
    code = past.sum(-1).to(torch.uint8) | (torch.signbit(t).to(torch.uint8) << 3)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), sf


def fp4_values(codes, sf):
    """Bytes [..., 64] and block scales [..., 8] -> 64-bit values [..., 128]."""
    n = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).long()
    v = E2M1[n & 7] * torch.where(n >= 8, -1.0, 1.0).double()
    return v * sf.view(E4M3).double().repeat_interleave(16, dim=-1)


def rotate(x, cos, sin, rot, interleaved, dtype):
    """bf16 [..., 128] -> rotated values in `dtype` (each step rounds to it)."""
    y = x.to(dtype).clone()
    cos, sin = cos.to(dtype), sin.to(dtype)
    first = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    second = first + 1 if interleaved else first + rot // 2
    a, b = y[..., first].clone(), y[..., second].clone()
    y[..., first] = a * cos - b * sin
    y[..., second] = b * cos + a * sin
    return y


def cache_values(kind, cache, sf):
    """A CPU cache [G, S, H, ...] (block scales [G, H, S, 8]) as 64-bit values, unscaled."""
    if kind == "fp4":
        return fp4_values(cache, sf.permute(0, 2, 1, 3).contiguous())
    if kind == "fp8":
        return cache.view(E4M3).double()
    return cache.double()


def gather(values, block_table, b, n):
    """Request b's first n tokens [n, H, 128] of paged or contiguous values."""
    if block_table is None:
        return values[b, :n]
    ps = values.shape[1]
    pages = block_table[b, :-(-n // ps)].long() if n > 0 else block_table[b, :0].long()
    return values[pages].flatten(0, 1)[:n]


def attention_rows(q, k, v, seen, scale):
    """q [R, 128], k / v [n, 128] (all 64 bits), seen [R, n] -> out, lse, and the bounds
    that error estimates need: sum_j w_j |v_j| and max_j scale * sum_d |q_d k_d|."""
    s = (q @ k.T) * scale
    s = torch.where(seen, s, -math.inf)
    lse = torch.logsumexp(s, 1) if k.shape[0] else torch.full((q.shape[0],), -math.inf).double()
    w = torch.where(seen, torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[:, None]), 0.0)
    mag = torch.where(seen, (q.abs() @ k.abs().T) * abs(scale), 0.0)
    top = mag.amax(1) if k.shape[0] else torch.zeros(q.shape[0]).double()
    return w @ v, lse, w @ v.abs(), top


def out_tolerance(out, wabs, mag):
    """|error| a bf16 output may have.  Its own rounding: 2^-8 |out|.  P rounded to
    f16: 2^-11 of each weight.  A score: 128 exact products added in fp32, each sum
    off by at most 2^-23 of the running magnitude: 2^-16 sum |q k| scale, entering
    the weights and their normalisation (twice); exponentials, rescalings and the
    sums of weights: under 2^-18."""
    rel = 2.0 ** -11 + 2 * 2.0 ** -16 * mag + 2.0 ** -18
    return 2.0 ** -8 * out.abs() + rel[..., None] * wabs + 1e-30


def bf16_p_tolerance(out, wabs, mag):
    """The same where P is rounded to bf16 (2^-8 of each weight, and of the sums of the
    rounded weights that normalise them)."""
    rel = 2 * 2.0 ** -8 + 2 * 2.0 ** -16 * mag + 2.0 ** -18
    return 2.0 ** -8 * out.abs() + rel[..., None] * wabs + 1e-30


def lse_tolerance(lse, mag):
    return 2.0 ** -16 * mag + 2.0 ** -18 + 2.0 ** -22 * torch.where(lse.isinf(), 0.0, lse).abs()


def digest_page(x):
    """Keys [n, 128] of one page (fp32 values) -> (min, max codes int8 [2, 128], scale)."""
    big = 3.3895313892515355e38
    nan = x.isnan()
    lo = torch.where(nan, math.inf, x).amin(0)
    hi = torch.where(nan, -math.inf, x).amax(0)
    none = lo > hi
    lo = torch.where(none, 0.0, lo.clamp(-big, big))
    hi = torch.where(none, 0.0, hi.clamp(-big, big))
    amax = torch.maximum(lo.abs(), hi.abs()).amax()
    inv = f32(127.0) / amax if amax > 0 else f32(0.0)
    code = (torch.stack([lo, hi]) * inv).round().clamp(-127, 127).to(torch.int8)
    return code, amax / f32(127.0)


def page_scores(q, digest, dscale):
    """q bf16 [G, 128], digests int8 [n, 2, 128], scales fp32 [n] -> fp32 scores [n]."""
    big = 3.3895313892515355e38
    best = None
    for row in q.float():
        row = torch.where(row.isnan(), 0.0, row.clamp(-big, big))
        a = row.abs().amax()
        inv = f32(127.0) / a if a > 0 else f32(0.0)
        qi = (row * inv).round().clamp(-127, 127).to(torch.int64)
        dg = digest.to(torch.int64)
        dot = (qi.clamp(max=0) * dg[:, 0] + qi.clamp(min=0) * dg[:, 1]).sum(1).float()
        s = (dot * dscale) * (a / f32(127.0))
        best = s if best is None else torch.maximum(best, s)
    return best


def pick(scores, top_k, sink, local):
    """Ascending places of the selected pages among scores [n]."""
    n = scores.shape[0]
    if n <= top_k:
        return torch.arange(n)
    s = scores.double().clamp(-1e300, 1e300)  # (a score may be infinite; the forced pages still come first)
    s[:sink] = math.inf
    s[n - local:] = math.inf
    return torch.sort(s, descending=True, stable=True).indices[:top_k].sort().values
