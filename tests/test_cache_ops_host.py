"""Host-side checks of the operators around the cache: struct layouts, refusals
before anything touches a GPU, and the frequencies of the rotary scalings."""
import ctypes
import math

import pytest

from split_kv_decode_attention_gb300 import binding as da
from split_kv_decode_attention_gb300 import build as cuda_build

NO_DEVICE_OR_OK = (0, -8, -9)  # what a call with good arguments may give here


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return da.lib()


def test_struct_sizes():
    assert ctypes.sizeof(da.DecodeAttnCache) == 56
    assert ctypes.sizeof(da.DecodeAttnRope) == 64
    assert ctypes.sizeof(da.DecodeAttnSelect) == 16


def params(fp4=True, **kw):
    p = da.decode_attn_params_init(2, 1, 8, 2, 128, 16, 4, 10, 64, False)
    if fp4:
        p.kv_stride_page, p.kv_stride_token, p.kv_stride_head = 16 * 2 * 64, 2 * 64, 64
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def cache(ctype=da.DA_CACHE_FP4_E2M1, **kw):
    c = da.DecodeAttnCache()
    c.type = ctype
    c.k = c.v = c.k_block_scale = c.v_block_scale = 1 << 20
    c.bs_stride_page, c.bs_stride_head = 2 * 16 * 8, 16 * 8
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def ref(x):
    return None if x is None else ctypes.byref(x)


A = 1 << 20  # an aligned address that no refused call reads


def attend(lib, p, c, q=A, bt=A, lens=A, out=A, lse=A, splits=1):
    return lib.decode_attn_cached(ref(p), ref(c), q, bt, lens, out, lse, splits, None, 0, None, None)


@pytest.mark.parametrize("c_kw,p_kw,call_kw,code", [
    (dict(type=7), {}, {}, -12), (dict(reserved=1), {}, {}, -2), (dict(k=0), {}, {}, -1),
    (dict(v_block_scale=0), {}, {}, -1), (dict(k=A + 8), {}, {}, -6), (dict(k_block_scale=A + 4), {}, {}, -6),
    (dict(bs_stride_head=12), {}, {}, -6), (dict(bs_stride_page=0), {}, {}, -6),
    ({}, dict(kv_stride_token=72), {}, -6), ({}, dict(k_scale=math.inf), {}, -2), ({}, dict(v_scale=math.nan), {}, -2),
    ({}, dict(head_dim=64), {}, -3), ({}, dict(page_size=24), {}, -4), ({}, dict(num_q_heads=2 * 129), {}, -5),
    ({}, {}, dict(q=None), -1), ({}, {}, dict(q=A + 2), -6), ({}, {}, dict(lens=None), -1), ({}, {}, dict(out=None), -1),
    ({}, dict(flags=4), {}, -2)])
def test_fp4_attention_refusals(lib, c_kw, p_kw, call_kw, code):
    assert attend(lib, params(**p_kw), cache(**c_kw), **call_kw) == code


def test_null_descriptors(lib):
    assert attend(lib, None, cache()) == -1
    assert attend(lib, params(), None) == -1
    n = ctypes.c_size_t()
    assert lib.decode_attn_cached_workspace_bytes(ref(params()), None, 1, ctypes.byref(n)) == -1
    assert lib.decode_attn_cached_workspace_bytes(ref(params()), ref(cache()), 2, None) == -1


def test_workspace_of_explicit_splits_needs_no_device(lib):
    n = ctypes.c_size_t()
    p = params(max_pages_per_seq=20, block_table_stride=20, max_seq_len=250)
    assert lib.decode_attn_cached_workspace_bytes(ref(p), ref(cache()), 4, ctypes.byref(n)) == 0
    assert n.value == 2 * 8 * 4 * 129 * 4        # chunks of 64 tokens
    assert lib.decode_attn_cached_workspace_bytes(ref(p), ref(cache()), 3, ctypes.byref(n)) == 0
    assert n.value == 2 * 8 * 2 * 129 * 4        # 84 tokens round up to 128: two chunks
    assert lib.decode_attn_cached_workspace_bytes(ref(p), ref(cache()), 1, ctypes.byref(n)) == 0
    assert n.value == 0


def test_type_of_the_cache_counts_not_the_flag(lib):
    """bf16 strides that are no multiple of 16 bytes per element size stay refused as bf16."""
    p = params(fp4=False, flags=da.DA_FLAG_KV_FP8_E4M3, kv_stride_head=8)   # 8 bytes as FP8: refused, 16 as bf16
    assert attend(lib, p, cache(da.DA_CACHE_BF16)) in NO_DEVICE_OR_OK
    assert attend(lib, p, cache(da.DA_CACHE_FP8_E4M3)) == -6


def rope(**kw):
    r = da.DecodeAttnRope()
    r.rotary_dim, r.table_positions = 64, 100
    for n in ("k", "v"):
        setattr(r, n + "_stride_batch", 256)
        setattr(r, n + "_stride_token", 256)
        setattr(r, n + "_stride_head", 128)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def append(lib, p=None, c=None, r=None, q=A, k=A, v=A, table=A, positions=None, new_lens=None, bt=A, lens=A, q_out=A):
    return lib.decode_attn_rope_append(ref(p or params()), ref(c or cache()), ref(r or rope()), q, k, v, table, positions,
                                       new_lens, bt, lens, q_out, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(r=rope(rotary_dim=3)), -2), (dict(r=rope(rotary_dim=130)), -2), (dict(r=rope(rotary_dim=-2)), -2),
    (dict(r=rope(reserved=1)), -2), (dict(r=rope(table_positions=-1)), -2), (dict(r=rope(k_stride_token=12)), -6),
    (dict(r=rope(v_stride_batch=0)), -6), (dict(table=None), -1), (dict(table=A + 4), -6), (dict(lens=None), -1),
    (dict(q=None), -1), (dict(q_out=None), -1), (dict(v=None), -1), (dict(k=None), -1),
    (dict(q=None, q_out=None, k=None, v=None), -1), (dict(k=A + 8), -6), (dict(positions=A + 2), -6),
    (dict(p=params(k_scale=0.0)), -2), (dict(p=params(v_scale=math.nan)), -2), (dict(p=params(v_scale=1e-39)), -2), (dict(c=cache(v=0)), -1),
    (dict(p=params(q_stride_token=4)), -6), (dict(p=params(max_seq_len=65)), -2), (dict(p=params(q_len=0)), -2)])
def test_append_refusals(lib, kw, code):
    assert append(lib, **kw) == code


def test_append_takes_any_number_of_tokens(lib):
    assert append(lib, p=params(q_len=5000)) in NO_DEVICE_OR_OK
    assert append(lib, p=params(batch=60000, q_len=60000)) == -2
    assert append(lib, p=params(batch=0), q=None, k=None) == 0


def digest(lib, p=None, c=None, bt=A, lens=A, new=0, dg=A, ds=A):
    return lib.decode_attn_block_digest(ref(p or params()), ref(c or cache()), bt, lens, new, dg, ds, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(bt=None), -1), (dict(lens=None), -1), (dict(dg=None), -1), (dict(ds=None), -1), (dict(dg=A + 8), -6),
    (dict(new=-1), -2), (dict(p=params(page_size=0)), -4), (dict(c=cache(k=0)), -1), (dict(c=cache(type=-1)), -12)])
def test_digest_refusals(lib, kw, code):
    assert digest(lib, **kw) == code


def test_digest_needs_no_v(lib):
    assert digest(lib, c=cache(v=0, v_block_scale=0)) in NO_DEVICE_OR_OK


def select(**kw):
    s = da.DecodeAttnSelect()
    s.top_k, s.sink, s.local = 3, 1, 1
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def sparse(lib, p=None, c=None, s=None, q=A, dg=A, ds=A, bt=A, lens=A, out=A, lse=A, blocks=None):
    return lib.decode_attn_sparse(ref(p or params()), ref(c or cache()), ref(s or select()), q, dg, ds, bt, lens, out, lse,
                                  blocks, None, 0, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(s=select(top_k=0)), -2), (dict(s=select(top_k=4097)), -2), (dict(s=select(local=0)), -2),
    (dict(s=select(sink=-1)), -2), (dict(s=select(sink=2, local=2)), -2), (dict(s=select(reserved=1)), -2),
    (dict(p=params(scale=0.0)), -2), (dict(p=params(scale=-1.0)), -2), (dict(p=params(k_scale=-1.0)), -2),
    (dict(p=params(page_size=0)), -4), (dict(bt=None), -1), (dict(dg=None), -1), (dict(ds=A + 2), -6),
    (dict(out=None), -1), (dict(lse=A + 2), -6), (dict(blocks=A + 2), -6), (dict(q=A + 8), -6), (dict(c=cache(v=0)), -1),
    (dict(p=params(q_len=2, q_stride_batch=8 * 128)), -2), (dict(p=params(batch=40000, q_len=2, num_q_heads=2)), -2)])
def test_sparse_refusals(lib, kw, code):
    assert sparse(lib, **kw) == code


def test_select_refusals_and_workspace(lib):
    p, n = params(), ctypes.c_size_t()
    assert lib.decode_attn_block_select_workspace_bytes(ref(p), ref(select()), ctypes.byref(n)) == 0
    assert n.value == 2 * 1 * 2 * 4 * 4          # rows x pages (rounded up to 4) x 4 bytes
    assert lib.decode_attn_block_select_workspace_bytes(ref(p), ref(select(top_k=4)), ctypes.byref(n)) == 0
    assert n.value == 0                          # every page is taken
    args = [ref(p), ref(select()), A, A, A, A, A, None, A, A, A, 64, None, None]
    assert lib.decode_attn_block_select(*args) in NO_DEVICE_OR_OK
    for i, code in ((2, -1), (3, -1), (5, -1), (6, -1), (8, -1), (9, -1), (10, -7)):
        bad = list(args)
        bad[i] = None
        assert lib.decode_attn_block_select(*bad) == code, i
    bad = list(args)
    bad[11] = 63
    assert lib.decode_attn_block_select(*bad) == -7


@pytest.mark.parametrize("args,code", [
    ((A, 0, 0, 10, 1.0, A), -2), ((A, 65, 0, 10, 1.0, A), -2), ((A, 8, -1, 10, 1.0, A), -2), ((A, 8, 0, -1, 1.0, A), -2),
    ((A, 8, 1, 1 << 31, 1.0, A), -2), ((None, 8, 0, 10, 1.0, A), -1), ((A, 8, 0, 10, 1.0, None), -1),
    ((A + 4, 8, 0, 10, 1.0, A), -6), ((None, 8, 0, 0, 1.0, None), 0)])
def test_rope_table_refusals(lib, args, code):
    assert lib.decode_attn_rope_table(*args, None) == code


# ------------------------------------------------------------------ the Python entry points
torch = pytest.importorskip("torch")


def test_python_refusals():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.uint8)
    sf = torch.zeros(4, 2, 16, 8, dtype=torch.uint8)
    bt = torch.zeros(1, 2, dtype=torch.int32)
    lens = torch.ones(1, dtype=torch.int32)
    q = torch.zeros(1, 1, 4, 128, dtype=torch.bfloat16)
    kw = dict(max_seq_len=32)
    for bad in (dict(k_sf=sf), dict(k_sf=sf[:, :1], v_sf=sf[:, :1]), dict(k_sf=sf.float(), v_sf=sf)):
        with pytest.raises(ValueError):
            da.decode_attn(q, k, k, bt, lens, **kw, **bad)
    with pytest.raises(ValueError):          # 128 wide, not 64
        da.decode_attn(q, torch.zeros(4, 16, 2, 128, dtype=torch.uint8), k, bt, lens, k_sf=sf, v_sf=sf, **kw)
    with pytest.raises(ValueError):
        da.decode_attn(q, k, k, bt.long(), lens, k_sf=sf, v_sf=sf, **kw)
    with pytest.raises(ValueError):
        da.decode_attn(q.float(), k, k, bt, lens, k_sf=sf, v_sf=sf, **kw)
    new = torch.zeros(1, 1, 2, 128, dtype=torch.bfloat16)
    for args in ((None, None, None), (None, new, None), (q, new[..., :1, :], new)):
        with pytest.raises(ValueError):
            da.rope_append(*args, None, k, k, bt, lens, k_sf=sf, v_sf=sf, **kw)
    with pytest.raises(ValueError):          # 3 query heads over 2
        da.rope_append(q[:, :, :3], new, new, None, k, k, bt, lens, k_sf=sf, v_sf=sf, **kw)
    with pytest.raises(ValueError):
        da.block_digest(k, None, lens, k_sf=sf, **kw)
    dg, ds = torch.zeros(4, 2, 2, 128, dtype=torch.int8), torch.zeros(4, 2)
    with pytest.raises(ValueError):
        da.decode_attn_sparse(q, k, k, bt, lens, dg[:3], ds, top_k=2, k_sf=sf, v_sf=sf, **kw)
    with pytest.raises(ValueError):
        da.rope_table(torch.zeros(3), 4)


def test_rope_frequencies():
    f, amp = da.rope_frequencies(64)
    i = torch.arange(32, dtype=torch.float64)
    assert amp == 1.0 and torch.allclose(f, 10000.0 ** (-i / 32), rtol=1e-14, atol=0)
    f2, _ = da.rope_frequencies(64, scaling="linear", factor=4.0)
    assert torch.allclose(f2, f / 4, rtol=1e-14, atol=0)
    f3, _ = da.rope_frequencies(64, scaling="ntk", factor=4.0)
    assert float(f3[0]) == 1.0 and abs(float(f3[-1] * 4 / f[-1]) - 1) < 1e-12
    f4, _ = da.rope_frequencies(128, base=500000.0, scaling="by_parts", factor=8.0, original_positions=8192)
    g, _ = da.rope_frequencies(128, base=500000.0)
    turns = 8192 * g / (2 * math.pi)
    assert torch.equal(f4[turns >= 4], g[turns >= 4])
    assert torch.allclose(f4[turns <= 1], g[turns <= 1] / 8, rtol=1e-14, atol=0)
    mid = (turns > 1) & (turns < 4)
    assert bool(mid.any()) and bool(((f4 < g) & (f4 > g / 8))[mid].all())
    f5, amp = da.rope_frequencies(128, scaling="yarn", factor=16.0, original_positions=4096)
    h, _ = da.rope_frequencies(128)
    turns = 4096 * h / (2 * math.pi)
    assert abs(amp - (0.1 * math.log(16) + 1)) < 1e-15
    assert torch.equal(f5[turns > 33], h[turns > 33]) and torch.allclose(f5[turns < 0.8], h[turns < 0.8] / 16, rtol=1e-14)
    assert bool((f5[1:] < f5[:-1]).all())
    for bad in (dict(rotary_dim=3), dict(rotary_dim=130), dict(rotary_dim=64, scaling="other"),
                dict(rotary_dim=64, factor=0.0), dict(rotary_dim=64, base=1.0), dict(rotary_dim=2, scaling="ntk", factor=2.0),
                dict(rotary_dim=64, scaling="by_parts", low=2.0, high=2.0)):
        with pytest.raises(ValueError):
            da.rope_frequencies(**bad)
