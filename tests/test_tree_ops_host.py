"""Host-side checks of trees of drafted tokens, cross attention and reading a cache
back: refusals before anything touches a GPU, and workspace sizes."""
import ctypes
import math

import pytest

from split_kv_decode_attention_gb300 import binding as da
from tests.test_cache_ops_host import A, NO_DEVICE_OR_OK, cache, lib, params, ref  # noqa: F401

NULL_OK = NO_DEVICE_OR_OK
B = 2 << 20  # another


def test_struct_size():
    assert ctypes.sizeof(da.DecodeAttnRead) == 40


def mask_call(lib, batch=2, q_len=4, max_len=64, parents=A, own=None, lens=A, mask=A, pos=None, status=None):
    return lib.decode_attn_tree_mask(batch, q_len, max_len, parents, own, lens, mask, pos, status, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), -2), (dict(batch=65536), -2), (dict(q_len=0), -2), (dict(q_len=1025), -2), (dict(max_len=-1), -2),
    (dict(parents=None), -1), (dict(lens=None), -1), (dict(mask=None), -1), (dict(parents=A + 2), -6), (dict(own=A + 1), -6),
    (dict(lens=A + 2), -6), (dict(mask=A + 2), -6), (dict(pos=A + 3), -6), (dict(status=A + 2), -6), (dict(batch=0, parents=None), 0)])
def test_tree_mask_refusals(lib, kw, code):  # noqa: F811
    assert mask_call(lib, **kw) == code


def tree_call(lib, p, c, q=A, mask=A, step=0, own=None, bt=A, lens=A, out=A, lse=A, splits=1, ws=None, ws_bytes=0, status=None):
    return lib.decode_attn_tree(ref(p), ref(c), q, mask, step, own, bt, lens, out, lse, splits, ws, ws_bytes, status, None)


def cross_call(lib, p, c, q=A, own=None, bt=A, lens=A, out=A, lse=A, splits=1, ws=None, ws_bytes=0, status=None):
    return lib.decode_attn_cross(ref(p), ref(c), q, own, bt, lens, out, lse, splits, ws, ws_bytes, status, None)


ROWS = [({}, {}, dict(q=None), -1), ({}, {}, dict(lens=None), -1), ({}, {}, dict(out=None), -1), ({}, {}, dict(lse=None), -1),
        ({}, {}, dict(q=A + 8), -6), ({}, {}, dict(out=A + 8), -6), ({}, {}, dict(lse=A + 2), -6), ({}, {}, dict(lens=A + 1), -6),
        ({}, {}, dict(own=A + 2), -6), ({}, {}, dict(status=A + 2), -6), (dict(type=7), {}, {}, -12), (dict(reserved=1), {}, {}, -2),
        (dict(k=0), {}, {}, -1), (dict(v=A + 8), {}, {}, -6), (dict(k_block_scale=0), {}, {}, -1), ({}, dict(kv_stride_token=72), {}, -6),
        ({}, dict(q_stride_token=7), {}, -6), ({}, dict(k_scale=math.inf), {}, -2), ({}, dict(scale=math.nan), {}, -2),
        ({}, dict(head_dim=64), {}, -3), ({}, dict(page_size=24), {}, -4), ({}, dict(num_q_heads=2 * 129), {}, -5),
        ({}, dict(num_q_heads=7), {}, -2), ({}, dict(q_len=0), {}, -2), ({}, dict(max_seq_len=65), {}, -2)]


@pytest.mark.parametrize("q_len", [1, 100])
@pytest.mark.parametrize("c_kw,p_kw,kw,code", ROWS)
def test_refusals_of_tree_and_cross_attention(lib, q_len, c_kw, p_kw, kw, code):  # noqa: F811
    """The same for few and for many query rows per KV head (4 and 400)."""
    a = dict(q_len=q_len)
    a.update(p_kw)
    assert cross_call(lib, params(**a), cache(**c_kw), **kw) == code
    assert tree_call(lib, params(**a), cache(**c_kw), **kw) == code


def test_refusals_of_tree_attention(lib):  # noqa: F811
    assert tree_call(lib, params(), cache(), mask=None) == -1
    assert tree_call(lib, params(), cache(), mask=A + 2) == -6
    assert tree_call(lib, params(), cache(), step=-1) == -2
    assert tree_call(lib, params(q_len=1025), cache()) == -2
    assert tree_call(lib, None, cache()) == -1 and tree_call(lib, params(), None) == -1
    assert tree_call(lib, params(batch=0), cache(), mask=None) == 0


def test_cross_attention_of_very_many_rows(lib):  # noqa: F811
    assert cross_call(lib, params(q_len=(1 << 29) + 1), cache()) == -2
    assert cross_call(lib, params(batch=0), cache(), q=None) == 0


def test_workspace_of_many_rows(lib):  # noqa: F811
    """Needs no device and no chunk count: partials (two pieces of 256 rows for each of 152 CTAs) and their merge's records;
    for a 4-bit cache and 400 rows (two pairs of tiles) also K and V of every request in bf16, unless those are more than 2 GB."""
    n = ctypes.c_size_t()
    part = 2 * 152 * 256 * 129 * 4 + 152 * 32
    for fp4, copy in ((False, 0), (True, 2 * 2 * 640 * 2 * 128 * 2)):
        p = params(fp4=fp4, q_len=100, max_pages_per_seq=40, block_table_stride=40, max_seq_len=640)
        c = cache() if fp4 else cache(da.DA_CACHE_BF16)
        for f in (lib.decode_attn_tree_workspace_bytes, lib.decode_attn_cross_workspace_bytes):
            for splits in (0, 1, 99):
                assert f(ref(p), ref(c), splits, ctypes.byref(n)) == 0 and n.value == copy + part
            assert f(ref(p), ref(c), 1, None) == -1
            assert f(ref(p), None, 1, ctypes.byref(n)) == -1
    long = params(q_len=100, max_pages_per_seq=1 << 18, block_table_stride=1 << 18, max_seq_len=1 << 21)
    assert lib.decode_attn_cross_workspace_bytes(ref(long), ref(cache()), 0, ctypes.byref(n)) == 0 and n.value == part
    few = params(q_len=50, max_pages_per_seq=40, block_table_stride=40, max_seq_len=640)
    assert lib.decode_attn_cross_workspace_bytes(ref(few), ref(cache()), 0, ctypes.byref(n)) == 0 and n.value == part
    far = params(q_len=1 << 28, max_seq_len=1 << 30, max_pages_per_seq=1 << 26, block_table_stride=1 << 26, num_kv_heads=1 << 13,
                 num_q_heads=1 << 13, batch=60000)
    assert lib.decode_attn_cross_workspace_bytes(ref(far), ref(cache(da.DA_CACHE_BF16)), 0, ctypes.byref(n)) == -2


def keep_call(lib, p, c, keep=A, most=4, counts=A, own=None, bt=A, lens=A, out=None, status=None):
    return lib.decode_attn_cache_keep(ref(p), ref(c), keep, most, counts, own, bt, lens, out, status, None)


@pytest.mark.parametrize("c_kw,p_kw,kw,code", [
    ({}, {}, dict(keep=None), -1), ({}, {}, dict(counts=None), -1), ({}, {}, dict(lens=None), -1), ({}, {}, dict(most=9), -2),
    ({}, {}, dict(most=-1), -2), ({}, {}, dict(out=A), -2), ({}, {}, dict(out=A + 4), -2), ({}, {}, dict(out=B, counts=B - 4), -2),
    ({}, {}, dict(out=B, own=B + 4), -2), ({}, {}, dict(out=B, keep=B - 28), -2), ({}, {}, dict(keep=A + 2), -6), ({}, {}, dict(counts=A + 2), -6),
    ({}, {}, dict(own=A + 2), -6), ({}, {}, dict(bt=A + 2), -6), ({}, {}, dict(out=A + 6), -6), ({}, {}, dict(status=A + 1), -6),
    (dict(k=0), {}, {}, -1), (dict(v_block_scale=0), {}, {}, -1), (dict(type=3), {}, {}, -12), ({}, dict(q_len=1025), {}, -2),
    ({}, dict(page_size=8), {}, -4), ({}, dict(kv_stride_page=8), {}, -6), ({}, dict(batch=0), dict(keep=None), 0)])
def test_cache_keep_refusals(lib, c_kw, p_kw, kw, code):  # noqa: F811
    a = dict(q_len=8)
    a.update(p_kw)
    assert keep_call(lib, params(**a), cache(**c_kw), **kw) == code


def read_args(**kw):
    r = da.DecodeAttnRead()
    r.max_tokens, r.rows, r.stride_batch, r.stride_token, r.stride_head = 64, 100, 64 * 256, 256, 128
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def read_call(lib, p, c, r, starts=None, offsets=None, bt=A, lens=A, k=A, v=A, status=None):
    return lib.decode_attn_cache_read(ref(p), ref(c), ref(r), starts, offsets, bt, lens, k, v, status, None)


@pytest.mark.parametrize("c_kw,r_kw,kw,code", [
    ({}, {}, dict(lens=None), -1), ({}, {}, dict(k=None), -1), ({}, dict(max_tokens=-1), {}, -2), ({}, dict(reserved=1), {}, -2),
    ({}, dict(rows=-1), dict(offsets=A), -2), ({}, dict(stride_token=4), {}, -6), ({}, dict(stride_head=0), {}, -6),
    ({}, dict(stride_batch=12), {}, -6), ({}, {}, dict(k=A + 8), -6), ({}, {}, dict(v=A + 2), -6), ({}, {}, dict(starts=A + 2), -6),
    ({}, {}, dict(offsets=A + 2), -6), ({}, {}, dict(status=A + 2), -6), (dict(k=0), {}, {}, -1), (dict(v=0), {}, {}, -1),
    (dict(type=9), {}, {}, -12), ({}, dict(max_tokens=0), dict(k=None), 0), ({}, dict(rows=0), dict(offsets=A, k=None), 0)])
def test_cache_read_refusals(lib, c_kw, r_kw, kw, code):  # noqa: F811
    assert read_call(lib, params(), cache(**c_kw), read_args(**r_kw), **kw) == code


def test_cache_read_null_descriptors(lib):  # noqa: F811
    assert read_call(lib, params(), cache(), None) == -1
    assert read_call(lib, None, cache(), read_args()) == -1
    # V alone may be left out: with no v_out its cache is not looked at
    assert read_call(lib, params(), cache(v=0, v_block_scale=0), read_args(), v=None) in NULL_OK[1:]


def test_python_refusals():
    """Shapes, types and devices that the Python entries turn down (CPU tensors: nothing is launched)."""
    torch = pytest.importorskip("torch")
    i32 = dict(dtype=torch.int32)
    k = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    q = torch.zeros(2, 5, 8, 128, dtype=torch.bfloat16)
    bt, lens = torch.zeros(2, 2, **i32), torch.full((2,), 20, **i32)
    mask = torch.zeros(2, 5, 1, **i32)

    def tree(**kw):
        a = dict(q=q, k=k, v=k, bt=bt, lens=lens, mask=mask, own=None)
        a.update(kw)
        return da.decode_attn_tree(a["q"], a["k"], a["v"], a["bt"], a["lens"], a["mask"], max_seq_len=32, new_lens=a["own"])

    for bad in (dict(mask=mask.long()), dict(mask=torch.zeros(2, 5, 2, **i32)), dict(mask=torch.zeros(3, 5, 1, **i32)),
                dict(mask=torch.zeros(2, 4, 1, **i32)), dict(mask=None), dict(own=torch.zeros(3, **i32)), dict(own=lens.long()),
                dict(lens=torch.zeros(3, **i32)), dict(q=q.float()), dict(q=q[..., :64]), dict(v=k.float()), dict(bt=bt.long()), {}):
        with pytest.raises(ValueError):  # ({}: no fault but the device)
            tree(**bad)
    with pytest.raises(ValueError):
        da.tree_mask(torch.zeros(2, 1025, **i32), lens, max_seq_len=32)
    with pytest.raises(ValueError):
        da.tree_mask(torch.zeros(2, 5), lens, max_seq_len=32)
    with pytest.raises(ValueError):
        da.cache_keep(k, k, bt, lens, torch.zeros(2, 6, **i32), lens, new_tokens=5, max_seq_len=32)
    with pytest.raises(ValueError):
        da.cache_keep(k, k, bt, lens, torch.zeros(2, 5).int().t(), lens, new_tokens=5, max_seq_len=32)
    with pytest.raises(ValueError):
        da.cache_read(k, k, bt, lens, max_seq_len=32, offsets=lens)
    with pytest.raises(ValueError):
        da.cache_read(k, k, bt, lens, max_seq_len=32, k_out=torch.zeros(2, 32, 2, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        da.cross_attn(q, k, k, None, lens, max_seq_len=32)  # (a contiguous cache of 4 requests for 2)
