"""Workspaces of trees and cross attention that were sized for another batch."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
from tests import cache_ref as R
from tests.strict import assert_attention
from tests.test_cache_ops_host import cache, params, ref
from tests.test_gpu_cache_ops import D, Paged, bf16, gen, status_word
from tests.test_gpu_tree_ops import SCALE, cross_call, da  # noqa: F401

pytestmark = pytest.mark.gpu


def check(c, q, out, lse, base):
    """Against 64 bits.  A row's largest weight is held in f16 as at least 2^6 and no step of f16 is above 2^-24 where
    weights are subnormal, so each of n weights is off by up to 2^-31 besides its relative error: where the dominant key's
    value is 0, as 4-bit ones often are, that is what is left."""
    G = q.shape[2] // c.heads
    kv, vv = (c.values(w) * s for w, s in (("k", c.ks), ("v", c.vs)))
    lost = max(c.lens) * 2.0 ** -31 * float(vv.abs().max())

    def tol(o, wabs, mag):
        return base(o, wabs, mag) + lost

    for b, n in enumerate(c.lens):
        k, v = R.gather(kv, c.bt, b, n), R.gather(vv, c.bt, b, n)
        for h in range(c.heads):
            assert_attention(out[b, :, h * G:(h + 1) * G].double().cpu().reshape(-1, D),
                             lse[b, :, h * G:(h + 1) * G].double().cpu().reshape(-1), q[b, :, h * G:(h + 1) * G].double().reshape(-1, D),
                             k[:, h], v[:, h], torch.ones(G * q.shape[1], n, dtype=torch.bool), SCALE, tol, (b, h))


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("lens,T,G,page", [([1500, 300, 0, 77], 200, 8, 16), ([2000, 129], 1400, 1, 0)])
def test_many_rows_without_room_for_a_copy(da, kind, lens, T, G, page):  # noqa: F811
    """Calls that would copy K and V to bf16 convert them instead where the workspace holds the partials alone; the C
    entry refuses one byte less."""
    c = Paged(kind, lens, 2, page, 31).gpu()
    q = bf16(gen(31), len(lens), T, 2 * G, D, std=2.0)
    dq = q.cuda()
    cross_call(da, c, dq)
    ws = torch.full((da.ROWS_WORKSPACE,), 0xff, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(dq), torch.empty(dq.shape[:3], device="cuda")
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    status = status_word()
    cross_call(da, c, dq, workspace=ws, out=out, lse=lse, status=status)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() <= before + 1024 and int(status) == 0  # (the status word's block)
    check(c, q, out, lse, R.out_tolerance)
    # the C entry, which makes no workspace of its own
    n = ctypes.c_size_t()
    pages = (16, c.dbt.shape[1], c.dk.shape[0]) if page else (0, 0, 0)
    p = da.decode_attn_params_init(len(lens), T, 2 * G, 2, D, *pages, c.max_len, False)
    p.kv_stride_head, p.kv_stride_token, p.kv_stride_page = c.dk.stride(2), c.dk.stride(1), c.dk.stride(0)
    kt = da.DA_CACHE_FP4_E2M1 if kind == "fp4" else da.DA_CACHE_FP8_E4M3
    assert da.lib().decode_attn_cross_workspace_bytes(ref(p), ref(cache(kt)), 0, ctypes.byref(n)) == 0
    assert n.value > da.ROWS_WORKSPACE
    got, _ = cross_call(da, c, dq, workspace=ws[:-16])  # (the Python entry makes its own: the whole one)
    check(c, q, got, lse, R.bf16_p_tolerance)
    if page == 0:
        return
    cc = cache(kt, k=c.dk.data_ptr(), v=c.dv.data_ptr())
    if kind == "fp4":
        cc.k_block_scale, cc.v_block_scale = c.dk_sf.data_ptr(), c.dv_sf.data_ptr()
    p.k_scale, p.v_scale = c.ks, c.vs
    for nbytes, code in ((da.ROWS_WORKSPACE - 1, -7), (da.ROWS_WORKSPACE, 0)):
        got = torch.zeros_like(dq)
        assert da.lib().decode_attn_cross(ref(p), ref(cc), dq.data_ptr(), None, c.dbt.data_ptr(), c.dlens.data_ptr(), got.data_ptr(),
                                          lse.data_ptr(), 0, ws.data_ptr(), nbytes, None, None) == code
        torch.cuda.synchronize()
        same = torch.equal(got, torch.zeros_like(dq) if code else out)
        assert same


def test_size_of_the_least_workspace(da):  # noqa: F811
    n = ctypes.c_size_t()
    p = params(fp4=False, q_len=100, max_pages_per_seq=400, block_table_stride=400, max_seq_len=6400)
    assert da.lib().decode_attn_cross_workspace_bytes(ref(p), ref(cache(da.DA_CACHE_BF16)), 0, ctypes.byref(n)) == 0
    assert n.value == da.ROWS_WORKSPACE


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("T,hq,hkv", [(1, 32, 8), (4, 32, 8), (7, 8, 1), (16, 32, 8), (32, 32, 8), (5, 48, 16)])
def test_a_workspace_serves_smaller_batches(da, kind, T, hq, hkv):  # noqa: F811
    """Up to 128 rows a smaller batch may be cut into more chunks: sizes that fell from 1 MB for 32 requests to nothing
    for 64 left a workspace, sized once for the largest batch, too small for most others."""
    n, kt = ctypes.c_size_t(), {"bf16": 0, "fp8": 1, "fp4": 2}[kind]
    for L in (40, 300, 640, 1500, 4096, 20000, 100000):
        pages = -(-L // 16)
        most = 0
        for B in (*range(1, 140), 152, 200, 304, 400, 608, 1000, 1024, 1025, 3000):
            p = da.decode_attn_params_init(B, T, hq, hkv, D, 16, pages, pages, L, False)
            if kind == "fp4":
                p.kv_stride_page, p.kv_stride_token, p.kv_stride_head = 16 * hkv * 64, hkv * 64, 64
            for f in (da.lib().decode_attn_tree_workspace_bytes, da.lib().decode_attn_cross_workspace_bytes):
                assert f(ref(p), ref(cache(kt)), 0, ctypes.byref(n)) == 0
                assert n.value >= most, (L, B, n.value, most)
            most = n.value


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_one_workspace_for_every_batch(da, kind):  # noqa: F811
    """Batches of 1 to 64 requests in the workspace of the largest, through the C entry."""
    T, hq, hkv, L = 1, 32, 8, 640
    c = Paged(kind, [L - 7 * (b % 9) for b in range(64)], hkv, 16, 32).gpu()
    q = bf16(gen(32), 64, T, hq, D, std=2.0).cuda()
    n, kt = ctypes.c_size_t(), {"bf16": 0, "fp8": 1, "fp4": 2}[kind]
    cc = cache(kt, k=c.dk.data_ptr(), v=c.dv.data_ptr())
    if kind == "fp4":
        cc.k_block_scale, cc.v_block_scale = c.dk_sf.data_ptr(), c.dv_sf.data_ptr()
        cc.bs_stride_page, cc.bs_stride_head = c.dk_sf.stride(0), c.dk_sf.stride(1)
    ws = None
    for B in (64, 33, 32, 24, 16, 9, 2, 1):
        p = da.decode_attn_params_init(B, T, hq, hkv, D, 16, c.dbt.shape[1], c.dk.shape[0], c.max_len, False)
        p.kv_stride_head, p.kv_stride_token, p.kv_stride_page = c.dk.stride(2), c.dk.stride(1), c.dk.stride(0)
        p.block_table_stride = c.dbt.stride(0)
        p.k_scale, p.v_scale = c.ks, c.vs
        if ws is None:
            assert da.lib().decode_attn_cross_workspace_bytes(ref(p), ref(cc), 0, ctypes.byref(n)) == 0
            ws = torch.full((n.value + 16,), 0xff, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(q[:B]), torch.empty(B, T, hq, device="cuda")
        assert da.lib().decode_attn_cross(ref(p), ref(cc), q.data_ptr(), None, c.dbt.data_ptr(), c.dlens.data_ptr(), out.data_ptr(),
                                          lse.data_ptr(), 0, ws.data_ptr(), n.value, None, None) == 0, B
        want, wlse = da.cross_attn(q[:B], c.dk, c.dv, c.dbt[:B], c.dlens[:B], max_seq_len=c.max_len, **c.scales())
        assert torch.equal(out, want) and torch.equal(lse, wlse), B
