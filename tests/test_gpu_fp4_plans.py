"""Chunks of equal-length calls over 4-bit caches: no more than a cluster merges only
where a cluster merges them."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
from tests.strict import assert_attention
from tests.test_gpu_cache_ops import Paged, bf16, gen
from tests import cache_ref as R

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


def call(da, requests, length, two_pass=False):
    """Runs a planned call; its workspace as 32-bit words."""
    pc = Paged("fp4", [length] * requests, 1, 64, 600).gpu()
    q = bf16(gen(601), requests, 1, 4, D, std=2.0)
    ws = torch.full((1 << 24,), -1, dtype=torch.int32, device="cuda")
    out, lse = da.decode_attn(q.cuda(), pc.dk, pc.dv, pc.dbt, pc.dlens, max_seq_len=length, workspace=ws,
                              two_pass=two_pass, **pc.scales())
    k64, v64 = pc.values("k") * pc.ks, pc.values("v") * pc.vs
    for b in range(requests):
        assert_attention(out[b, 0].cpu().double(), lse[b, 0].cpu().double(), q[b, 0].double(),
                         R.gather(k64, pc.bt, b, length)[:, 0], R.gather(v64, pc.bt, b, length)[:, 0],
                         torch.ones(4, length, dtype=torch.bool), D ** -0.5)
    return ws.cpu()


def test_device_plan_cuts_short_calls_as_the_cost_rule_says(da):
    # chunks of 256 tokens, the shortest of any plan: the GPU has more than 64 slots for them
    ws = call(da, 2, 8192)
    assert ws[:2].tolist() == [256, 64]


def test_one_request_that_keeps_partials(da):
    # 32 chunks x 4 rows x (128 + 1) floats
    p = da.decode_attn_params_init(1, 1, 4, 1, D, 64, 128, 128, 8192, False)
    p.kv_stride_page, p.kv_stride_token, p.kv_stride_head = 64 * 64, 64, 64
    p.k_scale = p.v_scale = 1.0
    c = da.DecodeAttnCache()
    c.type = da.DA_CACHE_FP4_E2M1
    c.bs_stride_page, c.bs_stride_head = 64 * 8, 64 * 8
    n = ctypes.c_size_t()
    p.flags = da.DA_FLAG_TWO_PASS
    assert da.lib().decode_attn_cached_workspace_bytes(ctypes.byref(p), ctypes.byref(c), 0, ctypes.byref(n)) == 0
    assert n.value == 32 * 4 * 129 * 4
    p.flags = 0                                   # (merged through a cluster: no workspace)
    assert da.lib().decode_attn_cached_workspace_bytes(ctypes.byref(p), ctypes.byref(c), 0, ctypes.byref(n)) == 0
    assert n.value == 0
    assert bool((call(da, 1, 8192, two_pass=True) != -1).any()) and not bool((call(da, 1, 8192) != -1).any())
