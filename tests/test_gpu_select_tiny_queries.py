"""Page selection for queries so small that 127 / max |q| overflows: entries that are
zero stay zero, all others become 127 of their sign, as clamped infinities do."""
import pytest

torch = pytest.importorskip("torch")

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


def reference(q, digest, dscale, top_k):
    """[G, 128] bf16, int8 [n, 2, 128], fp32 [n] -> ascending places; page 0 and the last forced."""
    best = None
    for row in q.float():
        a = row.abs().amax()
        inv = torch.tensor(127.0) / a if a > 0 else torch.tensor(0.0)
        code = torch.where(row == 0, 0.0, (row * inv).round().clamp(-127, 127)).to(torch.int64)
        dg = digest.to(torch.int64)
        dot = (code.clamp(max=0) * dg[:, 0] + code.clamp(min=0) * dg[:, 1]).sum(1).float()
        s = (dot * dscale) * (a / torch.tensor(127.0))
        best = s if best is None else torch.maximum(best, s)
    s = best.double()
    s[0] = s[-1] = float("inf")
    return torch.sort(s, descending=True, stable=True).indices[:top_k].sort().values


@pytest.mark.parametrize("G,T", [(2, 1), (12, 1), (3, 2)])     # one row tile and several, one token and more
@pytest.mark.parametrize("top", [1e-36, 3.0e-37, 1e-38, 9.2e-41])
def test_zero_channels(da, top, G, T):
    g = torch.Generator().manual_seed(int(1e42 * top) % 1000 + G)
    pages, top_k = 200, 20
    digest = torch.randint(-127, 128, (pages, 1, 2, D), generator=g).to(torch.int8)
    dscale = torch.rand(pages, 1, generator=g) * 1e30 + 1e29   # (scores stay normal numbers)
    q = (torch.randn(1, T, G, D, generator=g).clamp(-4, 4) * (top / 4)).to(torch.bfloat16)
    q[..., ::3] = 0.0
    q[..., 1::7] = -0.0
    bt = torch.randperm(pages, generator=g).to(torch.int32)[None]
    lens = torch.tensor([pages * 16], dtype=torch.int32)
    blocks, _, _ = da.block_select(q.cuda(), digest.cuda(), dscale.cuda(), bt.cuda(), lens.cuda(), page_size=16,
                                   max_seq_len=pages * 16, top_k=top_k)
    at = bt[0].long()
    for t in range(T):
        want = reference(q[0, t], digest[at, 0], dscale[at, 0], top_k)
        assert torch.equal(blocks[0, t, 0].cpu().long(), want), t


def test_digest_of_tiny_keys(da):
    """The digests' side of the same rule."""
    g = torch.Generator().manual_seed(3)
    k = (torch.randn(4, 16, 1, D, generator=g).clamp(-4, 4) * 1e-38).to(torch.bfloat16)
    k[..., ::3] = 0.0
    bt = torch.arange(4, dtype=torch.int32)[None].cuda()
    lens = torch.tensor([64], dtype=torch.int32).cuda()
    digest, scale = da.block_digest(k.cuda(), bt, lens, max_seq_len=64)
    x = k[:, :, 0].float()
    ends = torch.stack([x.amin(1), x.amax(1)], 1)              # [pages, 2, 128]
    want = (ends.sign() * 127).to(torch.int8)
    assert torch.equal(digest[:, 0].cpu(), want)
    assert torch.equal(scale[:, 0].cpu(), ends.abs().amax((1, 2)) / torch.tensor(127.0))
