"""Outputs of tree masks that share memory with the inputs or with each other are refused."""
import pytest

from tests.test_cache_ops_host import A, lib  # noqa: F401
from tests.test_tree_ops_host import mask_call

PARENTS, OWN, LENS, MASK, POS = (A + i * 4096 for i in range(5))  # [2, 40]: 320 bytes, masks 640, lengths 8


@pytest.mark.parametrize("kw", [
    dict(mask=PARENTS), dict(mask=PARENTS + 316), dict(mask=PARENTS - 636), dict(mask=OWN + 4), dict(mask=LENS - 636),
    dict(mask=POS - 636), dict(pos=MASK + 636), dict(pos=OWN), dict(pos=LENS + 4), dict(pos=PARENTS + 4), dict(pos=PARENTS - 316)])
def test_overlapping_outputs(lib, kw):  # noqa: F811
    a = dict(batch=2, q_len=40, parents=PARENTS, own=OWN, lens=LENS, mask=MASK, pos=POS)
    a.update(kw)
    assert mask_call(lib, **a) == -2


@pytest.mark.gpu
def test_positions_in_the_place_of_parents():
    torch = pytest.importorskip("torch")
    from split_kv_decode_attention_gb300 import binding as da

    parents = torch.tensor([[-1, 0, 0, 2] + list(range(3, 39))] * 300, dtype=torch.int32, device="cuda")
    lens = torch.full((300,), 77, dtype=torch.int32, device="cuda")
    mask, pos = da.tree_mask(parents, lens, max_seq_len=100)
    same = parents.clone()
    mask2, pos2 = da.tree_mask(same, lens, max_seq_len=100, positions=same)
    assert torch.equal(mask, mask2) and torch.equal(pos, pos2) and pos2.data_ptr() == same.data_ptr()


def test_apart_or_in_place_is_not_refused(lib):  # noqa: F811
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("the addresses are not memory")
    for kw in (dict(pos=PARENTS), dict(pos=None), dict(mask=PARENTS + 320), dict(mask=OWN + 8), dict(mask=POS - 640)):
        a = dict(batch=2, q_len=40, parents=PARENTS, own=OWN, lens=LENS, mask=MASK, pos=POS)
        a.update(kw)
        assert mask_call(lib, **a) not in (0, -2)
