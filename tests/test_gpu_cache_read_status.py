"""Status of reading a cache back where the outputs have no row, and where they have one."""
import pytest

torch = pytest.importorskip("torch")
from tests.test_gpu_cache_ops import D, Paged, status_word
from tests.test_gpu_tree_ops import da, ints  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_reads_into_no_row_set_no_status(da, kind):  # noqa: F811
    c = Paged(kind, [40, 20], 1, 16, 3).gpu()

    def bits(rows, lens, offsets=(0, 40), max_seq_len=None, tokens=None):
        status = status_word()
        shape = (rows, 1, D) if tokens is None else (2, tokens, 1, D)
        k, v = (torch.full(shape, 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        da.cache_read(c.dk, c.dv, c.dbt, ints(lens), max_seq_len=c.max_len if max_seq_len is None else max_seq_len,
                      offsets=None if tokens is not None else ints(list(offsets)), k_out=k, v_out=v, status=status, **c.scales())
        return int(status)

    for lens in ([40, 20], [41, -1], [0, 0]):
        assert bits(0, lens) == 0                       # no row to write to: nothing is looked at
        assert bits(0, lens, tokens=0) == 0
        assert bits(60, lens, max_seq_len=0) == 0
    assert bits(1, [40, 20]) == 2 and bits(1, [0, 0]) == 2 and bits(1, [0, 0], offsets=(0, 1)) == 0
    assert bits(60, [40, 20]) == 0 and bits(60, [41, 20]) == 2 and bits(0, [41, 20], tokens=3) == 2
