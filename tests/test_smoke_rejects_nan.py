"""The smoke step fails on outputs that are NaN (CPU, with a stand-in for the library)."""
import math

import pytest

torch = pytest.importorskip("torch")
import __graft_entry__ as entry
from split_kv_decode_attention_gb300 import binding


class Library:
    """The calls of the step over empty caches: zeros are right, as is no NaN."""

    def __init__(self, bad):
        self.bad = bad
        self.rope_frequencies = binding.rope_frequencies

    def rope_table(self, f, n, amplitude):
        return torch.zeros(n, 2 * f.numel())

    def rope_append(self, *a, **k):
        return None

    def block_digest(self, *a, **k):
        return None, None

    def result(self, q, name):
        out = torch.zeros_like(q)
        if name == self.bad:
            out[1, 0, 3, 5] = math.nan
        return out

    def decode_attn(self, q, *a, **k):
        return self.result(q, "dense"), None

    def decode_attn_sparse(self, q, *a, top_k, **k):
        blocks = torch.full((2, 1, 2, top_k), -1, dtype=torch.int32)
        blocks[..., 0] = 0
        return self.result(q, top_k), None, blocks


@pytest.mark.parametrize("bad", [None, "dense", 7, 3])
def test_smoke_step(monkeypatch, bad):
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: None)
    if bad is None:
        entry._smoke_step(Library(bad), torch, torch.device("cpu"))
    else:
        with pytest.raises(AssertionError):
            entry._smoke_step(Library(bad), torch, torch.device("cpu"))
