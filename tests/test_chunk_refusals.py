"""Calls of the chunk operators that cannot be right are refused before any launch."""

import pytest
import torch

from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv
from test_chunk_host import batch, rope, window


@pytest.fixture(scope="module")
def L():
    return ensure_built()


def test_in_place_with_another_stride(L):
    """The output may be the queries themselves, row for row only."""
    for qs, os_ in ((512, 1024), (1024, 512)):
        assert rope(L, q=16, qs=qs, o=16, os_=os_) == pkv.PKV_ERR_INVALID
        assert window(L, q=16, qs=qs, o=16, os_=os_) == pkv.PKV_ERR_INVALID


def test_buffers_of_more_new_tokens_than_tokens():
    """The largest sequence of a batch cannot bring more than the batch; the descriptor would fail at the first launch."""
    from types import SimpleNamespace
    from paged_kv_cache_56_gb300.runtime import ChunkBuffers
    cache = SimpleNamespace(device="cpu", max_blocks=4, int8=False)
    for args in ((2, 8, 9), (2, 8, -1), (-1, 8, 8), (2, 0, 1), (65536, 8, 8)):
        with pytest.raises(ValueError, match="max_"):
            ChunkBuffers(cache, *args)


def test_a_single_row_may_carry_any_stride():
    """The token stride of one row means nothing: a view of any wider row is taken, and is in place with itself."""
    b = batch(num_tokens=1, max_tokens=1, B=1)
    b.device = torch.device("cpu")
    for stride in (1, 511, 512, 514, 1028):
        x = torch.zeros(2048, dtype=torch.bfloat16).as_strided((1, 4, 128), (stride, 128, 1))
        assert pkv._rows(x, "q", b, 4, 128) == (x.data_ptr(), 512)
    wide = torch.zeros((3, 5, 128), dtype=torch.bfloat16)
    assert pkv._rows(wide[:, 1:], "q", b, 4, 128) == (wide.data_ptr() + 256, 512)
