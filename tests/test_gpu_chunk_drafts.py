"""Drafted tokens, some of them rejected: what is kept is what a cache holds that never saw the others."""

import pytest
import torch

from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv
from paged_kv_cache_56_gb300.runtime import ChunkBuffers, PagedKVCache, read_back, run_chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


HEADS = (4, 2, 64)


class Side:
    def __init__(self, int8, bs):
        self.cache = PagedKVCache(1, 24, *HEADS, bs, int8, max_slots=2, max_blocks_per_seq=12)
        self.bufs = ChunkBuffers(self.cache, 1, 40, 40)
        self.cache.add_sequence(1)

    def step(self, rows, keep=None):
        """Brings rows (q, k, v) [n, H, d]; keeps the first `keep`. Returns the outputs [n, Hq, d]."""
        n = rows[0].shape[0]
        q, k, v = (torch.zeros((1, 40) + x.shape[1:], dtype=torch.bfloat16, device="cuda") for x in rows)
        for buf, x in zip((q, k, v), rows):
            buf[0, :n] = x
        out = torch.zeros_like(q)
        plan = self.cache.plan_chunk([1], [n])
        self.cache.apply_cow(plan)
        self.bufs.upload(plan)
        run_chunk(self.cache, self.bufs, q, k, v, out, 0.125)
        self.cache.commit_chunk([1], [n if keep is None else keep])
        return out[0, :n]


@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("start,n,keep", [(14, 2, 1), (5, 6, 1), (5, 6, 0), (14, 5, 3), (14, 5, 2), (16, 9, 0), (3, 32, 29),
                                          (63, 3, 1), (64, 30, 17), (60, 10, 5), (14, 5, 1), (14, 5, 0), (60, 10, 2)])
def test_rejected_tokens_leave_no_trace(start, n, keep, int8, bs):
    g = torch.Generator().manual_seed(start * 100 + n)
    hq, hkv, d = HEADS

    def rows(m):
        return [torch.randn((m, h, d), generator=g).to(torch.bfloat16).cuda() for h in (hq, hkv, hkv)]

    drafted, plain = Side(int8, bs), Side(int8, bs)
    for at in range(0, start, 30):
        r = rows(min(30, start - at))
        assert torch.equal(drafted.step(r), plain.step(r))
    draft = rows(n)
    end = start + keep
    if int8 and end % bs and end // bs != (start + n) // bs:
        with pytest.raises(ValueError):
            drafted.step(draft, keep)
        return
    drafted.step(draft, keep)
    if keep:
        plain.step([x[:keep] for x in draft])
    assert drafted.cache.seqs[1].length == plain.cache.seqs[1].length == end
    for m in (1, 20):
        for a, b in zip(read_back(drafted.cache, 0, [1]), read_back(plain.cache, 0, [1])):
            assert torch.equal(torch.as_tensor(a), torch.as_tensor(b))
        r = rows(m)
        assert torch.equal(drafted.step(r), plain.step(r))
    assert pkv.pkv_sync_status([drafted.cache.layers[0].desc, plain.cache.layers[0].desc]) == 0


@pytest.mark.parametrize("bs", [16, 64])
def test_forked_sequences_with_blocks_ahead_of_their_tokens(bs):
    """Blocks that a sequence held before it was forked are each holder's own once it writes them, by chunk or by step."""
    from test_gpu_chunk_run import Model
    m = Model((8, 2, 64), bs, [False, True], seqs=3, blocks=40)
    m.cache.add_sequence(1, 5)
    m.step([1], [20], 0, 0)
    m.cache.fork(1, 2)
    m.step([1, 2], [70, 50], 0, 0)  # checks what each holds afterwards against the rows that it brought
    m.step([2, 1], [1, 1], 0, 0)
    m.cache.fork(2, 3)
    m.step([1, 2, 3], [9, 70, 3], 30, 4)
