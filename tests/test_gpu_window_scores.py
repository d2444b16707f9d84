"""Attention over the cache whose scores are as large as the interface allows: +-3e8
with many rows a kv head, +-5e29 with few."""

import numpy as np
import pytest
import torch

from chunk_ref import assert_attention
from libpkv import ensure_built
from paged_kv_cache_56_gb300.runtime import ChunkBuffers, PagedKVCache, extend_step, read_back
from test_gpu_prompt import Prompts
from test_gpu_prompt_scores import decided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("heads", [(4, 2, 64), (16, 8, 128)])
@pytest.mark.parametrize("e", [20, 23, 25])
def test_many_rows(e, heads, int8):
    """A standard normal score grows to 5.5 in 100 000: times 2^25, 1.9e8."""
    p = Prompts(11, [6, 1, 300, 131], heads, behind=0, q_mult=2.0 ** e)
    c = PagedKVCache(1, 60, *heads, 16, int8, max_slots=4, max_blocks_per_seq=24)
    for r in range(4):
        c.add_sequence(r)
    bufs, scale = ChunkBuffers(c, 4, p.T, 300), heads[2] ** -0.5
    out = torch.empty((p.T, *heads[::2]), dtype=torch.bfloat16, device="cuda")
    q, k, v = (x.clone() for x in (p.q, p.k, p.v))
    extend_step(c, bufs, list(range(4)), p.new, [q], [k], [v], [out], scale, window=200, sinks=3)
    p.k, p.v, _ = read_back(c, 0, list(range(4)), torch.float32)
    ok, best, top = decided(p, 200, 3)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all() and ok.mean() >= 0.8
    assert (np.abs(got) <= top * (1 + 2.0 ** -8) ** 2 + 1e-30).all()
    assert_attention(torch.as_tensor(got[ok]), best[ok], np.abs(best[ok]))
    assert c.layers[0].error_bits() == 0


@pytest.mark.parametrize("heads", [(4, 2, 64), (16, 8, 128)])
@pytest.mark.parametrize("e", [20, 28, 32, 64, 95])
def test_few_rows(e, heads):
    """The last token of each prompt by itself."""
    p = Prompts(11, [6, 1, 300, 131], heads, behind=0, q_mult=2.0 ** e)
    c = PagedKVCache(1, 60, *heads, 16, False, max_slots=4, max_blocks_per_seq=24)
    for r in range(4):
        c.add_sequence(r)
    last = np.cumsum(p.new) - 1
    rest = [i for i in range(p.T) if i not in last]
    scale, ids = heads[2] ** -0.5, list(range(4))
    q, k, v = (x[rest].clone() for x in (p.q, p.k, p.v))
    extend_step(c, ChunkBuffers(c, 4, p.T - 4, 300), ids, [n - 1 for n in p.new], [q], [k], [v], [torch.empty_like(q)], scale)
    at = torch.as_tensor(last).cuda()
    q, k, v = (x[at].clone() for x in (p.q, p.k, p.v))
    out = torch.empty_like(q)
    extend_step(c, ChunkBuffers(c, 4, 4, 1), ids, [1] * 4, [q], [k], [v], [out], scale)
    ok, best, _ = (x[last] for x in decided(p, 0, 0))
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all() and ok.mean() >= 0.6
    assert_attention(torch.as_tensor(got[ok]), best[ok], np.abs(best[ok]))
