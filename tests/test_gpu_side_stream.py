"""Forks, copies on write and prefills on a stream that has work to do, while the
current one goes on allocating: the ids and rows that they read stay theirs."""

import pytest
import torch

from libpkv import ensure_built
from paged_kv_cache_56_gb300.runtime import prefill, read_back
from test_gpu_planned import HEADS, begin, make_cache, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def busy(side):
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # cycles: some 10 ms


def others(n=64):
    """What small tensors of the current stream hold meanwhile."""
    return [torch.full((1,), 5, dtype=torch.int32, device="cuda") for _ in range(n)]


@pytest.mark.parametrize("int8", [False, True])
def test_forks_and_copies_on_write(int8):
    c, side = make_cache(int8, slots=8), torch.cuda.Stream()
    begin(c, [20, 33], 71)
    want = [read_back(c, 1, [r])[:2] for r in (0, 1)]
    busy(side)
    c.fork(0, 7, stream=side)
    keep = others()
    torch.cuda.synchronize()
    plan = c.plan_step([7, 1])
    assert len(plan.cow) == 1
    busy(side)
    c.apply_cow(plan, side)
    keep += others()
    torch.cuda.synchronize()
    for r, w in ((0, want[0]), (7, want[0]), (1, want[1])):
        assert all(torch.equal(x, y) for x, y in zip(read_back(c, 1, [r])[:2], w))
    assert all(lc.error_bits() == 0 for lc in c.layers) and len(keep) == 128


@pytest.mark.parametrize("int8", [False, True])
def test_prefill(int8):
    a, b, side = make_cache(int8), make_cache(int8), torch.cuda.Stream()
    k, v = (rows(80 + i, 1, 70, HEADS[1])[0] for i in range(2))
    for c, stream in ((a, None), (b, side)):
        c.add_sequence(0, n_blocks=5)
        c.add_sequence(1, n_blocks=5)
        for li in range(2):
            if stream is not None:
                busy(side)
            prefill(c, li, [0, 1], [k[:37], k[37:]], [v[:37], v[37:]], stream=stream)
            keep = [torch.full_like(k, 5.0) for _ in range(4)] + others()
        torch.cuda.synchronize()
        c.seqs[0].length, c.seqs[1].length = 37, 33
        assert all(lc.error_bits() == 0 for lc in c.layers) and keep
    for li in range(2):
        assert all(torch.equal(x, y) for x, y in zip(read_back(a, li, [0, 1])[:2], read_back(b, li, [0, 1])[:2]))
