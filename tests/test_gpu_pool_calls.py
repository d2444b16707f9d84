"""Calls of a DevicePool in other orders and on other streams: what they do is what
the host would have done, or they are refused."""

import numpy as np
import pytest
import torch

from libpkv import ensure_built
from paged_kv_cache_56_gb300.runtime import AxisPositions, ChunkBuffers, DevicePool, StepBuffers
from test_gpu_axes import positions_of
from test_gpu_planned import begin, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def lengths(c):
    return [s.length for s in c.seqs.values()]


def test_the_first_plan_on_another_stream():
    """The array of row starts is made with the first plan: its zeros must not land behind what
    the plan has put there, though the stream that they are on has work to do before."""
    c = make_cache(False)
    begin(c, [20, 33], 71)
    bufs, pool, side = StepBuffers(c, 2), DevicePool(c), torch.cuda.Stream()
    pool.use(bufs, [0, 1], stream=side)
    torch.cuda._sleep(20_000_000)  # cycles on the current stream: some 10 ms
    pool.plan(bufs, stream=side)
    side.wait_stream(torch.cuda.current_stream())
    pool.commit(bufs, stream=side)
    torch.cuda.synchronize()
    assert bufs.gpu_starts.tolist() == [0, 1, 2] and pool.error_bits() == 0
    pool.pull()
    assert lengths(c) == [21, 34]


def test_axis_positions_set_on_another_stream():
    """A sequence's segments set, and its positions worked out, on a stream of their own right after the arrays
    were made: the zeros that the arrays begin with do not land behind them."""
    c, side = make_cache(False), torch.cuda.Stream()
    c.add_sequence(0)
    bufs = ChunkBuffers(c, 1, 40, 40)
    plan = c.plan_chunk([0], [40])
    with torch.cuda.stream(side):
        bufs.upload(plan)
    segs = [(5, 0, 0, 1), (2, 3, 4, 2), (4, 0, 0, 1)]
    torch.cuda._sleep(20_000_000)  # cycles on the current stream: some 10 ms
    where = AxisPositions(c, 40, 4)
    where.set(0, segs, stream=side)
    where.update(bufs, stream=side)
    torch.cuda.synchronize()
    assert np.array_equal(where.positions.cpu().numpy(), positions_of(segs, 40)) and where.err.item() == 0
