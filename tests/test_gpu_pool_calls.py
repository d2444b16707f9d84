"""Calls of a DevicePool in other orders and on other streams: what they do is what
the host would have done, or they are refused."""

import pytest
import torch

from libpkv import ensure_built
from paged_kv_cache_56_gb300.runtime import DevicePool, StepBuffers
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
