"""How long a DevicePool and what is captured with it live: steps of several batch
sizes on the same buffers, and a pool that has been pulled."""

import pytest
import torch

from libpkv import ensure_built
from paged_kv_cache_56_gb300.runtime import DevicePool, GraphStep, StepBuffers, decode_step, read_back
from test_gpu_planned import HEADS, assert_same_rows, begin, caches_are_the_same, make_cache, rows

pytestmark = pytest.mark.gpu
SCALE = HEADS[2] ** -0.5


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def inputs(seed, B):
    return [rows(seed + i, 2, B, h) for i, h in enumerate((HEADS[0], HEADS[1], HEADS[1]))]


@pytest.mark.parametrize("int8", [False, True])
def test_captured_steps_of_two_batch_sizes_share_their_buffers(int8):
    """A step captured for two entries, one for four, then both replayed in turn:
    what the first one writes to is still there."""
    host, gpu = make_cache(int8), make_cache(int8)
    for c in (host, gpu):
        begin(c, [37, 16, 1, 60], 7)
    hb, gb = (StepBuffers(c, 4, split_tokens=64) for c in (host, gpu))
    pool = DevicePool(gpu)
    steps, places = {}, set()
    for n, order in enumerate([[2, 0], [3, 1, 0, 2], [2, 0], [0, 1, 2, 3], [1, 3], [2, 1, 0, 3]]):
        B = len(order)
        q, k, v = inputs(300 + 3 * n, B)
        want = torch.empty_like(q)
        decode_step(host, hb, order, q, k, v, want, SCALE)
        pool.use(gb, order)
        first = B not in steps
        if first:
            steps[B] = GraphStep(gpu, gb, SCALE, pool=pool)
        step = steps[B]
        for to, x in ((step.q, q), (step.k, k), (step.v, v)):
            to.copy_(x)
        if first:
            step.run_eager()
            got = step.out.clone()
            step.capture()
        else:
            step.replay()
            got = step.out
        assert_same_rows(got, want)
        places.add(pool._plan_of(gb)[1].token_starts)
    assert len(places) == 1
    assert pool.error_bits() == 0 and all(lc.error_bits() == 0 for lc in gpu.layers)
    pool.pull()
    caches_are_the_same(gpu, host)


def test_a_pulled_pool_plans_nothing():
    c = make_cache(False)
    begin(c, [20, 33], 71)
    bufs, pool = StepBuffers(c, 2), DevicePool(c)
    pool.use(bufs, [0, 1])
    step = GraphStep(c, bufs, SCALE, pool=pool)
    step.run_eager()
    step.capture()
    step.replay()
    pool.pull()
    for again in (False, True):  # a pool of its own later on does not bring the old one back
        newer = DevicePool(c) if again else None
        for call in (lambda: pool.use(bufs, [0, 1]), lambda: pool.plan(bufs), lambda: pool.commit(bufs),
                     lambda: pool.release([0]), pool.pull, step.replay, step.run_eager):
            with pytest.raises(RuntimeError, match="not in this pool"):
                call()
    newer.pull()
    assert [c.seqs[r].length for r in (0, 1)] == [22, 35]


def test_a_sequence_that_began_on_the_gpu_is_not_read_back_as_empty():
    c = make_cache(False)
    c.add_sequence(0)
    bufs, pool = StepBuffers(c, 1), DevicePool(c)
    pool.use(bufs, [0])
    step = GraphStep(c, bufs, SCALE, pool=pool)
    step.run_eager()
    with pytest.raises(RuntimeError, match="GPU"):
        read_back(c, 0, [0])
    pool.pull()
    assert read_back(c, 0, [0])[0].shape[0] == 1
