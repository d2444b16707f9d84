"""Calls of a DevicePool in other orders and on other streams: what they do is what
the host would have done, or they are refused."""

import ctypes

import numpy as np
import pytest
import torch

from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv
from paged_kv_cache_56_gb300.runtime import (AxisPositions, ChunkBuffers, DevicePool, GraphStep, StepBuffers, axis_pairs,
                                             decode_step, read_back, rope_frequencies, run_chunk, run_layers)
from test_gpu_axes import positions_of
from test_gpu_planned import HEADS, begin, caches_are_the_same, make_cache, rows

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


@pytest.mark.parametrize("int8", [False, True])
def test_a_removed_sequence_is_not_stepped(int8):
    """A captured step replayed after one of its sequences was removed, without use() in between: the
    others go on, the slot stays empty, and the next sequence that gets it begins empty."""
    c = make_cache(int8)
    begin(c, [20, 33, 47], 71)
    steps, chunks, pool = StepBuffers(c, 3), ChunkBuffers(c, 4, 8, 2), DevicePool(c)
    pool.use(steps, [2, 0, 1])
    pool.use(chunks, [1, 0])
    step = GraphStep(c, steps, 0.1, pool=pool)
    step.run_eager()
    step.capture()
    step.replay()
    slot, free = c.seqs[1].slot, pool.state[1].item()
    c.remove_sequence(1)
    assert pool.state[1].item() == free + 3  # 35 tokens
    step.out.fill_(7.0)
    step.replay()
    assert (step.out[:, 2] == 0).all() and (step.out[:, :2] != 7).any()
    pool.plan(chunks, torch.tensor([2, 2, 2, 2], dtype=torch.int32, device="cuda"))
    assert chunks.starts.tolist() == [0, 0, 2, 2, 2]  # the entry of 0 alone: the one of 1 has no sequence now
    assert pool.lens[slot].item() == pool.held[slot].item() == 0
    while slot in c.free_slots:  # the last of them gets the slot
        c.add_sequence(10 + len(c.seqs))
    step.replay()
    assert pool.error_bits() == 0 and all(lc.error_bits() == 0 for lc in c.layers)
    pool.pull()
    assert lengths(c) == [24, 51, 0, 0, 0, 0]
    assert all(read_back(c, 0, [r])[0].shape[0] == c.seqs[r].length for r in c.seqs)


def test_buffers_that_are_gone_are_forgotten():
    c = make_cache(False)
    begin(c, [20, 33], 71)
    a, b, pool = StepBuffers(c, 2), StepBuffers(c, 2), DevicePool(c)
    pool.use(a, [0, 1])
    pool.use(b, [1])
    del b
    c.remove_sequence(1)
    assert a.slot.tolist() == [c.seqs[0].slot, -1]
    pool.use(a, [None, 0])
    c.remove_sequence(0)
    assert a.slot.tolist() == [-1, -1]
    pool.plan(a)
    pool.commit(a)
    assert a.ctx.tolist() == [0, 0] and pool.error_bits() == 0
    pool.pull()
    assert not c.seqs and len(c.free_slots) == 6


def test_a_step_captured_for_fewer_entries_is_refused():
    """A replay after use() of more sequences than the step was captured for would leave the last ones where they are."""
    c = make_cache(False)
    begin(c, [20, 33, 47], 71)
    bufs, pool = StepBuffers(c, 3), DevicePool(c)
    pool.use(bufs, [0, 1])
    step = GraphStep(c, bufs, 0.1, pool=pool)
    step.run_eager()
    step.capture()
    pool.use(bufs, [2, 0, 1])
    for call in (step.replay, step.run_eager):
        with pytest.raises(ValueError, match="entries"):
            call()
    pool.use(bufs, [2])
    step.replay()
    step.replay()
    pool.use(bufs, [1, 2])
    step.replay()
    assert pool.error_bits() == 0
    pool.pull()
    assert lengths(c) == [21, 35, 50]


def test_a_step_takes_no_counts():
    """An entry of a step that brought no token would have its last one written over."""
    c = make_cache(False)
    begin(c, [20, 33], 71)
    bufs, chunks, pool = StepBuffers(c, 2), ChunkBuffers(c, 2, 2, 1), DevicePool(c)
    counts = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    for b in (bufs, chunks):
        pool.use(b, [0, 1])
    with pytest.raises(ValueError, match="one token"):
        pool.plan(bufs, counts)
    pool.plan(chunks, counts)  # the chunk operators write new tokens alone
    pool.commit(chunks)
    pool.pull()
    assert lengths(c) == [21, 33]


@pytest.mark.parametrize("int8", [False, True])
def test_unfused_steps_need_a_plan_of_the_host(int8):
    """The kernels that append and attend apart take block, offset and fill block of each row from an upload; what
    a pool plans does not say them, and the last upload's would be written over."""
    c = make_cache(int8)
    begin(c, [20, 33], 71)
    bufs = StepBuffers(c, 2)
    q, k, v = (rows(80 + i, 2, 2, h) for i, h in enumerate((HEADS[0], HEADS[1], HEADS[1])))
    decode_step(c, bufs, [0, 1], q, k, v, torch.empty_like(q), 0.1)
    unfused = GraphStep(c, bufs, 0.1, fused=False)
    unfused.capture()
    before = [read_back(c, 1, [r]) for r in (0, 1)]
    pool = DevicePool(c)
    pool.use(bufs, [1, 0])
    pool.plan(bufs)
    for call in (lambda: run_layers(c, bufs, q, k, v, torch.empty_like(q), 0.1, "always"), unfused.run_eager, unfused.replay,
                 unfused.capture):
        with pytest.raises(RuntimeError, match="GPU"):
            call()
    torch.cuda.synchronize()
    pool.pull()
    assert lengths(c) == [21, 34]
    for r in (0, 1):
        assert all(torch.equal(x, y) for x, y in zip(read_back(c, 1, [r])[:2], before[r][:2]))
    decode_step(c, bufs, [0, 1], q, k, v, torch.empty_like(q), 0.1)
    assert lengths(c) == [22, 35]


def test_only_buffers_that_were_used_with_the_pool_are_planned():
    """Slots that are not from this pool's use() -- zeros, an upload's, an earlier pool's -- name sequences
    that nobody asked for."""
    c = make_cache(False)
    begin(c, [20, 33], 71)
    fresh, steps = ChunkBuffers(c, 1, 4, 4), StepBuffers(c, 2)
    q, k, v = (rows(80 + i, 2, 2, h) for i, h in enumerate((HEADS[0], HEADS[1], HEADS[1])))
    decode_step(c, steps, [0, 1], q, k, v, torch.empty_like(q), 0.1)
    pool = DevicePool(c)
    for again in (False, True):
        for bufs in (fresh, steps):
            for call in (pool.plan, pool.commit):
                with pytest.raises(ValueError, match="use"):
                    call(bufs)
        if not again:
            pool.use(fresh, [1])
            pool.use(steps, [0])
            pool.plan(fresh)
            pool.commit(fresh)
            pool.pull()
            pool = DevicePool(c)
    assert pool.error_bits() == 0
    pool.pull()
    assert lengths(c) == [21, 35]


def test_buffers_of_another_cache_are_refused():
    """They would get this cache's blocks, and steps over them read and write the other's."""
    c, other = make_cache(False), make_cache(False)
    begin(c, [20, 33], 71)
    begin(other, [5], 72)
    pool = DevicePool(c)
    for bufs in (StepBuffers(other, 2), ChunkBuffers(other, 2, 4, 2)):
        with pytest.raises(ValueError, match="another cache"):
            pool.use(bufs, [0])
    pool.pull()
    assert lengths(c) == [20, 33] and lengths(other) == [5]


def test_error_bits_of_plans_on_another_stream():
    """They wait for every stream: a plan that is still to come on another one has its say."""
    c = make_cache(False, blocks=5)
    begin(c, [33, 30], 71)
    bufs, pool, side = ChunkBuffers(c, 2, 8, 4), DevicePool(c), torch.cuda.Stream()
    pool.use(bufs, [0, 1])
    counts = torch.tensor([4, 4], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # cycles: some 10 ms
        pool.plan(bufs, counts)  # the second sequence's third block is not there
    assert pool.error_bits() == pkv.PKV_DEVERR_OOM
    assert pool.error_bits() == 0
    pool.pull()
    assert lengths(c) == [33, 30]


@pytest.mark.parametrize("pdl", [False, True])
def test_launches_of_a_planned_step(pdl):
    c = make_cache(False)
    begin(c, [20, 33], 71)
    bufs, pool = StepBuffers(c, 2), DevicePool(c)
    pool.use(bufs, [0, 1])
    pkv.pkv_set_programmatic_launch(pdl)
    try:
        step = GraphStep(c, bufs, 0.1, pool=pool)
        step.run_eager()
        graph, n = torch.cuda.CUDAGraph(keep_graph=True), ctypes.c_size_t(0)
        with torch.cuda.graph(graph):
            step.run_eager()
        assert ctypes.CDLL("libcuda.so.1").cuGraphGetNodes(ctypes.c_void_p(graph.raw_cuda_graph()), None, ctypes.byref(n)) == 0
        assert step.launches_per_step() == n.value == c.L + 2 + pdl
    finally:
        pkv.pkv_set_programmatic_launch(False)
    assert GraphStep(c, bufs, 0.1).launches_per_step() == c.L
    pool.pull()


def test_what_the_gpu_has_put_into_the_slots_stays():
    """A program that stops sequences on the GPU, by an entry of -1, removes another one: its own entries stay."""
    c = make_cache(False)
    begin(c, [20, 33, 47], 71)
    bufs, pool = StepBuffers(c, 3), DevicePool(c)
    pool.use(bufs, [0, 1, 2])
    bufs.slot[1] = -1
    c.remove_sequence(0)
    assert bufs.slot.tolist() == [-1, -1, c.seqs[2].slot]
    pool.plan(bufs)
    pool.commit(bufs)
    assert pool.error_bits() == 0
    pool.pull()
    assert lengths(c) == [33, 48]


@pytest.mark.parametrize("int8", [False, True])
def test_steps_over_several_axes_captured_with_their_plan(int8):
    """Plan, positions, turn, append, attention and commit of one token a sequence in one graph: what the same calls do one
    by one, sequences that end and begin among the replays."""
    a, b = make_cache(int8), make_cache(int8)
    f, factor = rope_frequencies(HEADS[2])
    runs = []
    for c in (a, b):
        begin(c, [20, 33, 47], 71)
        chunks, where = ChunkBuffers(c, 4, 4, 1), AxisPositions(c, 4, 4)
        where.set(0, [(5, 0, 0, 1), (1, 4, 4, 1)])
        for r in (1, 2):
            where.set(r, [(2, 2, 3, 2)])
        rope = pkv.make_rope_axes(torch.as_tensor(f).cuda(), axis_pairs((16, 24, 24)), positions=where.positions, scale=factor)
        q, k, v = (torch.zeros((2, 4, h, HEADS[2]), dtype=torch.bfloat16, device="cuda") for h in (HEADS[0], HEADS[1], HEADS[1]))
        out, pool = torch.zeros_like(q), DevicePool(c)

        def step(c=c, chunks=chunks, where=where, rope=rope, q=q, k=k, v=v, out=out, pool=pool):
            pool.plan(chunks)
            where.update(chunks)
            run_chunk(c, chunks, q, k, v, out, HEADS[2] ** -0.5, rope)
            pool.commit(chunks)
        runs.append((c, chunks, where, q, k, v, out, pool, step))
    graph = None
    for n in range(24):
        for which, (c, chunks, where, q, k, v, out, pool, step) in enumerate(runs):
            if n == 0:
                pool.use(chunks, [2, 0, None, 1])
            if n == 9:
                c.remove_sequence(0)  # (its entry is one without a sequence until the next use)
            if n == 13:
                c.add_sequence(8)
                where.set(8, [(3, 0, 0, 1), (1, 2, 2, 1)])
                pool.use(chunks, [8, None, 2, 1])
            for i, x in enumerate((q, k, v)):
                x.copy_(rows(500 + 3 * n + i, 2, 4, x.shape[2]))
            if which == 0 or n == 0:
                step()
            else:
                if graph is None:
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph):
                        step()
                graph.replay()
        live = int(runs[0][1].starts[-1].item())
        assert live == (2 if 9 <= n < 13 else 3) and torch.equal(runs[0][6][:, :live], runs[1][6][:, :live])
    for c, _, where, *_, pool, _ in runs:
        assert pool.error_bits() == 0 and where.err.item() == 0 and all(lc.error_bits() == 0 for lc in c.layers)
        pool.pull()
    caches_are_the_same(a, b)
    assert lengths(b) == [57, 71, 11]


def test_waits_are_for_the_device_that_holds_the_pool(monkeypatch):
    """Not for the one that is current: with several GPUs that may be another."""
    waited, wait = [], torch.cuda.synchronize
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: (waited.append(device), wait(device)))
    c = make_cache(False)
    begin(c, [20], 71)
    here = c.layers[0].k_pool.device
    chunks, bufs = ChunkBuffers(c, 1, 20, 20), StepBuffers(c, 1)
    waited.clear()
    chunks.workspace(c.layers[0].desc, 0, 0)
    AxisPositions(c, 4, 4)
    pool = DevicePool(c)
    pool.use(bufs, [0])
    pool.plan(bufs)
    pool.commit(bufs)
    assert pool.error_bits() == 0
    pool.pull()
    assert waited == [here] * 6 and lengths(c) == [21]
