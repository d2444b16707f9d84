"""Batches planned on the GPU against the pool's definition in plain lists and
against the host allocator."""

import random

import numpy as np
import pytest
import torch

from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv
from plan_ref import DevicePoolOf, PoolModel, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def random_batch(rng, m, B, most, pad=True):
    slots = rng.sample(range(m.max_slots), min(B, m.max_slots))
    slots += [-1] * (B - len(slots))
    if pad:
        slots = [s if rng.random() > 0.15 else -1 for s in slots]
    rng.shuffle(slots)
    room = m.N - sum(map(len, m.lists))
    counts = []
    for s in slots:
        n = 0 if s == -1 else rng.choice([0, 1, 1, rng.randint(0, most), m.bs])
        n = min(n, most, m.max_blocks * m.bs - (m.lens[s] if s != -1 else 0))
        if s != -1:
            need = max(0, -(-(m.lens[s] + n) // m.bs) - len(m.lists[s]))
            if need > room:
                n, need = 0, 0
            room -= need
        counts.append(n)
    return slots, counts


@pytest.mark.parametrize("B,max_slots,max_blocks,bs,wide", [
    (1, 1, 1, 16, True), (4, 5, 8, 16, True), (7, 9, 13, 64, True), (33, 40, 36, 16, False), (130, 200, 64, 16, True),
    (512, 600, 12, 16, True), (513, 600, 7, 64, False), (1500, 1600, 20, 16, True),
])
def test_walks_of_plans_commits_and_releases(B, max_slots, max_blocks, bs, wide):
    """Plans (some made twice), commits of parts, releases: arrays, lists, ring and lengths as the definition has them."""
    rng = random.Random(B)
    N = max(2, max_slots * max_blocks // 3)
    order = list(range(N))
    rng.shuffle(order)
    for int8 in (False, True):
        m = PoolModel(max_slots, max_blocks, N, bs, int8, order)
        most = 3 * bs
        g = DevicePoolOf(m, B, B * most, most, head=rng.randrange(N), wide=wide)
        for turn in range(12):
            slots, counts = random_batch(rng, m, B, most)
            ds, dc = dev(slots), dev(counts)
            want = m.plan(slots, counts, B * most, most)
            assert isinstance(want, dict)
            pkv.pkv_plan_batch(g.pool, ds, g.plan_desc, dc)
            assert g.error() == 0
            g.check_plan(want)
            g.check_state()
            if turn % 3 == 0:  # again: everything is held already
                pkv.pkv_plan_batch(g.pool, ds, g.plan_desc, dc)
                g.check_plan(want)
                g.check_state()
            accepted = counts if turn % 2 else [rng.randint(-1, n + 1) if n else 0 for n in counts]
            bits = m.commit(slots, counts, accepted)
            pkv.pkv_commit_batch(g.pool, ds, g.plan_desc, None if turn % 2 else dev(accepted))
            assert g.error() == bits
            g.check_state()
            gone = [s if rng.random() < 0.3 else -1 for s in slots]
            assert m.release(gone) == 0
            pkv.pkv_release_batch(g.pool, dev(gone))
            assert g.error() == 0
            g.check_state()


def test_single_tokens_are_planned_without_counts():
    m = PoolModel(6, 4, 24, 16)
    g = DevicePoolOf(m, 3, 3, 1)
    for step in range(64):
        slots = [5, -1, 2]
        want = m.plan(slots, [1, 1, 1], 3, 1)
        pkv.pkv_plan_batch(g.pool, dev(slots), g.plan_desc)
        g.check_plan(want)
        m.commit(slots, [1, 1, 1], [1, 1, 1])
        pkv.pkv_commit_batch(g.pool, dev(slots), g.plan_desc)
    g.check_state()
    assert m.plan([5, -1, 2], [1, 1, 1], 3, 1) == pkv.PKV_DEVERR_CTX_LEN  # 64 tokens are all they may have
    pkv.pkv_plan_batch(g.pool, dev([5, -1, 2]), g.plan_desc)
    assert g.error() == pkv.PKV_DEVERR_CTX_LEN
    g.check_empty_plan()
    g.check_state()


@pytest.mark.parametrize("B", [4, 700])
def test_what_cannot_be_planned_changes_nothing(B):
    m = PoolModel(B + 2, 6, 3 * B + 20, 16)
    g = DevicePoolOf(m, B, 20 * B, 60)
    first = list(range(B))
    m.plan(first, [17] * B, 20 * B, 60)
    pkv.pkv_plan_batch(g.pool, dev(first), g.plan_desc, dev([17] * B))
    m.commit(first, [17] * B, [17] * B)
    pkv.pkv_commit_batch(g.pool, dev(first), g.plan_desc)
    zeros = [0] * B

    def put(a, **kw):
        a = list(a)
        for i, x in kw.items():
            a[int(i[1:])] = x
        return a
    last = f"i{B - 1}"
    for slots, counts, bits in [
            (put(first, **{last: 0}), zeros, pkv.PKV_DEVERR_SLOT),            # the same slot twice
            (put(first, i1=B + 2), zeros, pkv.PKV_DEVERR_SLOT), (put(first, i1=-2), zeros, pkv.PKV_DEVERR_SLOT),
            (first, put(zeros, **{last: -1}), pkv.PKV_DEVERR_BATCH), (first, put(zeros, i0=61), pkv.PKV_DEVERR_BATCH),
            (first, [21] * B, pkv.PKV_DEVERR_BATCH),                          # more rows than there are
            (first, put(zeros, i2=2 ** 31 - 1), pkv.PKV_DEVERR_BATCH),
            # 122 rows: too many for 4 entries, fine for 700
            (put(first, i0=-1), put([15 + 16] * 4 + [0] * (B - 4), i1=60), pkv.PKV_DEVERR_BATCH if B == 4 else 0)]:
        want = m.plan(slots, counts, 20 * B, 60)
        assert want == bits if bits else isinstance(want, dict)
        pkv.pkv_plan_batch(g.pool, dev(slots), g.plan_desc, dev(counts))
        assert g.error() == bits
        if bits:
            g.check_empty_plan()
            # nor does a commit of it
            pkv.pkv_commit_batch(g.pool, dev(first), g.plan_desc)
            assert g.error() == 0
        else:
            g.check_plan(want)
        g.check_state()
    # more blocks than are free: none is taken
    have = len(m.free)
    m2 = m.plan(first, [19] * B, 20 * B, 60)
    pkv.pkv_plan_batch(g.pool, dev(first), g.plan_desc, dev([19] * B))
    if isinstance(m2, dict):
        g.check_plan(m2)
    else:
        assert have < B and g.error() == pkv.PKV_DEVERR_OOM
        g.check_empty_plan()
    g.check_state()
    for gone in (put(first, **{last: 0}), put(first, i0=B + 2), put(first, i0=-3)):
        assert m.release(gone) == pkv.PKV_DEVERR_SLOT
        pkv.pkv_release_batch(g.pool, dev(gone))
        assert g.error() == pkv.PKV_DEVERR_SLOT
        g.check_state()


def test_too_few_free_blocks():
    m = PoolModel(8, 10, 20, 16)
    g = DevicePoolOf(m, 8, 8 * 160, 160, head=13)
    for counts, ok in (([30] * 8, True), ([1] * 8, True), ([1] * 4 + [65] * 4, False), ([33, 0, 0, 0, 0, 0, 0, 0], True),
                       ([16, 0, 0, 0, 0, 0, 0, 1], True)):
        slots = list(range(8))
        want = m.plan(slots, counts, 8 * 160, 160)
        assert isinstance(want, dict) == ok
        pkv.pkv_plan_batch(g.pool, dev(slots), g.plan_desc, dev(counts))
        if ok:
            assert g.error() == 0
            g.check_plan(want)
            m.commit(slots, counts, counts)
        else:
            assert want == g.error() == pkv.PKV_DEVERR_OOM
            g.check_empty_plan()
        pkv.pkv_commit_batch(g.pool, dev(slots), g.plan_desc)
        assert g.error() == 0
        g.check_state()


def test_a_plan_is_committed_once():
    m = PoolModel(2, 4, 8, 16)
    g = DevicePoolOf(m, 2, 16, 8)
    pkv.pkv_plan_batch(g.pool, dev([1, 0]), g.plan_desc, dev([5, 0]))
    m.plan([1, 0], [5, 0], 16, 8)
    m.commit([1, 0], [5, 0], [3, 0])
    pkv.pkv_commit_batch(g.pool, dev([1, 0]), g.plan_desc, dev([3, 7]))  # entry 1 brought nothing: not looked at
    assert g.error() == 0
    g.check_state()
    pkv.pkv_commit_batch(g.pool, dev([1, 0]), g.plan_desc, dev([3, 0]))
    assert g.error() == pkv.PKV_DEVERR_CTX_LEN
    g.check_state()


def test_lists_that_do_not_hold_together():
    m = PoolModel(3, 4, 8, 16)
    g = DevicePoolOf(m, 2, 16, 8)
    for lens, held in ((5, 0), (-1, 0), (0, 5), (0, -1), (17, 1)):
        g.lens[1], g.held[1] = lens, held
        for call in (lambda: pkv.pkv_plan_batch(g.pool, dev([1, 0]), g.plan_desc, dev([1, 1])),
                     lambda: pkv.pkv_release_batch(g.pool, dev([1, 0]))):
            call()
            assert g.error() == pkv.PKV_DEVERR_CTX_LEN
        g.lens[1], g.held[1] = 0, 0
        g.check_state()
    g.state[1] = 9  # more free blocks than there are
    pkv.pkv_plan_batch(g.pool, dev([1, 0]), g.plan_desc, dev([1, 1]))
    assert g.error() == pkv.PKV_DEVERR_CTX_LEN
    g.state[1] = 8
    g.held[2] = 1  # a block given back that the ring already has
    g.tables[2, 0] = 3
    pkv.pkv_release_batch(g.pool, dev([2]))
    assert g.error() == pkv.PKV_DEVERR_CTX_LEN


def test_the_host_allocator_takes_the_same_blocks():
    """The same requests planned here and by the runtime's host plan: the same tables, in the same order."""
    from paged_kv_cache_56_gb300.runtime import PagedKVCache
    rng = random.Random(3)
    order = list(range(60))
    rng.shuffle(order)
    c = PagedKVCache(1, 60, 4, 2, 64, 16, False, max_slots=6, max_blocks_per_seq=12, initial_order=np.array(order))
    m = PoolModel(6, 12, 60, 16, order=order)
    g = DevicePoolOf(m, 6, 600, 100)
    for r in range(6):
        c.add_sequence(r)
    for _ in range(8):
        reqs = rng.sample(range(6), 4)
        counts = [rng.randint(0, 40) if c.seqs[r].length < 100 else 0 for r in reqs]
        try:
            p = c.plan_chunk(reqs, counts)
        except pkv.PkvError:
            continue
        slots = [c.seqs[r].slot for r in reqs] + [-1, -1]
        pkv.pkv_plan_batch(g.pool, dev(slots), g.plan_desc, dev(counts + [0, 0]))
        assert g.error() == 0
        assert np.array_equal(g.out["tables"][:4].cpu().numpy(), p.tables)
        assert g.out["starts"][:5].tolist() == p.starts.tolist() and g.out["ctx"][:4].tolist() == p.ctx_lens.tolist()
        c.commit_chunk(reqs, counts)
        pkv.pkv_commit_batch(g.pool, dev(slots), g.plan_desc)
    c.close()


def test_replayed_and_on_another_stream():
    """Plan and commit captured once: replays walk the sequences on; the slots' array is refilled between them."""
    m = PoolModel(5, 8, 40, 16)
    g = DevicePoolOf(m, 4, 4, 1, head=39)
    slots = dev([4, 0, -1, 2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkv.pkv_plan_batch(g.pool, slots, g.plan_desc)
        pkv.pkv_commit_batch(g.pool, slots, g.plan_desc)
    g.check_state()
    now = [4, 0, -1, 2]
    for step in range(70):
        if step == 30:
            now = [1, 0, 3, -1]
            slots.copy_(dev(now))
        want = m.plan(now, [1] * 4, 4, 1)
        m.commit(now, [1] * 4, [1] * 4)
        graph.replay()
        g.check_plan(want)
    g.check_state()


def test_programmatic_launches():
    m = PoolModel(5, 8, 40, 16)
    g = DevicePoolOf(m, 4, 4, 1)
    slots = dev([4, 0, -1, 2])
    pkv.pkv_set_programmatic_launch(True)
    try:
        for _ in range(40):
            want = m.plan([4, 0, -1, 2], [1] * 4, 4, 1)
            m.commit([4, 0, -1, 2], [1] * 4, [1] * 4)
            pkv.pkv_plan_batch(g.pool, slots, g.plan_desc)
            pkv.pkv_commit_batch(g.pool, slots, g.plan_desc)
    finally:
        pkv.pkv_set_programmatic_launch(False)
    g.check_plan(want)
    g.check_state()
