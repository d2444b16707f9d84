"""Steps that are planned on the GPU, prompts with positions on several axes that
attend from their rows, and the two together, against the host-planned path and fp64."""

import numpy as np
import pytest
import torch

from chunk_ref import assert_attention, turned
from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv
from paged_kv_cache_56_gb300.runtime import (AxisPositions, ChunkBuffers, DevicePool, GraphStep, PagedKVCache, StepBuffers,
                                             axis_pairs, decode_step, extend_step, read_back, rope_frequencies, run_chunk)
from test_gpu_axes import positions_of, turned_axes
from test_gpu_chunk import same

pytestmark = pytest.mark.gpu
HEADS = (8, 2, 128)


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def make_cache(int8, L=2, blocks=96, bs=16, slots=6):
    order = torch.randperm(blocks, generator=torch.Generator().manual_seed(5)).numpy()
    return PagedKVCache(L, blocks, *HEADS, bs, int8, max_slots=slots, max_blocks_per_seq=24, initial_order=order)


def rows(seed, L, T, heads):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((L, T, heads, HEADS[2]), generator=g).to(torch.bfloat16).cuda()


def caches_are_the_same(a, b):
    assert {r: a.table(r) for r in a.seqs} == {r: b.table(r) for r in b.seqs}
    assert {r: s.length for r, s in a.seqs.items()} == {r: s.length for r, s in b.seqs.items()}
    assert pkv.pkv_free_list(a.alloc) == pkv.pkv_free_list(b.alloc)
    for li in range(a.L):
        for r in a.seqs:
            x, y = read_back(a, li, [r]), read_back(b, li, [r])
            assert same(x[0], y[0]) and same(x[1], y[1])


def begin(cache, lens, seed):
    """The same prompts in any cache."""
    for r in range(len(lens)):
        cache.add_sequence(r)
    bufs = ChunkBuffers(cache, len(lens), sum(lens), max(lens))
    q, k, v = (rows(seed + i, cache.L, sum(lens), n) for i, n in enumerate((HEADS[0], HEADS[1], HEADS[1])))
    extend_step(cache, bufs, list(range(len(lens))), lens, q, k, v, torch.empty_like(q), HEADS[2] ** -0.5)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("pdl", [False, True])
def test_decode_steps_replayed_without_the_host(int8, pdl):
    """A captured step with its plan and commit, replayed 40 times, does what host-planned steps do."""
    lens, scale = [37, 16, 1, 60], HEADS[2] ** -0.5
    host, gpu = make_cache(int8), make_cache(int8)
    for c in (host, gpu):
        begin(c, lens, 7)
    hb, gb = (StepBuffers(c, 4, split_tokens=64) for c in (host, gpu))
    pool = DevicePool(gpu)
    order = [2, 0, 3, 1]
    pool.use(gb, order)
    pkv.pkv_set_programmatic_launch(pdl)
    try:
        step = GraphStep(gpu, gb, scale, pool=pool)
        for n in range(41):
            q, k, v = (rows(100 + 3 * n + i, 2, 4, h) for i, h in enumerate((HEADS[0], HEADS[1], HEADS[1])))
            want = torch.empty_like(q)
            decode_step(host, hb, order, q, k, v, want, scale)
            step.q.copy_(q)
            step.k.copy_(k)
            step.v.copy_(v)
            if n == 0:
                step.run_eager()
                got = step.out.clone()
                step.capture()
            else:
                step.replay()
                got = step.out
            # (the host path's kernels are the unfused ones: the same numbers)
            assert_same_rows(got, want)
        torch.cuda.synchronize()
    finally:
        pkv.pkv_set_programmatic_launch(False)
    assert pool.error_bits() == 0 and all(lc.error_bits() == 0 for lc in gpu.layers)
    with pytest.raises(RuntimeError, match="GPU"):
        gpu.table(0)
    pool.pull()
    caches_are_the_same(gpu, host)
    # the host goes on where the GPU stopped
    q, k, v = (rows(900 + i, 2, 4, h) for i, h in enumerate((HEADS[0], HEADS[1], HEADS[1])))
    outs = []
    for c, b in ((host, hb), (gpu, gb)):
        outs.append(torch.empty_like(q))
        decode_step(c, b, order, q, k, v, outs[-1], scale)
    assert torch.equal(*outs)
    caches_are_the_same(gpu, host)


def assert_same_rows(got, want):
    """Fused and unfused decode kernels: the same values in another order of sums, both within
    2^-8 of the result's rounding and the weights' two bf16 parts: 2^-7 of the row's size holds both."""
    g, w = got.float(), want.float()
    assert ((g - w).abs() <= 2.0 ** -7 * w.abs().amax(dim=-1, keepdim=True)).all()


@pytest.mark.parametrize("int8", [False, True])
def test_entries_without_a_sequence_and_sequences_that_end(int8):
    scale = HEADS[2] ** -0.5
    host, gpu = make_cache(int8), make_cache(int8)
    for c in (host, gpu):
        begin(c, [20, 33, 47], 11)
    hb, gb = StepBuffers(host, 4), StepBuffers(gpu, 4)
    pool = DevicePool(gpu)
    step = None
    batches = [[0, None, 1, 2]] * 3 + [[None, 2, None, 0]] * 20 + [[5, 0, None, 2]] * 5
    for n, order in enumerate(batches):
        live = [i for i, r in enumerate(order) if r is not None]
        if order[0] == 5 and 5 not in gpu.seqs:
            for c in (host, gpu):
                c.remove_sequence(1)
                c.add_sequence(5)
        q, k, v = (rows(200 + 3 * n + i, 2, 4, h) for i, h in enumerate((HEADS[0], HEADS[1], HEADS[1])))
        part = [x[:, live].contiguous() for x in (q, k, v)]
        want = torch.empty_like(part[0])
        decode_step(host, hb, [order[i] for i in live], *part, want, scale)
        pool.use(gb, order)
        if step is None:
            step = GraphStep(gpu, gb, scale, pool=pool)
        step.q.copy_(q)
        step.k.copy_(k)
        step.v.copy_(v)
        if step.graph is None:
            step.run_eager()
            got = step.out.clone()
            step.capture()
        else:
            step.replay()
            got = step.out
        assert_same_rows(got[:, live], want)
        empty = [i for i in range(4) if i not in live]
        assert (got[:, empty] == 0).all()
    assert pool.error_bits() == 0 and all(lc.error_bits() == 0 for lc in gpu.layers)
    pool.pull()
    caches_are_the_same(gpu, host)


def test_a_plan_that_cannot_be_made_leaves_the_cache_alone():
    c = make_cache(False, blocks=8)
    begin(c, [60, 60], 13)  # every block is held
    before = [read_back(c, 0, [r])[0] for r in (0, 1)]
    bufs = StepBuffers(c, 2)
    pool = DevicePool(c)
    pool.use(bufs, [0, 1])
    step = GraphStep(c, bufs, 0.1, pool=pool)
    step.k.fill_(3.0)
    step.run_eager()
    step.capture()
    for _ in range(12):  # the ninth step would need a block each
        step.replay()
    assert pool.error_bits() == pkv.PKV_DEVERR_OOM and pool.error_bits() == 0
    assert (step.out == 0).all()
    pool.pull()
    assert [c.seqs[r].length for r in (0, 1)] == [64, 64]
    for r in (0, 1):
        k = read_back(c, 0, [r])[0]
        assert torch.equal(k[:60], before[r]) and (k[60:] == 3).all()


SEGMENTS = {0: [(11, 0, 0, 1), (1, 6, 9, 1), (5, 0, 0, 1), (3, 4, 5, 2)], 1: [(1, 0, 0, 1)], 2: [], 3: [(2, 8, 8, 3)]}


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), ([24, 0], [4, 0])])
def test_prompts_with_images_then_steps_all_planned_on_the_gpu(int8, window, sinks):
    """Prompts whose blocks, positions, rotary turn and attention are worked out on the GPU, then drafted
    tokens and single ones over the cache; against fp64 from the definitions."""
    hq, hkv, d = HEADS
    L, lens, scale = 2, [140, 1, 77, 250], d ** -0.5
    cache = make_cache(int8, L=L)
    for r in range(4):
        cache.add_sequence(r)
    prompt_bufs, step_bufs = ChunkBuffers(cache, 4, 512, 256), ChunkBuffers(cache, 4, 12, 3)
    where = {b: AxisPositions(cache, b.max_tokens, 6) for b in (prompt_bufs, step_bufs)}
    f, factor = rope_frequencies(d)
    axis = axis_pairs((16, 24, 24), in_turn=int8)
    ropes = {}
    for b, w in where.items():
        for r in range(4):
            w.set(r, SEGMENTS[r])
        ropes[b] = pkv.make_rope_axes(torch.as_tensor(f).cuda(), axis, positions=w.positions, scale=factor)
    win = window if isinstance(window, list) else [window] * L
    snk = sinks if isinstance(sinks, list) else [sinks] * L
    pool = DevicePool(cache)
    history = {(li, r): [np.zeros((0, hkv, d))] * 2 for li in range(L) for r in range(4)}
    length = [0] * 4

    def go(bufs, counts, accepted, seed, prompts):
        T = sum(counts)
        q, k, v = (rows(seed + i, L, bufs.max_tokens, h) for i, h in enumerate((hq, hkv, hkv)))
        q0, k0 = q.clone(), k.clone()
        out = torch.full_like(q, 7.0)
        pool.use(bufs, [3, 0, 2, 1])
        order = [3, 0, 2, 1]
        counts = [counts[r] for r in order]
        pool.plan(bufs, torch.tensor(counts, dtype=torch.int32, device="cuda"))
        where[bufs].update(bufs)
        run_chunk(cache, bufs, q, k, v, out, scale, ropes[bufs], window, sinks, prompts=prompts)
        pool.commit(bufs, None if accepted is None else torch.tensor([accepted[r] for r in order], dtype=torch.int32, device="cuda"))
        assert (out[:, T:] == 7).all()
        at = 0
        for r, n in zip(order, counts):
            pos = positions_of(SEGMENTS[r], length[r] + n)[:, length[r]:]
            assert np.array_equal(where[bufs].positions[:, at:at + n].cpu().numpy(), pos)
            for li in range(L):
                kt = turned_axes(k0[li, at:at + n].cpu(), pos, axis, f, False, factor)
                qt = q[li, at:at + n].double().cpu().numpy()  # turned in place
                want_q = turned_axes(q0[li, at:at + n].cpu(), pos, axis, f, False, factor)
                assert (np.abs(qt - want_q) <= 2.0 ** -8 * np.abs(want_q) + 2.0 ** -18).all()
                if prompts:
                    rounded = k[li, at:at + n].double().cpu().numpy()
                    assert (np.abs(rounded - kt) <= 2.0 ** -8 * np.abs(kt) + 2.0 ** -18).all()
                    hist = [rounded, v[li, at:at + n].double().cpu().numpy()]
                else:
                    hist = cache_rows(cache, pool, li, r, length[r] + n)
                for i in range(n):
                    p = length[r] + i
                    t = np.arange(p + 1)
                    if win[li]:
                        t = t[(p - t < win[li]) | (t < snk[li])]
                    x = np.einsum("hgd,thd->hgt", qt[i].reshape(hkv, -1, d), hist[0][t]) * scale
                    w = np.exp(x - x.max(-1, keepdims=True))
                    w /= w.sum(-1, keepdims=True)
                    ref = np.einsum("hgt,thd->hgd", w, hist[1][t]).reshape(hq, d)
                    mag = np.einsum("hgt,thd->hgd", w, np.abs(hist[1][t])).reshape(hq, d)
                    assert_attention(out[li, at + i], ref, mag, f"layer {li} sequence {r} row {i}")
            at += n
        for r in range(4):
            length[r] += dict(zip(order, counts))[r] if accepted is None else accepted[r]

    go(prompt_bufs, lens, None, 31, True)
    if not int8:
        go(step_bufs, [3, 3, 3, 3], [2, 0, 3, 1], 41, False)
    for n in range(3):
        go(step_bufs, [1, 1, 0, 1], None, 51 + 10 * n, False)
    assert pool.error_bits() == 0 and all(lc.error_bits() == 0 for lc in cache.layers)
    assert all(int(w.err.item()) == 0 for w in where.values())
    pool.pull()
    assert [cache.seqs[r].length for r in range(4)] == length


def cache_rows(cache, pool, li, r, n):
    """K and V rows of tokens 0 .. n-1 of a sequence, as the cache holds them now."""
    slot = cache.seqs[r].slot
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = pkv.make_batch(dev([0, n]), pool.tables[slot][None].contiguous(), dev([n]), dev([slot]), num_tokens=n, max_tokens=n)
    out = [torch.empty((n, cache.hkv, cache.d), dtype=torch.float32, device="cuda") for _ in range(2)]
    pkv.pkv_gather_kv(cache.layers[li].desc, batch, *out)
    return [x.double().cpu().numpy() for x in out]


@pytest.mark.parametrize("int8", [False, True])
def test_host_planned_prompts_attend_from_their_rows(int8):
    """extend_step(prompts=True) with a one-axis rotary turn: the cache is the one the plain path leaves, the outputs
    those of the rows."""
    hq, hkv, d = HEADS
    a, b = make_cache(int8), make_cache(int8)
    f, factor = rope_frequencies(d)
    rope = pkv.make_rope(torch.as_tensor(f).cuda(), scale=factor)
    lens = [130, 3, 64]
    outs = []
    for c in (a, b):
        for r in range(3):
            c.add_sequence(r)
        bufs = ChunkBuffers(c, 3, 200, 130)
        q, k, v = (rows(61 + i, 2, 200, h) for i, h in enumerate((hq, hkv, hkv)))
        outs.append(torch.full_like(q, 7.0))
        extend_step(c, bufs, [0, 1, 2], lens, q, k, v, outs[-1], d ** -0.5, rope, 40, 3, prompts=c is b)
    caches_are_the_same(a, b)
    assert (outs[1][:, 197:] == 7).all()
    k0 = rows(62, 2, 200, hkv)
    for li in range(2):
        at = 0
        for n in lens:
            kt = turned(k0[li, at:at + n].cpu(), np.arange(n), f, False, factor)
            assert (np.abs(k[li, at:at + n].double().cpu().numpy() - kt) <= 2.0 ** -8 * np.abs(kt) + 2.0 ** -18).all()
            for i in range(n):
                t = np.arange(i + 1)
                t = t[(i - t < 40) | (t < 3)]
                kk, vv = (x[li, at:at + n].double().cpu().numpy()[t] for x in (k, v))
                x = np.einsum("hgd,thd->hgt", q[li, at + i].double().cpu().numpy().reshape(hkv, -1, d), kk) * d ** -0.5
                w = np.exp(x - x.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                ref, mag = (np.einsum("hgt,thd->hgd", w, y).reshape(hq, d) for y in (vv, np.abs(vv)))
                assert_attention(outs[1][li, at + i], ref, mag)
            at += n
    with pytest.raises(ValueError, match="has tokens"):
        extend_step(b, bufs, [0], [1], q, k, v, outs[1], d ** -0.5, rope, prompts=True)


def test_what_a_pool_refuses():
    c = make_cache(False)
    begin(c, [20, 33], 71)
    c.fork(0, 7)
    with pytest.raises(ValueError, match="forks"):
        DevicePool(c)
    c.remove_sequence(7)
    c.plan_chunk([0], [3])
    with pytest.raises(ValueError, match="committed"):
        DevicePool(c)
    c.commit_chunk([0], [0])
    bufs, step = ChunkBuffers(c, 2, 8, 4), StepBuffers(c, 2)
    pool = DevicePool(c)
    for call in (lambda: c.plan_step([0]), lambda: c.plan_chunk([0], [1]), lambda: c.commit_step([0]), lambda: c.table(0),
                 lambda: c.commit_chunk([0], [0]), lambda: c.fork(0, 9), lambda: read_back(c, 0, [0])):
        with pytest.raises(RuntimeError, match="GPU"):
            call()
    for call in (lambda: c.add_sequence(9, n_blocks=1), lambda: pool.use(bufs, [0, 0]), lambda: pool.use(bufs, [0, 1, 0]),
                 lambda: pool.plan(step), lambda: pool.release([1, 1]),
                 lambda: GraphStep(c, step, 0.1, fused=False, pool=pool)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(pkv.PkvError):
        c.add_sequence(0)
    pool.pull()
    with pytest.raises(RuntimeError):
        pool.pull()
    assert len(c.table(0)) == 2 and c.seqs[1].length == 33 and len(c.free_slots) == 4
