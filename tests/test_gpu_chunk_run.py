"""The chunk operators together, as a program uses them: prompts written in
chunks, drafted tokens, decode steps, forks, graphs, programmatic launches and
other streams, over layers of both cache types."""

import math

import numpy as np
import pytest
import torch

from chunk_ref import Setup, assert_attention, attention, bf16, quantize_heads, turned
from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv
from paged_kv_cache_56_gb300.runtime import (ChunkBuffers, PagedKVCache, extend_step, read_back, rope_frequencies,
                                             run_chunk)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


class Model:
    """L layers of a cache, and the rows that a model would bring."""

    def __init__(self, heads, bs, int8, blocks=64, seqs=4, max_tokens=400, max_new=300, seed=0):
        self.hq, self.hkv, self.d = heads
        self.int8 = int8
        self.cache = PagedKVCache(len(int8), blocks, *heads, bs, int8, max_slots=seqs, max_blocks_per_seq=blocks // 2)
        self.bufs = ChunkBuffers(self.cache, seqs, max_tokens, max_new)
        self.g = torch.Generator().manual_seed(seed)
        self.scale = 1 / math.sqrt(self.d)
        f, self.factor = rope_frequencies(self.d, 10000.0, stretch=4, trained=256)
        self.f = f
        self.rope = pkv.make_rope(torch.from_numpy(f).cuda(), scale=self.factor)

    def rows(self, n, heads):
        return torch.randn((len(self.int8), n, heads, self.d), generator=self.g).to(torch.bfloat16)

    def step(self, reqs, counts, window, sinks, **kw):
        """One extend_step of new random rows; checks its outputs against fp64 attention over what the cache holds
        afterwards, and that against the rows that were brought."""
        T, n = self.bufs.max_tokens, sum(counts)
        q, k, v = self.rows(T, self.hq), self.rows(T, self.hkv), self.rows(T, self.hkv)
        dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
        out = torch.full((len(self.int8), T, self.hq, self.d), 3.0, dtype=torch.bfloat16, device="cuda")
        before = [self.cache.seqs[r].length for r in reqs]
        plan = extend_step(self.cache, self.bufs, reqs, counts, dq, dk, dv, out, self.scale, self.rope, window, sinks, **kw)
        torch.cuda.synchronize()
        assert pkv.pkv_sync_status([lc.desc for lc in self.cache.layers]) == 0
        assert (out[:, n:] == 3).all()
        pos = np.concatenate([np.arange(b, b + c) for b, c in zip(before, counts)])
        for li in range(len(self.int8)):
            self.check_layer(li, reqs, counts, before, plan, q[li, :n], dq[li, :n].cpu(), k[li, :n], v[li, :n],
                             out[li, :n], window[li] if isinstance(window, list) else window,
                             sinks[li] if isinstance(sinks, list) else sinks, pos)

    def check_layer(self, li, reqs, counts, before, plan, q, q_turned, k, v, out, window, sinks, pos):
        bs = self.cache.bs
        ref = turned(q, pos, self.f, False, self.factor)
        big = q.double().abs().amax(dim=2, keepdim=True).numpy() * self.factor
        # half a bf16 step, and fp32 products and angles
        assert (np.abs(q_turned.double().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * big).all()
        kb, vb, starts = read_back(self.cache, li, reqs, torch.float32)
        kb, vb = kb.cpu().double().numpy(), vb.cpu().double().numpy()
        k_turned = turned(k, pos, self.f, False, self.factor)
        s = Setup.__new__(Setup)  # what attention() needs
        s.new, s.ctx, s.starts, s.B = list(counts), plan.ctx_lens.tolist(), plan.starts, len(reqs)
        s.T, s.hq, s.hkv, s.d, s.G, s.int8 = sum(counts), self.hq, self.hkv, self.d, self.hq // self.hkv, self.int8[li]
        s.q = q_turned
        s.values = {"k": [kb[a:b] for a, b in zip(starts, starts[1:])], "v": [vb[a:b] for a, b in zip(starts, starts[1:])]}
        for b, (c, p0) in enumerate(zip(counts, before)):
            for name, want in (("k", k_turned), ("v", v.double().numpy())):
                got = s.values[name][b][p0:p0 + c]
                w = want[plan.starts[b]:plan.starts[b] + c]
                tol = 2.0 ** -8 * np.abs(w) + 2.0 ** -20 * np.abs(w).max(initial=0)
                if self.int8[li]:
                    # half a step of the block's scale, max / 127 of at most the largest value there is, and its
                    # rounding; the block's maximum may be an earlier token's
                    top = max(np.abs(s.values[name][b]).max(initial=0), np.abs(w).max(initial=0))
                    tol = tol + top * (1 + 2.0 ** -7) / 254
                assert (np.abs(got - w) <= tol).all(), (li, name, b)
        ref, mag = attention(s, window, sinks, self.scale)
        assert_attention(out, ref, mag, f"layer {li} block {bs}")


@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("heads", [(4, 2, 64), (16, 8, 128), (8, 1, 128)])
def test_prompts_drafts_and_steps(heads, bs):
    """A windowed layer, a full one and an INT8 one of each kind, from prompts in chunks to single steps."""
    m = Model(heads, bs, [False, True, True, False], seqs=3, blocks=48, max_tokens=330, max_new=256)
    window, sinks = [50, 0, 33, 0], [4, 0, 20, 0]
    for r in (7, 8, 9):
        m.cache.add_sequence(r)
    m.step([7, 8], [37, 200], window, sinks)
    m.step([9, 7, 8], [5, 100, 57], window, sinks)      # continues inside blocks
    m.step([7, 8, 9], [1, 0, 1], window, sinks)
    m.step([9, 8, 7], [4, 3, 2], window, sinks)         # drafted tokens
    for _ in range(3):
        m.step([8, 9, 7], [1, 1, 1], window, sinks)
    m.cache.fork(7, 10) if m.cache.free_slots else m.cache.remove_sequence(9)
    m.step([7, 8], [6, 70], window, sinks)


def test_forked_sequences_go_their_own_ways():
    m = Model((8, 2, 128), 16, [False, True], seqs=3, blocks=40)
    m.cache.add_sequence(1)
    m.step([1], [45], 0, 0)
    m.cache.fork(1, 2)
    m.step([1, 2], [30, 3], 0, 0)
    m.step([2, 1], [1, 1], 0, 0)
    # the parent's and the child's first 45 tokens are the same rows still
    for li in range(2):
        k, _, st = read_back(m.cache, li, [1, 2], torch.float32)
        n = 32 if m.int8[li] else 45  # (INT8: token 32 .. 44 were quantized with different neighbours)
        assert torch.equal(k[:n], k[st[1]:st[1] + n])


@pytest.mark.parametrize("pdl", [False, True])
def test_captured_chunk_is_replayed_on_other_batches(pdl):
    m = Model((16, 8, 128), 16, [False, True], seqs=4, blocks=64, max_tokens=120, max_new=60)
    pkv.pkv_set_programmatic_launch(pdl)
    try:
        L, T = 2, 120
        q, k, v = m.rows(T, m.hq).cuda(), m.rows(T, m.hkv).cuda(), m.rows(T, m.hkv).cuda()
        out = torch.zeros((L, T, m.hq, m.d), dtype=torch.bfloat16, device="cuda")
        for r in range(4):
            m.cache.add_sequence(r)
        graph = None
        for reqs, counts in (([0, 1], [50, 13]), ([2, 0, 1], [60, 1, 7]), ([3], [33]), ([0, 1, 2, 3], [1, 1, 1, 1]),
                             ([2, 3], [20, 44])):
            plan = m.cache.plan_chunk(reqs, counts)
            m.cache.apply_cow(plan)
            m.bufs.upload(plan)
            n = sum(counts)
            qs, ks, vs = m.rows(T, m.hq), m.rows(T, m.hkv), m.rows(T, m.hkv)
            q.copy_(qs)
            k.copy_(ks)
            v.copy_(vs)
            if graph is None:
                run_chunk(m.cache, m.bufs, q, k, v, out, m.scale, m.rope, 40, 4)
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    run_chunk(m.cache, m.bufs, q, k, v, out, m.scale, m.rope, 40, 4)
            else:
                graph.replay()
            torch.cuda.synchronize()
            assert pkv.pkv_sync_status([lc.desc for lc in m.cache.layers]) == 0
            before = [m.cache.seqs[r].length for r in reqs]
            m.cache.commit_chunk(reqs, counts)
            pos = np.concatenate([np.arange(b, b + c) for b, c in zip(before, counts)])
            for li in range(L):
                m.check_layer(li, reqs, counts, before, plan, qs[li, :n], q[li, :n].cpu(), ks[li, :n], vs[li, :n],
                              out[li, :n], 40, 4, pos)
    finally:
        pkv.pkv_set_programmatic_launch(False)


def test_decode_reads_what_a_chunk_wrote_under_programmatic_launch():
    """pkv_decode_attention reads blocks before its predecessor is done: a chunk written just before must be there."""
    ctx, heads = [3000, 2500], (16, 8, 128)
    s = Setup(5, ctx, ctx, heads, 16, False, appended=False)
    k, v = s.new_rows("k").cuda(), s.new_rows("v").cuda()
    q = torch.randn((2, 16, 128), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    outs = []
    pkv.pkv_set_programmatic_launch(True)
    try:
        for _ in range(5):
            s.lc.k_pool.zero_()
            s.lc.v_pool.zero_()
            out = torch.empty_like(q)
            pkv.pkv_rope_append(s.lc.desc, s.batch, None, None, k, v)
            pkv.pkv_decode_attention(s.lc.desc, q, s.d_table, s.d_ctx, None, 128 ** -0.5, out)
            outs.append(out)
    finally:
        pkv.pkv_set_programmatic_launch(False)
    torch.cuda.synchronize()
    want = torch.empty_like(q)
    pkv.pkv_decode_attention(s.lc.desc, q, s.d_table, s.d_ctx, None, 128 ** -0.5, want)
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("int8", [False, True])
def test_many_ragged_sequences(int8):
    """More sequences than a warp has lanes, some without tokens, some one, some many."""
    rng = np.random.default_rng(3)
    new = rng.choice([0, 1, 1, 2, 15, 16, 17, 40, 90], size=77).tolist()
    ctx = [n + int(rng.integers(0, 60)) for n in new]
    s = Setup(9, new, ctx, (8, 2, 64), 16, int8)
    for window, sinks in ((0, 0), (20, 3)):
        ref, mag = attention(s, window, sinks)
        out = torch.zeros((s.T, s.hq, s.d), dtype=torch.bfloat16, device="cuda")
        split = pkv.pkv_window_split_tokens(s.lc.desc, s.batch, window, sinks)
        n = pkv.pkv_window_ws_bytes(s.lc.desc, s.batch, window, sinks, split)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None
        pkv.pkv_window_attention(s.lc.desc, s.batch, s.q.cuda(), out, window, sinks, 0.125, split, ws)
        assert_attention(out, ref, mag)
    back = [torch.empty((s.T, s.hkv, s.d), dtype=torch.float32, device="cuda") for _ in range(2)]
    pkv.pkv_gather_kv(s.lc.desc, s.batch, *back)
    for name, b in zip("kv", back):
        want = np.concatenate([x[c - m:] for x, m, c in zip(s.values[name], new, ctx)])
        assert torch.equal(b.cpu(), torch.as_tensor(want).float())
    k, v = s.new_rows("k").cuda(), s.new_rows("v").cuda()
    pools = [s.lc.k_pool.clone(), s.lc.v_pool.clone()]
    t = Setup(9, new, ctx, (8, 2, 64), 16, int8, appended=False)  # the same contexts, appended here
    pkv.pkv_rope_append(t.lc.desc, t.batch, None, None, k, v)
    for b in range(s.B):
        full = ctx[b] // 16 if int8 else -(-ctx[b] // 16)
        for i in range(full):
            rows = min(16, ctx[b] - 16 * i)
            for pool, mine in zip(pools, (t.lc.k_pool, t.lc.v_pool)):
                assert torch.equal(pool[s.table[b, i], :, :rows], mine[t.table[b, i], :, :rows])
    assert s.error_bits() == 0 and t.error_bits() == 0


def test_quantizer_over_all_significands():
    """Every bf16 significand of the block's maximum with every significand below it: the oracle's codes and scales."""
    blocks, rng = [], np.random.default_rng(1)
    for top in range(128, 256):
        for e in (0, 5, -12):
            x = np.concatenate([np.arange(128, 256) * 2.0 ** k for k in range(-8, 0)] + [np.arange(128, top + 1) * 1.0])
            x = np.resize(x, 16 * 64) * np.where(rng.random(16 * 64) < 0.5, 1, -1) * 2.0 ** (e - 7)
            blocks.append(x.reshape(16, 1, 64))
    rows = bf16(np.concatenate(blocks))
    n = rows.shape[0]
    s = Setup(1, [n], [n], (1, 1, 64), 16, True, appended=False)
    pkv.pkv_rope_append(s.lc.desc, s.batch, None, None, rows.cuda(), rows.cuda().flip(2).contiguous())
    k, v, sc = s.lc.k_pool.cpu().numpy(), s.lc.v_pool.cpu().numpy(), s.lc.scales.cpu().numpy()
    for i in range(n // 16):
        for kv, (pool, r) in enumerate(((k, rows), (v, rows.flip(2)))):
            code, scale = quantize_heads(r[16 * i:16 * i + 16].transpose(0, 1))
            assert np.array_equal(pool[s.table[0, i]], code), (i, kv)
            assert np.array_equal(sc[s.table[0, i], :, kv], scale), (i, kv)


def test_not_a_number_and_infinite_rows_quantize_as_before():
    rows = torch.randn((48, 2, 64), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    rows[3, 0, 5], rows[20, 1, 9], rows[33, 0, 0] = float("nan"), float("inf"), -float("inf")
    s = Setup(1, [48], [48], (2, 2, 64), 16, True, appended=False)
    pkv.pkv_rope_append(s.lc.desc, s.batch, None, None, rows.cuda(), rows.cuda())
    got = [x.clone() for x in (s.lc.k_pool, s.lc.v_pool, s.lc.scales)]
    ids = torch.as_tensor(s.table[0, :3].copy()).cuda()
    pkv.pkv_quantize_blocks_from(s.lc.desc, rows.cuda(), rows.cuda(), ids)
    for a, b in zip(got, (s.lc.k_pool, s.lc.v_pool, s.lc.scales)):
        assert torch.equal(a.view(torch.int8), b.view(torch.int8))


def test_another_stream():
    s = Setup(2, [40, 3], [90, 64], (8, 2, 128), 16, True)
    ref, mag = attention(s, 30, 4)
    q, out = s.q.cuda(), torch.zeros((s.T, s.hq, s.d), dtype=torch.bfloat16, device="cuda")
    back = [torch.empty((s.T, s.hkv, s.d), dtype=torch.float32, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkv.pkv_window_attention(s.lc.desc, s.batch, q, out, 30, 4, s.d ** -0.5, stream=side)
    with torch.cuda.stream(side):
        pkv.pkv_gather_kv(s.lc.desc, s.batch, *back)
    side.synchronize()
    assert_attention(out, ref, mag)
    assert torch.isfinite(back[0]).all()


def test_window_agrees_with_decode_attention():
    s = Setup(3, [1, 1, 1], [500, 64, 7], (16, 8, 128), 16, True)
    ref, mag = attention(s, 0, 0)
    q, out = s.q.cuda(), torch.empty((3, 16, 128), dtype=torch.bfloat16, device="cuda")
    pkv.pkv_decode_attention(s.lc.desc, q, s.d_table, s.d_ctx, s.d_slots, s.d ** -0.5, out)
    assert_attention(out, ref, mag)
    pkv.pkv_window_attention(s.lc.desc, s.batch, q, out, 0, 0, s.d ** -0.5)
    assert_attention(out, ref, mag)


def test_workspaces_are_checked():
    s = Setup(4, [1], [500], (16, 8, 128), 16, False)
    q, out = s.q.cuda(), torch.empty((1, 16, 128), dtype=torch.bfloat16, device="cuda")
    n = pkv.pkv_window_ws_bytes(s.lc.desc, s.batch, 0, 0, 64)
    assert n > 0 and pkv.pkv_window_ws_bytes(s.lc.desc, s.batch, 0, 0, 0) == 0
    for ws in (None, torch.zeros(n - 1, dtype=torch.uint8, device="cuda"),
               torch.zeros(n + 16, dtype=torch.uint8, device="cuda")[16:]):
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_window_attention(s.lc.desc, s.batch, q, out, 0, 0, 0.1, 64, ws)
        assert e.value.code == pkv.PKV_ERR_INVALID
    with pytest.raises(ValueError):  # positions of fewer rows
        r = pkv.make_rope(torch.ones(32, dtype=torch.float64, device="cuda"),
                          positions=torch.zeros(0, dtype=torch.int32, device="cuda"))
        kv = torch.zeros((1, 8, 128), dtype=torch.bfloat16, device="cuda")
        pkv.pkv_rope_append(s.lc.desc, s.batch, r, None, kv, kv)


def test_output_in_place_of_the_queries():
    for new, split in (([1, 3], 48), ([1, 3], 0), ([40, 300], 0), ([40, 300], 128)):
        s = Setup(6, new, [400, 300], (8, 2, 128), 16, False)
        ref, mag = attention(s, 100, 4)
        n = pkv.pkv_window_ws_bytes(s.lc.desc, s.batch, 100, 4, split)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None
        q = s.q.cuda()
        pkv.pkv_window_attention(s.lc.desc, s.batch, q, q, 100, 4, s.d ** -0.5, split, ws)
        assert_attention(q, ref, mag)
        assert s.error_bits() == 0


@pytest.mark.parametrize("new", [[1], [70]])
def test_largest_and_smallest_scale(new):
    """sm_scale 0 weighs every visible token alike; with the largest one the best score takes all, and q = 0 does as 0."""
    s = Setup(8, new, [100], (4, 2, 64), 16, False)
    ref, mag = attention(s, 0, 0, 0.0)
    q, out = s.q.cuda(), torch.empty((s.T, 4, 64), dtype=torch.bfloat16, device="cuda")
    pkv.pkv_window_attention(s.lc.desc, s.batch, q, out, 0, 0, 0.0)
    assert_attention(out, ref, mag)
    pkv.pkv_window_attention(s.lc.desc, s.batch, torch.zeros_like(q), out, 0, 0, 3.0e38)
    assert_attention(out, ref, mag)


@pytest.mark.parametrize("handle", [False, True])
def test_a_step_on_another_stream(handle):
    """Uploads, copies and kernels of a step are ordered on the stream that it is given."""
    m = Model((8, 2, 128), 16, [False, True], seqs=2, blocks=40)
    m.cache.add_sequence(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.step([1], [45], 30, 4, stream=side.cuda_stream if handle else side)
    m.cache.fork(1, 2)
    torch.cuda.synchronize()
    m.step([1, 2], [30, 3], 30, 4, stream=side.cuda_stream if handle else side)
    want = read_back(m.cache, 0, [1, 2], torch.float32)
    got = read_back(m.cache, 0, [1, 2], torch.float32, side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_too_long_a_split_is_refused():
    s = Setup(8, [40], [100], (4, 2, 64), 16, False)
    q, out = s.q.cuda(), torch.empty((40, 4, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.full((1, (2 ** 25 + 256) // 16), -1, dtype=torch.int32, device="cuda")
    table[:, :s.width] = s.d_table
    batch = pkv.make_batch(s.d_starts, table, s.d_ctx, num_tokens=40, max_tokens=40)
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_window_attention(s.lc.desc, batch, q, out, 0, 0, 0.125)
    assert e.value.code == pkv.PKV_ERR_UNSUPPORTED
    ws = torch.zeros(pkv.pkv_window_ws_bytes(s.lc.desc, batch, 0, 0, 2 ** 24), dtype=torch.uint8, device="cuda")
    for args in ((0, 0, 0.125, 2 ** 24, ws), (4096, 4, 0.125)):
        pkv.pkv_window_attention(s.lc.desc, batch, q, out, *args)
        ref, mag = attention(s, 0, 0, 0.125)
        assert_attention(out, ref, mag)
    assert s.error_bits() == 0


@pytest.mark.parametrize("pdl", [False, True])
@pytest.mark.parametrize("heads", [(2, 2, 64), (8, 8, 128)])
def test_blocks_of_64_quantize_as_before(pdl, heads):
    """Blocks of 64 tokens, whose rows several CTAs hold: the bits of the block quantizer, with not-a-numbers and
    infinities in each quarter, in one call and token by token."""
    n, hkv, d = 320, heads[1], heads[2]
    rows = torch.randn((n, hkv, d), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    for i, x in ((3, float("nan")), (70, float("inf")), (100, 300.0), (175, -float("inf")), (255, -500.0)):
        rows[i, i % hkv, i % d] = x
    s = Setup(1, [n], [n], heads, 64, True, appended=False)
    dev = rows.cuda()
    back = dev.flip(0).contiguous()
    pkv.pkv_set_programmatic_launch(pdl)
    try:
        pkv.pkv_rope_append(s.lc.desc, s.batch, None, None, dev, back)
        got = [x.clone() for x in (s.lc.k_pool, s.lc.v_pool, s.lc.scales)]
        for x in (s.lc.k_pool, s.lc.v_pool, s.lc.scales):
            x.zero_()
        one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        ctx = torch.arange(1, n + 1, dtype=torch.int32, device="cuda")
        batches = [pkv.make_batch(one, s.d_table, ctx[i:i + 1], s.d_slots, num_tokens=1, max_tokens=1) for i in range(n)]
        for i, b in enumerate(batches):
            pkv.pkv_rope_append(s.lc.desc, b, None, None, dev[i:i + 1], back[i:i + 1])
    finally:
        pkv.pkv_set_programmatic_launch(False)
    ids = torch.as_tensor(s.table[0, :n // 64].copy()).cuda().long()
    for a, b in zip(got, (s.lc.k_pool, s.lc.v_pool, s.lc.scales)):
        assert torch.equal(a[ids].view(torch.int8), b[ids].view(torch.int8))
    pkv.pkv_quantize_blocks_from(s.lc.desc, dev, back, ids.int())
    for a, b in zip(got, (s.lc.k_pool, s.lc.v_pool, s.lc.scales)):
        assert torch.equal(a[ids].view(torch.int8), b[ids].view(torch.int8))
    assert s.error_bits() == 0


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("heads", [(32, 32, 128), (12, 12, 64), (40, 20, 64)])
@pytest.mark.parametrize("seqs", [3, 60])
def test_many_heads(seqs, heads, bs, int8):
    """More kv heads than one CTA's round of rows: written, attended and read back, few sequences and many."""
    rng = np.random.default_rng(seqs)
    ctx = rng.integers(1, 90, size=seqs).tolist()
    new = [int(rng.integers(0, c + 1)) for c in ctx]
    s = Setup(12, new, ctx, heads, bs, int8)
    back = [torch.full((s.T + 1, s.hkv, s.d), 3.0, dtype=torch.float32, device="cuda") for _ in range(2)]
    pkv.pkv_gather_kv(s.lc.desc, s.batch, *back)
    for name, b in zip("kv", back):
        want = np.concatenate([x[c - m:] for x, m, c in zip(s.values[name], new, ctx)])
        assert torch.equal(b[:-1].cpu(), torch.as_tensor(want).float()) and (b[-1] == 3).all()
    ref, mag = attention(s, 20, 3)
    out = torch.zeros((s.T, s.hq, s.d), dtype=torch.bfloat16, device="cuda")
    pkv.pkv_window_attention(s.lc.desc, s.batch, s.q.cuda(), out, 20, 3, s.d ** -0.5)
    assert_attention(out, ref, mag)
    whole = Setup(12, ctx, ctx, heads, bs, int8, appended=False)
    pkv.pkv_rope_append(whole.lc.desc, whole.batch, None, None, whole.new_rows("k").cuda(), whole.new_rows("v").cuda())
    both = [torch.empty((whole.T, s.hkv, s.d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pkv.pkv_gather_kv(whole.lc.desc, whole.batch, *both)
    for name, b in zip("kv", both):
        want = torch.as_tensor(np.concatenate(s.values[name])).float().to(torch.bfloat16)
        assert torch.equal(b.cpu(), want)
    assert s.error_bits() == 0 and whole.error_bits() == 0
