"""Positions and their append as a program calls them: captured and replayed with
other lengths on a stream of its own, with programmatic launches, two calls at once."""

import numpy as np
import pytest
import torch

from chunk_ref import Setup
from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv
from plan_ref import dev
from test_gpu_axes import axes_of, positions_of
from test_gpu_chunk import freqs, same

pytestmark = pytest.mark.gpu
HEADS = (16, 8, 128)
SEGS = [[(5, 0, 0, 1), (2, 3, 4, 2), (9, 0, 0, 1)], [], [(1, 6, 7, 1)], [(70, 0, 0, 1), (4, 4, 4, 3)]]


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


class Call:
    """A batch, its positions and its append; the batch's descriptor bounds hold any of LENGTHS."""

    def __init__(self, seed, new, ctx, bs, int8):
        self.s = s = Setup(seed, new, ctx, HEADS, bs, int8, appended=False)
        table = np.zeros((4, 3, 4), np.int32)
        for b, x in enumerate(SEGS):
            if x:
                table[b, :len(x)] = x
        self.segs, self.count, self.ctx = dev(table), dev([len(x) for x in SEGS]), list(ctx)
        self.pos = torch.zeros((3, s.T), dtype=torch.int32, device="cuda")
        self.rope = pkv.make_rope_axes(torch.as_tensor(freqs(64)).cuda(), axes_of(64, "in_turn"), positions=self.pos)
        self.q, self.k, self.v = s.q.cuda(), s.new_rows("k").cuda(), s.new_rows("v").cuda()
        self.q_out, self.k_out = torch.empty_like(self.q), torch.empty_like(self.k)

    def run(self, stream=None):
        pkv.pkv_axis_positions(self.s.batch, self.segs, self.count, self.pos, stream=stream)
        pkv.pkv_rope_append_axes(self.s.lc.desc, self.s.batch, self.rope, self.q, self.k, self.v, self.q_out, self.k_out, stream)

    def result(self):
        names = ("k_pool", "v_pool") + (("k_tail", "v_tail", "scales") if self.s.lc.int8 else ())
        return [self.pos, self.q_out, self.k_out] + [getattr(self.s.lc, n) for n in names]


NEW, CTX = [38, 20, 42, 130], [38, 51, 42, 134]


def positions_wanted(new, ctx):
    return np.concatenate([positions_of(x, c)[:, c - n:] for x, n, c in zip(SEGS, new, ctx)], axis=1)


@pytest.mark.parametrize("pdl", [False, True])
@pytest.mark.parametrize("int8,bs", [(False, 16), (True, 16), (True, 64)])
def test_replayed_with_other_lengths_on_another_stream(int8, bs, pdl):
    call, eager = Call(9, NEW, CTX, bs, int8), Call(9, NEW, CTX, bs, int8)
    pkv.pkv_set_programmatic_launch(pdl)
    try:
        eager.run()
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            call.run()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(call.pos.cpu().numpy(), positions_wanted(NEW, CTX))
        assert all(same(a, b) for a, b in zip(call.result(), eager.result()))
        # fewer tokens behind the same descriptor, one sequence without any
        new, ctx = [38, 0, 42, 17], [38, 51, 42, 134]
        for x in (call, eager):
            x.s.batch.keep[0].copy_(dev(np.cumsum([0] + new)))
            for y in (x.q_out, x.k_out):
                y.fill_(5.0)
            x.pos.fill_(-7)
        eager.run()
        graph.replay()
        torch.cuda.synchronize()
    finally:
        pkv.pkv_set_programmatic_launch(False)
    T = sum(new)
    assert np.array_equal(call.pos[:, :T].cpu().numpy(), positions_wanted(new, ctx))
    assert (call.pos[:, T:] == -7).all() and (call.q_out[T:] == 5).all() and (call.k_out[T:] == 5).all()
    assert all(same(a, b) for a, b in zip(call.result(), eager.result()))
    assert call.s.error_bits() == 0 and eager.s.error_bits() == 0


@pytest.mark.parametrize("int8,bs", [(False, 16), (True, 16), (True, 64)])
def test_two_calls_at_once(int8, bs):
    # one after the other, as often: a chunk that passes a block's end leaves other rows in an
    # INT8 sequence's tail, so that the same append again is another one
    alone = [Call(21 + i, NEW, CTX, bs, int8) for i in range(2)]
    for c in alone:
        for _ in range(8):
            c.run()
            torch.cuda.synchronize()
    calls = [Call(21 + i, NEW, CTX, bs, int8) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(8):
        for c, s in zip(calls, streams):
            c.run(s)
    torch.cuda.synchronize()
    for c, a in zip(calls, alone):
        assert all(same(x, y) for x, y in zip(c.result(), a.result()))
        assert c.s.error_bits() == 0
