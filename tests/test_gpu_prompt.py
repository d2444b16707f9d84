"""Attention of whole prompts from their rows against fp64, at the sizes and masks
where it can go wrong."""

import numpy as np
import pytest
import torch

from chunk_ref import NAN, assert_attention
from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv
from paged_kv_cache_56_gb300.runtime import LayerCache
from plan_ref import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


class Prompts:
    """Rows of packed prompts: q, k, v as parts of one projection's output, and behind them rows of not-a-numbers."""

    def __init__(self, seed, new, heads, behind=2, q_mult=1.0, v_mult=1.0):
        g = torch.Generator().manual_seed(seed)
        self.new, (self.hq, self.hkv, self.d) = list(new), heads
        self.T, self.behind = sum(new), behind
        x = torch.randn((self.T, self.hq + 2 * self.hkv, self.d), generator=g)
        x[:, :self.hq] *= q_mult
        x[:, -self.hkv:] *= v_mult
        rows = torch.full((self.T + behind, *x.shape[1:]), NAN, dtype=torch.bfloat16)
        rows[:self.T] = x.to(torch.bfloat16)
        self.rows = rows.cuda()
        self.q, self.k, self.v = self.rows[:, :self.hq], self.rows[:, self.hq:-self.hkv], self.rows[:, -self.hkv:]
        self.lc = LayerCache(1, self.hq, self.hkv, self.d, 16, False, 0)
        self.starts, self.ctx = dev(np.cumsum([0] + self.new)), dev(self.new)
        width = max(self.new + [16]) // 16 + 1
        self.batch = pkv.make_batch(self.starts, dev(np.zeros((len(new), width))), self.ctx, num_tokens=self.T + behind,
                                    max_tokens=max(self.new + [0]))

    def run(self, window=0, sinks=0, sm_scale=None, out=None, stream=None):
        out = torch.full((self.T + self.behind, self.hq, self.d), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        pkv.pkv_prompt_attention(self.lc.desc, self.batch, self.q, self.k, self.v, out, window, sinks,
                                 self.d ** -0.5 if sm_scale is None else sm_scale, stream)
        return out

    def reference(self, window=0, sinks=0, sm_scale=None, only=None):
        """(output, sum of weights times |v|), fp64 [T, hq, d]; `only`: of these rows of each sequence."""
        sm_scale = self.d ** -0.5 if sm_scale is None else sm_scale
        outs, mags, at = [], [], 0
        for n in self.new:
            q, k, v = (x[at:at + n].double() for x in (self.q, self.k, self.v))
            at += n
            p = torch.arange(n, device="cuda") if only is None else torch.as_tensor(only(n), device="cuda")
            for i in range(0, len(p), 256):
                r = p[i:i + 256]
                t = torch.arange(n, device="cuda")
                hide = t > r[:, None]
                if window > 0:
                    hide |= (r[:, None] - t >= window) & (t >= sinks)
                x = torch.einsum("mhgd,thd->hgmt", q[r].view(len(r), self.hkv, -1, self.d), k) * sm_scale
                w = torch.softmax(x.masked_fill(hide, -float("inf")), dim=-1)
                for dst, y in ((outs, v), (mags, v.abs())):
                    dst.append(torch.einsum("hgmt,thd->mhgd", w, y).reshape(len(r), self.hq, self.d))
        empty = torch.zeros((0, self.hq, self.d), device="cuda", dtype=torch.float64)
        return torch.cat(outs + [empty]).cpu().numpy(), torch.cat(mags + [empty]).cpu().numpy()

    def check(self, window=0, sinks=0, what="", **kw):
        out = self.run(window, sinks, **kw)
        ref, mag = self.reference(window, sinks, kw.get("sm_scale"))
        assert_attention(out[:self.T], ref, mag, f"window {window} sinks {sinks} {what}")
        assert (out[self.T:] == 7).all(), "rows behind the batch"
        assert self.lc.error_bits() == 0
        return out


HEADS = [(4, 2, 64), (8, 8, 64), (8, 1, 64), (16, 8, 128), (8, 2, 128), (8, 1, 128), (3, 3, 128)]
BATCHES = {
    "one": [1], "singles": [1, 1, 0, 1, 1], "edges": [15, 16, 17, 127, 128, 129], "tiles": [255, 256, 257, 0, 33],
    "long": [1100], "ragged": [3, 700, 0, 64, 385],
}
MASKS = [(0, 0), (1, 0), (1, 1), (16, 4), (130, 0), (100, 137), (300, 5), (5000, 3)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("name", list(BATCHES))
def test_prompt_attention(name, heads):
    p = Prompts(len(name) + heads[0], BATCHES[name], heads)
    for window, sinks in MASKS:
        p.check(window, sinks)


@pytest.mark.parametrize("heads", [(4, 2, 64), (16, 8, 128)])
def test_scores_of_every_size(heads):
    """Softmax from uniform to one-hot, and scales of zero and in between."""
    for e in (-20, -3, 2, 5):
        Prompts(11, [6, 1, 300], heads, q_mult=2.0 ** e).check(what=f"2^{e}")
    for scale in (0.0, 1e-30, 1.0):
        Prompts(12, [6, 1, 300], heads).check(sm_scale=scale, what=f"scale {scale}")


@pytest.mark.parametrize("mult", [1e-15, 1e-6, 1e6, 1e30])
def test_values_of_every_size(mult):
    Prompts(13, [150, 290], (8, 2, 128), v_mult=mult).check(64, 4)


@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 2, 128), (8, 8, 128)])
@pytest.mark.parametrize("what", [NAN, float("inf"), -float("inf")])
def test_other_sequences_values_do_not_matter(what, heads):
    """Not-a-numbers and infinities in every second sequence: the others come out right."""
    new = [100, 3, 129, 200, 65, 1, 300]
    p = Prompts(17, new, heads)
    ref, mag = p.reference(70, 3)
    keep = p.rows.clone()
    at = np.cumsum([0] + new)
    for b in range(1, len(new), 2):
        p.rows[at[b]:at[b + 1]] = what
    out = p.run(70, 3)
    for b in range(0, len(new), 2):
        assert_attention(out[at[b]:at[b + 1]], ref[at[b]:at[b + 1]], mag[at[b]:at[b + 1]], f"sequence {b}")
    p.rows.copy_(keep)
    assert_attention(p.run(70, 3)[:p.T], ref, mag, "afterwards")


def test_masked_not_a_numbers_in_k_do_not_matter():
    """Keys that no row sees: those behind a sequence's end that share a key tile with it."""
    p = Prompts(18, [130, 40], (8, 2, 128))
    ref, mag = p.reference()
    p.k[130:] = NAN
    p.q[130:] = NAN
    assert_attention(p.run()[:130], ref[:130], mag[:130])


def test_sequences_with_earlier_tokens_are_refused():
    new = [20, 300, 5, 64]
    p = Prompts(19, new, (8, 2, 64))
    ref, mag = p.reference()
    p.ctx[1], p.ctx[2] = 301, 4
    out = p.run()
    assert p.lc.error_bits() == pkv.PKV_DEVERR_CTX_LEN
    assert (out[20:325] == 0).all()
    for lo, hi in ((0, 20), (325, 389)):
        assert_attention(out[lo:hi], ref[lo:hi], mag[lo:hi])
    p.lc.err.zero_()
    p.ctx.copy_(dev(new))
    p.starts[2] = 400  # past the rows there are: sequences 1 and 2 hold no rows together
    out = p.run()
    assert p.lc.error_bits() & pkv.PKV_DEVERR_BATCH
    assert_attention(out[:20], ref[:20], mag[:20])
    assert (out[20:325] == 7).all()


@pytest.mark.parametrize("heads", [(8, 2, 64), (32, 32, 128)])
def test_many_sequences(heads):
    """More items than SMs, most sequences short or empty."""
    rng = np.random.default_rng(3)
    new = [int(x) for x in rng.choice([0, 0, 1, 2, 17, 128, 200], size=400)]
    p = Prompts(23, new, heads)
    p.check()
    p.check(20, 2)


def test_a_long_prompt():
    p = Prompts(29, [20011], (8, 1, 64))
    rows = lambda n: np.unique(np.r_[0:3, 127:130, np.arange(0, n, 371), n - 3:n])  # noqa: E731
    for window, sinks in ((0, 0), (4096, 5)):
        out = p.run(window, sinks)
        ref, mag = p.reference(window, sinks, only=rows)
        assert_attention(out[torch.as_tensor(rows(20011)).cuda()], ref, mag)


def test_in_place_and_on_another_stream():
    p = Prompts(31, [77, 400, 1], (16, 8, 128))
    want = p.check(50, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.full_like(want, 7.0)
    torch.cuda.synchronize()
    p.run(50, 2, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    assert torch.equal(p.run(50, 2, out=p.q)[:p.T], want[:p.T])
    assert torch.isnan(p.q[p.T:]).all()


def test_replayed_with_other_lengths():
    """One captured call serves every batch within its bounds."""
    p = Prompts(37, [300, 200, 100], (8, 2, 128))
    out = p.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(out=out)
    for new in ([300, 200, 100], [1, 299, 300], [0, 0, 17], [256, 0, 256], [0, 0, 0]):
        p.new, p.T = new, sum(new)
        p.starts.copy_(dev(np.cumsum([0] + new)))
        p.ctx.copy_(dev(new))
        out.fill_(7.0)
        graph.replay()
        ref, mag = p.reference()
        assert_attention(out[:p.T], ref, mag, str(new))
        assert (out[p.T:] == 7).all()


def test_the_same_call_gives_the_same_bits():
    p = Prompts(41, [2000, 31, 900], (32, 8, 128))
    first = p.run(500, 4)
    for _ in range(3):
        assert torch.equal(p.run(500, 4), first)


def test_two_calls_at_once():
    a, b = Prompts(43, [1500, 700], (16, 8, 128)), Prompts(47, [333] * 5, (8, 1, 64))
    want = [a.check(), b.check(100, 3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.full_like(x, 7.0) for x in want]
    torch.cuda.synchronize()
    for _ in range(5):
        a.run(out=outs[0], stream=streams[0])
        b.run(100, 3, out=outs[1], stream=streams[1])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, want))


def test_programmatic_launches():
    p = Prompts(53, [500, 20], (8, 2, 128))
    want = p.check()
    pkv.pkv_set_programmatic_launch(True)
    try:
        outs = [p.run() for _ in range(6)]
        torch.cuda.synchronize()
    finally:
        pkv.pkv_set_programmatic_launch(False)
    assert all(torch.equal(x, want) for x in outs)


@pytest.mark.parametrize("heads", [(16, 8, 64), (16, 8, 128)])
@pytest.mark.parametrize("item", [0, 1])
def test_the_call_after_a_wait_that_ran_out_is_right(heads, item):
    """The library's test hook leaves the queries of one item uncopied: the call reports it and returns."""
    p = Prompts(59, [6000, 700], heads)  # 424 items: every CTA has two or three
    want = p.run()
    assert pkv.pkv_sync_status([p.lc.desc]) == 0
    pkv.pkv_debug_skip_copy(item)
    try:
        p.run()
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_sync_status([p.lc.desc])
        assert e.value.code == pkv.PKV_ERR_DEVICE_TIMEOUT
    finally:
        pkv.pkv_debug_skip_copy(-1)
    for _ in range(2):
        assert torch.equal(p.run()[:p.T], want[:p.T])
        assert pkv.pkv_sync_status([p.lc.desc]) == 0


def test_contexts_need_no_block_table():
    """Only that there are no earlier tokens matters: a table too short for the rows is not looked at."""
    p = Prompts(61, [2000, 30], (8, 1, 64))
    want = p.check()
    p.batch = pkv.make_batch(p.starts, dev(np.zeros((2, 1))), p.ctx, num_tokens=p.T + p.behind, max_tokens=2000)
    assert torch.equal(p.check(), want)


def test_empty_calls():
    for new in ([], [0, 0]):
        p = Prompts(1, new, (4, 2, 64), behind=0)
        p.run()
        assert p.lc.error_bits() == 0
