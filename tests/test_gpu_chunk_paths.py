"""Windowed attention at the sizes where its kernels change course: batches of
many sequences, long key lists, whole items beside split ones, and bad device
values on every kernel."""

import numpy as np
import pytest
import torch

from chunk_ref import Setup, assert_attention, attention
from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def dev(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


def run(s, batch, window=0, sinks=0, split=None, T=None, desc=None):
    desc = s.lc.desc if desc is None else desc
    split = pkv.pkv_window_split_tokens(desc, batch, window, sinks) if split is None else split
    n = pkv.pkv_window_ws_bytes(desc, batch, window, sinks, split)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None
    T = s.T if T is None else T
    q = torch.zeros((T, s.hq, s.d), dtype=torch.bfloat16, device="cuda")
    q[:s.T] = s.q.cuda()
    out = torch.full_like(q, 7.0)
    pkv.pkv_window_attention(desc, batch, q, out, window, sinks, s.d ** -0.5, split, ws)
    torch.cuda.synchronize()
    return out


def spread(s, B, at, extra=0):
    """The batch of s as sequences at[0] < at[1] < ... of B, the others without tokens."""
    counts, ctx, slots = np.zeros(B, np.int32), np.zeros(B, np.int32), np.zeros(B, np.int32)
    table = np.full((B, s.width), -1, np.int32)
    counts[at], ctx[at], slots[at], table[at] = s.new, s.ctx, s.slots, s.table
    starts = np.concatenate([[0], np.cumsum(counts)])
    return pkv.make_batch(dev(starts), dev(table), dev(ctx), dev(slots) if s.int8 else None,
                          num_tokens=s.T + extra, max_tokens=max(s.new))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("B", [33, 3000, 65535])
def test_few_sequences_of_a_large_batch_have_tokens(B, int8):
    s = Setup(13, [40, 300, 17], [60, 310, 200], (16, 8, 64), 16, int8)
    batch = spread(s, B, [0, B // 2, B - 1])
    for window, sinks in ((0, 0), (50, 4)):
        ref, mag = attention(s, window, sinks)
        for split in (None, 0, 128):
            assert_attention(run(s, batch, window, sinks, split), ref, mag, f"{window} {split}")
    assert s.error_bits() == 0


@pytest.mark.parametrize("int8", [False, True])
def test_many_sequences_with_tokens(int8):
    rng = np.random.default_rng(4)
    new = rng.choice([0, 1, 2, 9, 17, 30], size=700).tolist()
    ctx = [n + int(rng.integers(0, 50)) for n in new]
    s = Setup(14, new, ctx, (8, 2, 64), 16, int8)
    ref, mag = attention(s, 20, 3)
    for extra in (0, 5000):  # num_tokens as the batch has them, and as buffers may hold
        s.batch.num_tokens = s.T + extra
        out = run(s, s.batch, 20, 3, T=s.T + extra)
        assert_attention(out[:s.T], ref, mag)
        assert (out[s.T:] == 7).all()
    assert s.error_bits() == 0


def test_too_many_pieces_of_work_are_refused():
    s = Setup(15, [17], [17], (4096, 4096, 64), 16, False)
    batch = spread(s, 65535, [7])
    with pytest.raises(pkv.PkvError) as e:
        run(s, batch, split=0)
    assert e.value.code == pkv.PKV_ERR_UNSUPPORTED
    batch = spread(s, 32768, [7])  # 2^27
    ref, mag = attention(s, 0, 0)
    assert_attention(run(s, batch, split=0), ref, mag)
    assert s.error_bits() == 0


# ---------------------------------------------------------------------------
# Long contexts: a part of the rows against the definition, fp64 on the GPU
# ---------------------------------------------------------------------------

def some_rows(s, window, sinks, values=None, per_seq=24, skip=None):
    """(rows, output, magnitude) of the definition for some rows of each sequence, its first and last among them; the
    magnitude as in chunk_ref.attention. skip[b]: tokens that count as not visible."""
    rows, outs, mags = [], [], []
    for b in range(s.B):
        if s.new[b] == 0:
            continue
        k, v = (torch.as_tensor((values or s.values)[n][b]).cuda() for n in "kv")
        i = np.unique(np.linspace(0, s.new[b] - 1, per_seq).astype(int))
        pos = torch.as_tensor(s.ctx[b] - s.new[b] + i).cuda()[:, None]
        t = torch.arange(s.ctx[b], device="cuda")[None]
        see = t <= pos
        if window > 0:
            see &= (pos - t < window) | (t < sinks)
        if skip and b in skip:
            see[:, skip[b]] = False
        q = s.q[s.starts[b] + i].cuda().double().reshape(len(i), s.hkv, s.G, s.d)
        x = torch.einsum("rhgd,thd->rhgt", q, k) * s.d ** -0.5
        x = x.masked_fill(~see[:, None, None], -float("inf"))
        w = torch.softmax(x, -1).nan_to_num(0.0)
        o = torch.einsum("rhgt,thd->rhgd", w, v)
        m = torch.einsum("rhgt,thd->rhgd", w, v.abs())
        if s.int8:
            top = v.abs().amax(dim=(0, 2)).nan_to_num(0.0)
            m = m + top[None, :, None, None] * (see.sum(1) * 2.0 ** -30)[:, None, None, None]
        rows.append(s.starts[b] + i)
        outs.append(o.reshape(len(i), s.hq, s.d).cpu().numpy())
        mags.append(m.reshape(len(i), s.hq, s.d).cpu().numpy())
    return np.concatenate(rows), np.concatenate(outs), np.concatenate(mags)


def check(s, out, window, sinks, what="", **kw):
    rows, ref, mag = some_rows(s, window, sinks, **kw)
    assert torch.isfinite(out[:s.T]).all()
    assert_attention(out[rows], ref, mag, what)


@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("int8", [False, True])
def test_whole_items_beside_split_ones(int8, bs):
    """22 row tiles of 8 kv heads: 152 SMs take a whole item each, the 24 that are left are split. Long lists of keys
    (up to 40 tiles of 128 tokens), the same bits every time."""
    s = Setup(16, [900, 700, 640, 300], [3000, 2100, 5000, 2500], (16, 8, 64), bs, int8)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if sms == 152:  # both kinds, so the workspace is that of the 24 (and of what raggedness may add)
        n = pkv.pkv_window_ws_bytes(s.lc.desc, s.batch, 0, 0, 256)
        assert 0 < n < 16384 * 4 + 176 * 256 * 20 * (64 * 4 + 8)
    for window, sinks in ((0, 0), (1500, 70)):
        first = None
        for split in (None, 256, 640, 0):
            out = run(s, s.batch, window, sinks, split)
            check(s, out, window, sinks, f"{window} {split}")
            if split == 256:
                first = out
        for _ in range(3):
            assert torch.equal(run(s, s.batch, window, sinks, 256), first)
    assert s.error_bits() == 0


@pytest.mark.parametrize("heads", [(8, 1, 128), (8, 2, 64)])
@pytest.mark.parametrize("int8", [False, True])
def test_more_than_32_parts_are_merged(int8, heads):
    s = Setup(17, [20, 37], [6000, 4500], heads, 16, int8)
    for window, sinks in ((0, 0), (4200, 130)):
        out = run(s, s.batch, window, sinks, 128)
        check(s, out, window, sinks)
        assert torch.equal(run(s, s.batch, window, sinks, 128), out)
    assert s.error_bits() == 0


def scale_values(s, factor):
    """Multiplies the V scales of block i of every sequence by factor(i); the values are those of the rounded scales."""
    for b in range(s.B):
        for i in range(s.ctx[b] // s.bs):
            s.lc.scales[int(s.table[b, i]), :, 1] *= factor(i)
    sc, codes = s.lc.scales.cpu().double().numpy(), s.lc.v_pool.cpu().double().numpy()
    for b in range(s.B):
        for i in range(s.ctx[b] // s.bs):
            blk = int(s.table[b, i])
            s.values["v"][b][i * s.bs:(i + 1) * s.bs] = (codes[blk] * sc[blk, :, 1, None, None]).transpose(1, 0, 2)


@pytest.mark.parametrize("int8,trend", [(False, "level"), (True, "level"), (True, "growing"), (True, "falling")])
@pytest.mark.parametrize("heads,new", [((4, 2, 64), [1, 3]), ((8, 2, 128), [1, 4]), ((8, 1, 128), [2, 1])])
def test_one_cta_over_thousands_of_tokens(heads, new, int8, trend):
    """Up to 16 rows, no split: more than 256 tiles of 16 tokens a CTA, whose ids and scales come in several pieces; over
    INT8 the accumulators' units follow the largest V scale from piece to piece."""
    s = Setup(18, new, [9001, 4097], heads, 16, int8)
    if trend != "level":
        scale_values(s, lambda i: 2.0 ** (i // 128 * 3 * (1 if trend == "growing" else -1)))
    for window, sinks in ((0, 0), (6000, 40)):
        for split in (0, 4800):
            check(s, run(s, s.batch, window, sinks, split), window, sinks, f"{window} {split}")
    assert s.error_bits() == 0


@pytest.mark.parametrize("split", [0, 256])
@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("int8", [False, True])
def test_bad_device_values_with_many_rows(int8, bs, split):
    """What the few-row kernel is tested with, on the tensor-core kernel: left out, zero or not visible, and reported."""
    s = Setup(19, [60, 300, 17, 40], [1700, 700, 330, 400], (4, 2, 64), bs, int8)
    rows, ref, mag = some_rows(s, 0, 0)
    seq = np.searchsorted(s.starts, rows, side="right") - 1

    def others(out, b, what):
        keep = seq != b
        assert_attention(out[rows[keep]], ref[keep], mag[keep], what)

    # more new tokens than the context holds, and a context behind the table's end: zero rows
    for bad in (200, -3, s.width * bs + 1):
        s.d_ctx[1] = bad
        out = run(s, s.batch, split=split)
        assert s.error_bits() == pkv.PKV_DEVERR_CTX_LEN
        assert (out[60:360] == 0).all()
        others(out, 1, "context")
        s.lc.err.zero_()
    s.d_ctx[1] = 700
    # block ids out of range, early and behind the eighth tile of 128 tokens: their tokens are not visible
    gone = [1, 1300 // bs]
    old = [int(s.d_table[0, i]) for i in gone]
    s.d_table[0, gone[0]], s.d_table[0, gone[1]] = s.num_blocks, -7
    out = run(s, s.batch, split=split)
    assert s.error_bits() == pkv.PKV_DEVERR_BLOCK_ID
    others(out, 0, "block")
    tokens = np.concatenate([np.arange(i * bs, (i + 1) * bs) for i in gone])
    check(s, out, 0, 0, "block", skip={0: tokens})
    s.d_table[0, gone[0]], s.d_table[0, gone[1]] = old
    s.lc.err.zero_()
    # token_starts behind num_tokens: left out
    s.d_starts[4] = s.T + 1
    out = run(s, s.batch, split=split)
    assert s.error_bits() == pkv.PKV_DEVERR_BATCH and (out[s.starts[3]:] == 7).all()
    others(out, 3, "starts")
    s.d_starts[4] = s.T
    s.lc.err.zero_()
    if int8:
        # a bad slot: the tail's tokens are not visible
        for bad in (99, -1):
            s.d_slots[2] = bad
            out = run(s, s.batch, split=split)
            assert s.error_bits() == pkv.PKV_DEVERR_SLOT
            check(s, out, 0, 0, "slot", skip={2: np.arange(330 // bs * bs, 330)})
            s.lc.err.zero_()
        s.d_slots[2] = int(s.slots[2])
    assert_attention(run(s, s.batch, split=split)[rows], ref, mag)
    assert s.error_bits() == 0


@pytest.mark.parametrize("e", [-60, 0, 100])
@pytest.mark.parametrize("new", [[1, 3], [60, 130]])
def test_bf16_values_of_every_size(new, e):
    """V of 2^-60 and more keeps its precision with every number of rows."""
    s = Setup(20, new, [150, 700], (8, 2, 128), 16, False)
    s.lc.v_pool *= 2.0 ** e
    for b in range(s.B):
        s.values["v"][b] *= 2.0 ** e
    for window, sinks in ((0, 0), (64, 4)):
        check(s, run(s, s.batch, window, sinks), window, sinks)


def test_two_calls_at_once():
    """Calls of both kernels on two streams at the same time, each with a workspace of its own, replayed from graphs."""
    sets = [Setup(21, [200, 33], [900, 700], (8, 2, 64), 16, False), Setup(22, [1, 2, 1], [2000, 900, 1500], (8, 2, 128), 16, True),
            Setup(23, [400], [1400], (8, 1, 128), 64, True)]
    calls = []
    for s in sets:
        n = pkv.pkv_window_ws_bytes(s.lc.desc, s.batch, 0, 0, 256)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        q, out = s.q.cuda(), torch.empty((s.T, s.hq, s.d), dtype=torch.bfloat16, device="cuda")
        call = (s.lc.desc, s.batch, q, out, 0, 0, s.d ** -0.5, 256, ws)
        pkv.pkv_window_attention(*call)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(5):
                pkv.pkv_window_attention(*call)
        calls.append((g, torch.cuda.Stream(), out, out.clone(), call))  # (a graph does not keep its tensors alive)
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for g, stream, *_ in calls:
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    for s, (_, _, out, want, _) in zip(sets, calls):
        assert torch.equal(out, want)
        check(s, out, 0, 0)
        assert s.error_bits() == 0


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("new", [[1, 3], [40, 300]])
def test_rows_that_see_nothing_are_zero(new, int8):
    """A sequence none of whose blocks is there (nor its slot), beside one that is whole; with splits, and with a window."""
    s = Setup(24, new, [500, 900], (8, 2, 64), 16, int8)
    s.d_table[0, :] = -1
    if int8:
        s.d_slots[0] = -1
    for window, sinks in ((0, 0), (100, 20)):
        rows, ref, mag = some_rows(s, window, sinks)
        mine = rows >= s.starts[1]
        for split in (0, 128):
            out = run(s, s.batch, window, sinks, split)
            assert (out[:s.starts[1]] == 0).all()
            assert_attention(out[rows[mine]], ref[mine], mag[mine])
    assert s.error_bits() == pkv.PKV_DEVERR_BLOCK_ID | (pkv.PKV_DEVERR_SLOT if int8 else 0)
