"""The chunk operators (rotary append, windowed attention, read-back) against
fp64 references, at the sizes and masks where they can go wrong."""

import numpy as np
import pytest
import torch

from chunk_ref import NAN, Setup, assert_attention, attention, bf16, quantize_heads, turned
from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def run_window(s, window, sinks, split="auto", sm_scale=None, ws=None, q=None, out=None):
    desc = s.lc.desc
    split = pkv.pkv_window_split_tokens(desc, s.batch, window, sinks) if split == "auto" else split
    n = pkv.pkv_window_ws_bytes(desc, s.batch, window, sinks, split)
    if n and ws is None:
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    out = torch.full((s.T, s.hq, s.d), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    pkv.pkv_window_attention(desc, s.batch, s.q.cuda() if q is None else q, out, window, sinks,
                             s.d ** -0.5 if sm_scale is None else sm_scale, split, ws)
    torch.cuda.synchronize()
    return out


HEADS = [(4, 2, 64), (8, 8, 64), (8, 1, 64), (16, 8, 128), (8, 2, 128), (8, 1, 128), (3, 3, 128)]
# new tokens and contexts of a batch
BATCHES = {
    "step": ([1, 1, 1, 1], [1, 17, 33, 100]),
    "step_edges": ([1, 1, 1, 1, 1], [15, 16, 64, 65, 128]),
    "draft": ([3, 1, 5, 2], [3, 40, 200, 129]),
    "chunk": ([20, 1, 64, 0, 33], [20, 300, 64, 10, 150]),
    "prompt": ([130, 257], [130, 257]),
    "long_row": ([9], [1000]),
}
MASKS = [(0, 0), (1, 0), (1, 1), (16, 4), (33, 16), (100, 37), (5000, 3)]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("name", list(BATCHES))
def test_window_attention(name, heads, bs, int8):
    new, ctx = BATCHES[name]
    s = Setup(len(name) + heads[0], new, ctx, heads, bs, int8)
    for window, sinks in MASKS:
        ref, mag = attention(s, window, sinks)
        for split in ("auto", 0, 16, 48):
            out = run_window(s, window, sinks, split)
            assert_attention(out, ref, mag, f"window {window} sinks {sinks} split {split}")
    assert s.error_bits() == 0


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("new", [[1, 1], [4, 2], [70, 300]])
def test_hidden_blocks_are_not_looked_up(new, int8):
    """Blocks between the sinks and the first row's window: -1 in the table, NaN in memory."""
    ctx, window, sinks, bs = [700, 900], 50, 20, 16
    first = [(max(0, c - n - window + 1) // bs) for n, c in zip(new, ctx)]
    s = Setup(5, new, ctx, (8, 2, 128), bs, int8, hidden=lambda b, i: -(-sinks // bs) <= i < first[b])
    ref, mag = attention(s, window, sinks)
    for split in ("auto", 0, 32):
        assert_attention(run_window(s, window, sinks, split), ref, mag)
    assert s.error_bits() == 0


@pytest.mark.parametrize("heads", [(4, 2, 64), (16, 8, 128)])
@pytest.mark.parametrize("int8", [False, True])
def test_scores_of_every_size(heads, int8):
    """Softmax from uniform to one-hot: the query scaled over 2^-20 .. 2^5."""
    s = Setup(11, [6, 1, 40], [100, 64, 40], heads, 16, int8)
    for e in (-20, -3, 0, 2, 5):
        keep = s.q
        s.q = bf16(s.q.float() * 2.0 ** e)
        ref, mag = attention(s, 0, 0)
        assert_attention(run_window(s, 0, 0), ref, mag, f"2^{e}")
        s.q = keep


@pytest.mark.parametrize("mult", [1e-6, 1e-3, 1e4, 1e12])
@pytest.mark.parametrize("new", [[1, 2], [60, 130]])
def test_int8_value_ranges(mult, new):
    """V of any size (K left alone: the scores stay moderate), some blocks far larger than others."""
    s = Setup(3, new, [150, 300], (8, 2, 128), 16, True)
    for b in range(s.B):
        for i in range(s.ctx[b] // 16):
            f = mult * (1000.0 if i % 3 == 0 else 1.0)
            s.lc.scales[int(s.table[b, i]), :, 1] *= f
            s.values["v"][b][i * 16:(i + 1) * 16] *= np.float32(1.0) * f
    # the scales are rounded to fp32 once more: read the cache's own
    sc = s.lc.scales.cpu().double().numpy()
    codes = s.lc.v_pool.cpu().double().numpy()
    for b in range(s.B):
        for i in range(s.ctx[b] // 16):
            blk = int(s.table[b, i])
            s.values["v"][b][i * 16:(i + 1) * 16] = (codes[blk] * sc[blk, :, 1, None, None]).transpose(1, 0, 2)
    ref, mag = attention(s, 64, 4)
    assert_attention(run_window(s, 64, 4), ref, mag)


def test_strided_rows_and_rows_behind():
    """q as a part of one projection's output, out as a part of a wider buffer; rows behind the last sequence stay."""
    s = Setup(21, [3, 50], [90, 64], (16, 8, 128), 16, False)
    wide = torch.full((s.T + 2, 32, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    wide[:s.T, :16] = s.q.cuda()
    out = torch.full((s.T + 2, 20, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    ref, mag = attention(s, 40, 4)
    s.batch.num_tokens = s.T + 2
    run_window(s, 40, 4, q=wide[:, :16], out=out[:, :16])
    assert_attention(out[:s.T, :16], ref, mag)
    assert (out[:, 16:] == 5).all() and (out[s.T:] == 5).all()


def test_workspace_is_shared_by_calls_of_other_shapes():
    """One zeroed workspace serves calls of different batches, replayed from graphs in turn."""
    a = Setup(31, [1] * 3, [700, 900, 64], (16, 8, 128), 16, False)
    b = Setup(32, [5, 2], [2000, 333], (8, 2, 128), 16, True)
    need = max(pkv.pkv_window_ws_bytes(x.lc.desc, x.batch, 0, 0, 32) for x in (a, b))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    outs, graphs, refs = [], [], []
    for x in (a, b):
        q, out = x.q.cuda(), torch.empty((x.T, x.hq, x.d), dtype=torch.bfloat16, device="cuda")
        run_window(x, 0, 0, 32, ws=ws, q=q, out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.pkv_window_attention(x.lc.desc, x.batch, q, out, 0, 0, x.d ** -0.5, 32, ws)
        outs.append(out)
        graphs.append((g, q))
        refs.append(attention(x, 0, 0))
    first = None
    for turn in range(3):
        for out, (g, _) in zip(outs, graphs):
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        for out, (ref, mag) in zip(outs, refs):
            assert_attention(out, ref, mag, f"replay {turn}")
        now = [o.clone() for o in outs]
        assert first is None or all(torch.equal(x, y) for x, y in zip(first, now))  # the same bits
        first = now


@pytest.mark.parametrize("int8", [False, True])
def test_bad_device_values_are_reported(int8):
    s = Setup(41, [2, 3, 1, 4], [50, 70, 33, 20], (4, 2, 64), 16, int8)
    ref, mag = attention(s, 0, 0)
    # sequence 1: more tokens new than its context holds -> zero rows
    s.d_ctx[1] = 2
    out = run_window(s, 0, 0)
    assert s.error_bits() == pkv.PKV_DEVERR_CTX_LEN
    assert (out[2:5] == 0).all()
    keep = np.r_[0:2, 5:10]
    assert_attention(out[keep], ref[keep], mag[keep])
    s.lc.err.zero_()
    s.d_ctx[1] = 70
    # a block id out of range: its tokens are not visible
    old = int(s.d_table[0, 1])
    s.d_table[0, 1] = s.num_blocks
    out = run_window(s, 0, 0)
    assert s.error_bits() == pkv.PKV_DEVERR_BLOCK_ID
    sub = {n: [v.copy() for v in s.values[n]] for n in "kv"}
    keep_tok = np.r_[0:16, 32:50]
    q = s.q.double().numpy()
    for i in range(2):
        t = keep_tok[keep_tok <= 48 + i]
        x = np.einsum("hgd,thd->hgt", q[i].reshape(2, 2, 64), sub["k"][0][t]) / 8
        w = np.exp(x - x.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        r = np.einsum("hgt,thd->hgd", w, sub["v"][0][t]).reshape(4, 64)
        m = np.einsum("hgt,thd->hgd", w, np.abs(sub["v"][0][t])).reshape(4, 64)
        assert_attention(out[i], r, m)
    s.d_table[0, 1] = old
    s.lc.err.zero_()
    # token_starts that give a sequence more rows than max_tokens, or pass num_tokens: left out
    s.d_starts[4] = 12
    out = run_window(s, 0, 0)
    assert s.error_bits() == pkv.PKV_DEVERR_BATCH and (out[6:] == 7).all()
    assert_attention(out[:6], ref[:6], mag[:6])
    s.d_starts[4] = 10
    s.lc.err.zero_()
    if int8:
        s.d_slots[2] = 99
        out = run_window(s, 0, 0)
        assert s.error_bits() == pkv.PKV_DEVERR_SLOT
        assert torch.isfinite(out).all()


# ---------------------------------------------------------------------------
# Rotary append
# ---------------------------------------------------------------------------

def freqs(n, base=10000.0):
    return base ** (-np.arange(n) / max(n, 1))


def expected_cache(s, k_rows, v_rows):
    """Pool, scales and tail after appending rows (bf16 [T, hkv, d]) by the framework's definition: the oracle's
    quantizer on the bf16 rows of every block that is full, the last partial block's new rows in the tail."""
    pools = {n: getattr(s.lc, n + "_pool").cpu().clone() for n in "kv"}
    tails = {n: getattr(s.lc, n + "_tail").cpu().clone() for n in "kv"} if s.int8 else None
    scales = s.lc.scales.cpu().clone() if s.int8 else None
    for kv, (n, rows) in enumerate(zip("kv", (k_rows, v_rows))):
        for b in range(s.B):
            c, m = s.ctx[b], s.new[b]
            if m == 0:
                continue
            seq = torch.cat([s.rows[n][b][:c - m], rows[s.starts[b]:s.starts[b] + m]])
            for i in range((c - m) // s.bs, (c - 1) // s.bs + 1):
                lo, hi = i * s.bs, min(c, (i + 1) * s.bs)
                fresh = max(lo, c - m)
                if not s.int8:
                    pools[n][s.table[b, i], :, fresh - lo:hi - lo] = seq[fresh:hi].transpose(0, 1)
                elif hi - lo == s.bs:
                    code, sc = quantize_heads(seq[lo:hi].transpose(0, 1))
                    pools[n][s.table[b, i]] = torch.as_tensor(code)
                    scales[s.table[b, i], :, kv] = torch.as_tensor(sc)
                else:
                    tails[n][s.slots[b], :, fresh - lo:hi - lo] = seq[fresh:hi].transpose(0, 1)
    return pools, scales, tails


def same(a, b):
    a, b = a.cpu().contiguous(), b.cpu().contiguous()
    if a.dtype == torch.int8:
        return torch.equal(a, b)
    kind = torch.int32 if a.dtype == torch.float32 else torch.int16
    return torch.equal(a.view(kind), b.view(kind))


APPENDS = {
    "step": ([1, 1, 1, 1, 1], [1, 16, 17, 64, 100]),
    "begun_block": ([30, 40, 7, 16], [45, 47, 15, 32]),
    "prompts": ([100, 16, 64, 1, 130], [100, 16, 64, 1, 130]),
    "none_and_many": ([0, 129, 3, 0], [5, 200, 131, 64]),
}


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 8, 64), (16, 8, 128), (8, 1, 128)])
@pytest.mark.parametrize("name", list(APPENDS))
def test_rope_append(name, heads, bs, int8):
    new, ctx = APPENDS[name]
    d = heads[2]
    for rotary, inter, scale, far in ((d, False, 1.0, 0), (d // 2, True, 1.25, 0), (d // 4, False, 1.0, 10 ** 6),
                                      (d, True, 1.0, 2 ** 30), (48, False, 1.0, 0), (0, False, 1.0, 0)):
        s = Setup(61, new, ctx, heads, bs, int8, appended=False)
        f = freqs(rotary // 2)
        pos = np.concatenate([np.arange(c - n, c) for n, c in zip(new, ctx)]) + far
        rope = None
        if rotary:
            rope = pkv.make_rope(torch.as_tensor(f).cuda(), interleaved=inter, scale=scale,
                                 positions=torch.as_tensor(pos.astype(np.int32)).cuda() if far else None)
        k, v = s.new_rows("k"), s.new_rows("v")
        qkv = torch.cat([s.q, k, v], dim=1).cuda()
        q_out = torch.empty((s.T, s.hq, d), dtype=torch.bfloat16, device="cuda")
        k_turned = turned(k, pos, f, inter, scale)
        # an append into a bf16 cache gives the turned rows themselves
        t = s if not int8 else Setup(61, new, ctx, heads, bs, False, appended=False)
        pkv.pkv_rope_append(t.lc.desc, t.batch, rope, qkv[:, :s.hq], qkv[:, s.hq:-s.hkv], qkv[:, -s.hkv:], q_out)
        got_k = torch.cat([t.lc.k_pool[t.table[b, p // bs], :, p % bs] for b in range(t.B)
                           for p in [np.arange(ctx[b] - new[b], ctx[b])]]).cpu()
        # half a bf16 step of the result; products and angles in fp32: 2^-22 of the pair's size
        for got, src, ref in ((q_out.cpu(), s.q, turned(s.q, pos, f, inter, scale)), (got_k, k, k_turned)):
            big = src.double().abs().amax(dim=2, keepdim=True).numpy() * scale
            err = np.abs(got.double().numpy() - ref) - (2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * big)
            assert (err <= 0).all(), (rotary, inter, far, err.max())
            if rotary < d:
                assert torch.equal(got[:, :, rotary:], src[:, :, rotary:])
        pools, scales, tails = expected_cache(s, got_k, v)
        if int8:
            pkv.pkv_rope_append(s.lc.desc, s.batch, rope, qkv[:, :s.hq], qkv[:, s.hq:-s.hkv], qkv[:, -s.hkv:], q_out)
            assert same(s.lc.scales, scales)
            assert all(same(getattr(s.lc, n + "_tail"), tails[n]) for n in "kv")
        assert all(same(getattr(s.lc, n + "_pool"), pools[n]) for n in "kv")
        assert s.error_bits() == 0
        # in place, and keys alone
        q2 = s.q.cuda()
        pkv.pkv_rope_append(s.lc.desc, s.batch, rope, q2, qkv[:, s.hq:-s.hkv], qkv[:, -s.hkv:])
        assert torch.equal(q2, q_out)
        if "begun" not in name and name != "none_and_many":
            pkv.pkv_rope_append(s.lc.desc, s.batch, rope, None, qkv[:, s.hq:-s.hkv], qkv[:, -s.hkv:])
            assert all(same(getattr(s.lc, n + "_pool"), pools[n]) for n in "kv")


def test_rope_append_bad_values():
    s = Setup(71, [20, 3, 5], [40, 30, 70], (4, 2, 64), 16, True, appended=False)
    before = [x.clone() for x in (s.lc.k_pool, s.lc.v_pool, s.lc.k_tail)]
    s.d_ctx[0] = 10000
    s.d_slots[1] = -1
    s.d_table[2, 4] = -5  # not filled by these tokens: its id is not looked at
    k, v = s.new_rows("k").cuda(), s.new_rows("v").cuda()
    pkv.pkv_rope_append(s.lc.desc, s.batch, None, None, k, v)
    assert s.error_bits() == pkv.PKV_DEVERR_CTX_LEN | pkv.PKV_DEVERR_SLOT
    assert torch.equal(s.lc.k_pool, before[0]) and torch.equal(s.lc.v_pool, before[1])
    assert same(s.lc.k_tail[s.slots[0]], before[2][s.slots[0]]) and same(s.lc.k_tail[s.slots[1]], before[2][s.slots[1]])
    assert same(s.lc.k_tail[s.slots[2], :, 1:6], k[23:].transpose(0, 1))


# ---------------------------------------------------------------------------
# Read-back
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("heads", [(4, 2, 64), (16, 8, 128), (3, 3, 128)])
def test_gather(heads, bs, int8, dtype):
    ctx = [1, 100, 64, 131, 0, 17]
    for new, first in ((ctx, None), ([1, 37, 64, 5, 0, 3], None), ([1, 50, 3, 16, 0, 17], [0, 13, 1, 100, 0, 0])):
        s = Setup(81, new, ctx, heads, bs, int8)
        outs = [torch.full((s.T + 1, s.hkv, s.d), 3.0, dtype=dtype, device="cuda") for _ in range(2)]
        f = None if first is None else torch.tensor(first, dtype=torch.int32, device="cuda")
        pkv.pkv_gather_kv(s.lc.desc, s.batch, outs[0], outs[1], f)
        assert s.error_bits() == 0
        for n, out in zip("kv", outs):
            parts = []
            for b in range(s.B):
                lo = ctx[b] - new[b] if first is None else first[b]
                parts.append(s.values[n][b][lo:lo + new[b]])
            # code * scale is rounded once to fp32, then (bf16) once more: the same bits
            ref = torch.as_tensor(np.concatenate(parts)).float().to(dtype)
            assert torch.equal(out[:-1].cpu(), ref)
            assert (out[-1] == 3).all()


def test_gather_bad_values():
    s = Setup(91, [10, 20, 5, 30], [40, 30, 70, 30], (4, 2, 64), 16, True)
    outs = [torch.full((s.T, s.hkv, s.d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    s.d_slots[1] = 50
    s.d_table[2, 4] = s.num_blocks   # tokens 64..: in the tail, not looked up
    s.d_table[3, 1] = -1
    first = torch.tensor([35, 10, 65, 0], dtype=torch.int32, device="cuda")
    pkv.pkv_gather_kv(s.lc.desc, s.batch, outs[0], outs[1], first)
    assert s.error_bits() == pkv.PKV_DEVERR_CTX_LEN | pkv.PKV_DEVERR_SLOT
    assert (outs[0][:10] == 3).all()                       # 35 .. 44 of 40
    assert (outs[0][10 + 6:30] == 3).all()                 # tokens 16 .. 29 of a bad slot's tail
    ref = torch.as_tensor(s.values["k"][1][10:16]).float().to(torch.bfloat16)
    assert torch.equal(outs[0][10:16].cpu(), ref)
    assert torch.equal(outs[0][30:35].cpu(), torch.as_tensor(s.values["k"][2][65:70]).to(torch.bfloat16))


def test_long_offsets():
    """Blocks behind 2^31 bytes and 2^31 elements of a pool: written, attended and read back."""
    hq, hkv, d, bs, blocks = 2, 1, 128, 64, 280000  # 64 * 128 * 280000 = 2.29e9 elements
    from paged_kv_cache_56_gb300.runtime import LayerCache
    lc = LayerCache(blocks, hq, hkv, d, bs, False, 0)
    ids = [blocks - 1, 3, blocks - 2]
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = pkv.make_batch(dev([0, 150]), dev([ids]), dev([150]), num_tokens=150, max_tokens=150)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((150, hkv, d), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn((150, hq, d), generator=g).to(torch.bfloat16).cuda()
    pkv.pkv_rope_append(lc.desc, batch, None, None, k, v)
    back = [torch.empty_like(k) for _ in range(2)]
    pkv.pkv_gather_kv(lc.desc, batch, *back)
    assert torch.equal(back[0], k) and torch.equal(back[1], v)
    out = torch.empty_like(q)
    pkv.pkv_window_attention(lc.desc, batch, q, out, 0, 0, d ** -0.5)
    x = torch.einsum("ihd,jd->hij", q.double(), k[:, 0].double()) / d ** 0.5
    x = x.masked_fill(torch.triu(torch.ones(150, 150, device="cuda", dtype=torch.bool), 1), -float("inf"))
    w = torch.softmax(x, -1)
    ref = torch.einsum("hij,jd->ihd", w, v[:, 0].double()).cpu().numpy()
    mag = torch.einsum("hij,jd->ihd", w, v[:, 0].double().abs()).cpu().numpy()
    assert_attention(out, ref, mag)
    assert lc.error_bits() == 0


def test_empty_calls():
    s = Setup(1, [0, 0], [5, 20], (4, 2, 64), 16, False)
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    kv = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    pkv.pkv_window_attention(s.lc.desc, s.batch, e, e, 0, 0, 0.1)
    pkv.pkv_rope_append(s.lc.desc, s.batch, None, None, kv, kv)
    pkv.pkv_gather_kv(s.lc.desc, s.batch, kv, kv)
    assert NAN != NAN and s.error_bits() == 0


@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("new", [[1, 2], [60, 130]])
def test_blocks_whose_scale_is_zero(heads, new):
    """An INT8 block with scales of zero (one that another program wrote) stands for zeros, whatever its codes."""
    s = Setup(7, new, [100, 200], heads, 16, True)
    for b, i in ((0, 0), (0, 5), (1, 3), (1, 11)):
        s.lc.scales[int(s.table[b, i])] = 0.0
        for n in "kv":
            s.values[n][b][i * 16:(i + 1) * 16] = 0.0
    back = [torch.full((s.T, s.hkv, s.d), 3.0, dtype=torch.float32, device="cuda") for _ in range(2)]
    pkv.pkv_gather_kv(s.lc.desc, s.batch, *back)
    for n, got in zip("kv", back):
        want = np.concatenate([x[c - m:] for x, m, c in zip(s.values[n], s.new, s.ctx)])
        assert torch.equal(got.cpu(), torch.as_tensor(want).float())
    for window, sinks in ((0, 0), (40, 4)):
        ref, mag = attention(s, window, sinks)
        for split in ("auto", 48):
            assert_attention(run_window(s, window, sinks, split), ref, mag)
    assert s.error_bits() == 0
