"""Rotary positions on several axes, and the rotary append that uses them."""

import random

import numpy as np
import pytest
import torch

from chunk_ref import Setup, turned
from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv
from plan_ref import dev
from test_gpu_chunk import APPENDS, expected_cache, freqs, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


# ---------------------------------------------------------------------------
# Positions
# ---------------------------------------------------------------------------

def positions_of(segs, upto):
    """Positions of tokens 0 .. upto-1, token by token."""
    out, base = [], 0
    for t, h, w, step in segs:
        top = base - 1
        if h == 0 and w == 0:
            for i in range(t):
                out.append((base + i,) * 3)
            top = base + t - 1
        else:
            for i in range(t):
                for j in range(h):
                    for k in range(w):
                        out.append((base + i * step, base + j, base + k))
                        top = max(top, *out[-1])
        base = top + 1
    while len(out) < upto:
        out.append((base,) * 3)
        base += 1
    return np.array(out[:upto], np.int64).reshape(-1, 3).T


def make(seqs, new, ctx, max_segments=None, pad=3):
    most = max([len(x) for x in seqs] + [1]) if max_segments is None else max_segments
    table = np.full((len(seqs), most, 4), -5, np.int32)  # behind a list's end: not looked at
    for b, x in enumerate(seqs):
        if x:
            table[b, :len(x)] = x
    T = sum(new)
    batch = pkv.make_batch(dev(np.cumsum([0] + new)), dev(np.zeros((len(new), 1))), dev(ctx), num_tokens=T + pad,
                           max_tokens=max(new + [0]))
    out = torch.full((3, T + pad + 2), -9, dtype=torch.int32, device="cuda")
    return batch, dev(table), dev([len(x) for x in seqs]), out


def random_segments(rng, most):
    segs = []
    for _ in range(rng.randint(0, most)):
        if rng.random() < 0.5:
            segs.append((rng.choice([0, 1, 2, 40, 700]), 0, 0, rng.randint(0, 3)))
        else:
            segs.append((rng.randint(0, 4), rng.randint(1, 12), rng.randint(1, 12), rng.randint(0, 5)))
    return segs


@pytest.mark.parametrize("most", [1, 5, 40, 300, 700])
@pytest.mark.parametrize("kind", ["step", "chunk", "prompt"])
def test_axis_positions(kind, most):
    rng = random.Random(most)
    seqs = [random_segments(rng, most) for _ in range(9)] + [[], [(1, 1, 1, 1)]]
    lens = [sum(t if h == 0 else t * h * w for t, h, w, _ in x) for x in seqs]
    ctx = [max(1, n + rng.choice([-1, 0, 1, 5, -n // 2])) for n in lens]
    new = [1 if kind == "step" else c if kind == "prompt" else min(c, rng.randint(0, 1500)) for c in ctx]
    batch, segs, count, out = make(seqs, new, ctx)
    err = dev([0])
    pkv.pkv_axis_positions(batch, segs, count, out, err=err)
    T = sum(new)
    want = np.concatenate([positions_of(x, c)[:, c - n:] for x, n, c in zip(seqs, new, ctx)], axis=1)
    assert np.array_equal(out[:, :T].cpu().numpy(), want)
    assert (out[:, T:] == -9).all() and err.item() == 0
    # lists kept by slot
    order = list(range(len(seqs) + 4))
    rng.shuffle(order)
    rows = order[:len(seqs)]
    kept, have = torch.full((len(order), *segs.shape[1:]), -5, dtype=torch.int32, device="cuda"), dev([-3] * len(order))
    kept[rows], have[rows] = segs, count
    again = torch.full_like(out, -9)
    pkv.pkv_axis_positions(batch, kept, have, again, rows=dev(rows), err=err)
    assert torch.equal(again, out) and err.item() == 0


def test_large_segments_and_the_last_position():
    big = 2 ** 31 - 1
    seqs = [[(big, 0, 0, 1)], [(1, 1, big, 1)], [(2, 1, 1, big)], [(2, 1, 1, 2 ** 30), (2, 1, 1, 2 ** 30), (5, 0, 0, 0)]]
    new, ctx = [5, 4, 3, 9], [2 ** 30, 70000, 3, 9]
    batch, segs, count, out = make(seqs, new, ctx)
    pkv.pkv_axis_positions(batch, segs, count, out)
    got = out[:, :21].cpu().numpy()
    assert got[:, :5].tolist() == [[2 ** 30 - 5 + i for i in range(5)]] * 3
    assert got[:, 5:9].tolist() == [[0] * 4, [0] * 4, [69996 + i for i in range(4)]]
    assert got[:, 9:12].tolist() == [[0, big, big], [0, 0, big], [0, 0, big]]
    # 0, 2^30 | 2^30 + 1, 2^31 + 1 | from 2^31 + 2 on: the last position
    assert got[:, 12:].tolist() == [[0, 2 ** 30, 2 ** 30 + 1] + [big] * 6, [0, 0, 2 ** 30 + 1, 2 ** 30 + 1] + [big] * 5,
                                    [0, 0, 2 ** 30 + 1, 2 ** 30 + 1] + [big] * 5]


def test_segments_that_cannot_be():
    bad = [(-1, 0, 0, 1), (1, 2, 0, 1), (1, 0, 2, 1), (1, -1, 2, 1), (2, 2, 2, -1), (-2, 2, 2, 1), (2, 2 ** 30, 2, 1),
           (3, 1, 1, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1), (-2 ** 31, 2, 2, 2)]
    seqs = [[(3, 0, 0, 1), x, (2, 2, 2, 1)] for x in bad]
    new = ctx = [13] * len(bad)
    batch, segs, count, out = make(seqs, new, ctx)
    err = dev([0])
    pkv.pkv_axis_positions(batch, segs, count, out, err=err)
    want = positions_of([(3, 0, 0, 1), (2, 2, 2, 1)], 13)  # it counts as empty
    assert np.array_equal(out[:, :13 * len(bad)].cpu().numpy(), np.tile(want, (1, len(bad))))
    assert err.item() == pkv.PKV_DEVERR_SEGMENT
    # numbers of segments, rows and lengths that cannot be: those sequences' rows stay
    for arrays, bits in ((dict(count=[3, -1, 3, 4]), pkv.PKV_DEVERR_SEGMENT), (dict(rows=[0, 4, 2, -1]), pkv.PKV_DEVERR_SLOT),
                         (dict(ctx=[13, 12, 13, -1]), pkv.PKV_DEVERR_CTX_LEN),
                         (dict(ctx=[13, 2 ** 31 - 1, 13, 2 ** 31 - 2 ** 16]), pkv.PKV_DEVERR_CTX_LEN), (dict(starts=[0, 13, 12, 39, 60]), pkv.PKV_DEVERR_BATCH)):
        batch, segs, count, out = make([[(3, 0, 0, 1), (2, 2, 2, 1), (0, 0, 0, 0)]] * 4, [13] * 4, arrays.get("ctx", [13] * 4))
        if "starts" in arrays:
            batch.keep[0].copy_(dev(arrays["starts"]))
        if "count" in arrays:
            count = dev(arrays["count"])
        rows = dev(arrays["rows"]) if "rows" in arrays else None
        err = dev([0])
        pkv.pkv_axis_positions(batch, segs, count, out, rows=rows, err=err)
        assert err.item() == bits
        got = out.cpu().numpy()
        assert np.array_equal(got[:, :13], want)
        if "starts" not in arrays:
            assert (got[:, 13:26] == -9).all() and np.array_equal(got[:, 26:39], want) and (got[:, 39:] == -9).all()
        else:
            assert (got[:, 39:] == -9).all()


# ---------------------------------------------------------------------------
# Rotary append
# ---------------------------------------------------------------------------

def axes_of(half, kind):
    side = 3 * half // 8
    return {"one": [0] * half, "parts": [0] * (half - 2 * side) + [1] * side + [2] * side,
            "in_turn": [j % 3 for j in range(half)], "four": [(7 * j) % 4 for j in range(half)]}[kind]


def turned_axes(x, pos, axis, inv_freq, interleaved, scale):
    """Rows x [T, H, d] turned, fp64: each axis' pairs by that axis' positions."""
    y = x.double().numpy().copy()
    half = len(inv_freq)
    for a in sorted(set(axis)):
        z = turned(x, pos[a], inv_freq, interleaved, scale)
        for j in range(half):
            if axis[j] == a:
                for e in ((2 * j, 2 * j + 1) if interleaved else (j, j + half)):
                    y[:, :, e] = z[:, :, e]
    return y


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 8, 64), (16, 8, 128), (8, 1, 128)])
@pytest.mark.parametrize("name", list(APPENDS))
def test_rope_append_axes(name, heads, bs, int8):
    new, ctx = APPENDS[name]
    hq, hkv, d = heads
    rng = np.random.default_rng(5)
    for rotary, inter, scale, kind in ((d, False, 1.0, "parts"), (d // 2, True, 1.25, "in_turn"), (48, False, 1.0, "four"),
                                       (d, True, 1.0, "parts"), (0, False, 1.0, "one")):
        s = Setup(61, new, ctx, heads, bs, int8, appended=False)
        f, axis = freqs(rotary // 2), axes_of(rotary // 2, kind)
        pos = rng.integers(0, 100000, (4, s.T + 1)).astype(np.int32)
        rope = None
        if rotary:
            wide = torch.full((4, s.T + 6), 7, dtype=torch.int32, device="cuda")  # rows of a wider array
            wide[:, :s.T + 1] = torch.as_tensor(pos)
            rope = pkv.make_rope_axes(torch.as_tensor(f).cuda(), axis, positions=wide[:, :s.T + 1], interleaved=inter,
                                      scale=scale)
        k, v = s.new_rows("k"), s.new_rows("v")
        qkv = torch.cat([s.q, k, v], dim=1).cuda()
        parts = qkv[:, :hq], qkv[:, hq:-hkv], qkv[:, -hkv:]
        q_out = torch.empty((s.T, hq, d), dtype=torch.bfloat16, device="cuda")
        k_out = torch.full((s.T + 1, hkv + 1, d), 3.0, dtype=torch.bfloat16, device="cuda")
        pkv.pkv_rope_append_axes(s.lc.desc, s.batch, rope, *parts, q_out, k_out[:, :hkv])
        got_k = k_out[:s.T, :hkv].cpu()
        # half a bf16 step of the result; products and angles in fp32: 2^-20 of the pair's size holds them
        for got, src in ((q_out.cpu(), s.q), (got_k, k)):
            want = turned_axes(src, pos[:, :s.T], axis, f, inter, scale) if rotary else src.double().numpy()
            big = src.double().abs().amax(dim=2, keepdim=True).numpy() * scale
            err = np.abs(got.double().numpy() - want) - (2.0 ** -8 * np.abs(want) + 2.0 ** -20 * big)
            assert (err <= 0).all(), (rotary, inter, kind, err.max())
            assert torch.equal(got[:, :, rotary:], src[:, :, rotary:])
        assert (k_out[s.T:] == 3).all() and (k_out[:, hkv:] == 3).all()
        # the cache holds those rows, quantized as the definition says
        pools, scales, tails = expected_cache(s, got_k, v)
        assert all(same(getattr(s.lc, n + "_pool"), pools[n]) for n in "kv")
        if int8:
            assert same(s.lc.scales, scales)
            assert all(same(getattr(s.lc, n + "_tail"), tails[n]) for n in "kv")
        assert s.error_bits() == 0
        # in place
        t = Setup(61, new, ctx, heads, bs, int8, appended=False)
        pkv.pkv_rope_append_axes(t.lc.desc, t.batch, rope, *parts, None, parts[1])
        assert torch.equal(parts[0], q_out) and torch.equal(parts[1], k_out[:s.T, :hkv])
        assert all(same(getattr(t.lc, n + "_pool"), pools[n]) for n in "kv")


@pytest.mark.parametrize("int8", [False, True])
def test_one_axis_is_the_plain_append(int8):
    new, ctx = [30, 1, 70, 16], [45, 33, 131, 16]
    for positions in (False, True):
        a, b = (Setup(7, new, ctx, (16, 8, 128), 16, int8, appended=False) for _ in range(2))
        f = torch.as_tensor(freqs(64)).cuda()
        pos = dev(np.arange(a.T) * 17 + 5) if positions else None
        q1, q2 = a.q.cuda(), b.q.cuda()
        k, v = a.new_rows("k").cuda(), a.new_rows("v").cuda()
        pkv.pkv_rope_append(a.lc.desc, a.batch, pkv.make_rope(f, positions=pos), q1, k, v)
        rope = pkv.make_rope_axes(f, [0] * 64, positions=None if pos is None else pos[None])
        pkv.pkv_rope_append_axes(b.lc.desc, b.batch, rope, q2, k, v)
        assert torch.equal(q1, q2)
        for n in ("k_pool", "v_pool") + (("k_tail", "v_tail", "scales") if int8 else ()):
            assert same(getattr(a.lc, n), getattr(b.lc, n))


@pytest.mark.parametrize("int8,bs", [(False, 16), (True, 16), (True, 64)])
def test_turned_rows_leave_even_where_the_cache_cannot_take_them(int8, bs):
    """A bad block id or slot is reported and nothing of its block is written; q and the turned k are there all the same."""
    s, good = (Setup(71, [100, 3, 20], [100, 30, 64], (4, 2, 64), bs, int8, appended=False) for _ in range(2))
    s.d_table[0, 0] = -5
    if int8:
        s.d_slots[1] = 99
    rope = pkv.make_rope_axes(torch.as_tensor(freqs(32)).cuda(), [0] * 32)
    k, v = s.new_rows("k").cuda(), s.new_rows("v").cuda()
    outs = []
    for x in (s, good):
        q_out, k_out = torch.empty_like(x.q, device="cuda"), torch.full_like(k, 9.0)
        pkv.pkv_rope_append_axes(x.lc.desc, x.batch, rope, x.q.cuda(), k, v, q_out, k_out)
        outs.append((q_out, k_out))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert s.error_bits() == pkv.PKV_DEVERR_BLOCK_ID | (pkv.PKV_DEVERR_SLOT if int8 else 0) and good.error_bits() == 0
