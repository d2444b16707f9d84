"""Operators for steps that are planned on the GPU and for prompts with images,
as they are called and in plain torch.

  plan       block tables, row offsets, context lengths and slot maps of a batch
             from the requests' lengths: blocks come off a ring of free ids;
  positions  rotary positions (time, height, width) of a batch's tokens from
             their sequences' segments of text and of t x h x w grids;
  axes       the rotary turn of q and k with a position for each axis, and the
             write of k, v into the cache (case key "int8"); the turned k also
             leaves as rows;
  prompt     causal attention of whole prompts, packed one after another, from
             their rows of q, k and v, with an optional window and sinks.

`own` False computes them with elementary torch operations (32 bits, angles in
64), `own` True makes the calls of this package.
"""

import math
import random

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _case(op, B, new, ctx, **kw):
    """new, ctx: (smallest, largest) tokens brought and context after them."""
    c = dict(op=op, batch=B, new_min=new[0], new_max=new[1], ctx_min=ctx[0], ctx_max=ctx[1], shape_seed=1)
    c.update(kw)
    return c


def _plan(B, new, ctx, bs, width, pad=0, **kw):
    """width: blocks a sequence may have; pad: entries of the batch without a sequence."""
    return _case("plan", B, new, ctx, block=bs, width=width, pad=pad, **kw)


def _positions(B, new, ctx, segments, **kw):
    return _case("positions", B, new, ctx, segments=segments, **kw)


def _axes(B, new, ctx, heads, bs, int8, **kw):
    c = dict(hq=heads[0], hkv=heads[1], dim=heads[2], block=bs, int8=int8, rotary=heads[2], interleaved=False,
             cycled=False)
    c.update(kw)
    return _case("axes", B, new, ctx, **c)


def _prompt(B, new, heads, window=0, sinks=0, **kw):
    return _case("prompt", B, new, new, hq=heads[0], hkv=heads[1], dim=heads[2], window=window, sinks=sinks, **kw)


TINY, TTS, MHA, GQA = (4, 2, 64), (16, 8, 128), (32, 32, 128), (32, 8, 128)


def listed():
    return [
        # one decode step of a few short sequences: what a call costs in latency
        _plan(4, (1, 1), (1, 100), 16, 8, name="plan_step_tiny"),
        # a decode step of a full batch, contexts of all lengths, some entries without a sequence
        _plan(128, (1, 1), (16, 16384), 16, 1024, pad=16, name="plan_step"),
        # chunks of prompts of many sequences planned at once
        _plan(512, (1, 200), (200, 16384), 16, 1024, name="plan_chunks"),
        # one token each, behind prompts with some images
        _positions(128, (1, 1), (16, 16384), 24, name="positions_step"),
        # whole prompts with images and video
        _positions(8, (5000, 8192), (5000, 8192), 48, name="positions_prompt"),
        # one token each for a full batch, INT8 cache: written, and the row read back
        _axes(128, (1, 1), (16, 4096), GQA, 16, True, name="axes_step_int8"),
        # prompts with images into a bf16 cache
        _axes(4, (7000, 8000), (7000, 8000), TTS, 16, False, name="axes_prompt_bf16"),
        # ragged prompts, axes dealt out in turn, quantized as they are written, and read back
        _axes(16, (16, 4096), (16, 4096), GQA, 16, True, cycled=True, name="axes_prompt_int8"),
        # a few short prompts of a very small model
        _prompt(4, (1, 100), TINY, name="prompt_tiny"),
        # prompts of all lengths packed into one call
        _prompt(32, (16, 4096), GQA, name="prompt_ragged"),
        # prompts of a windowed model
        _prompt(2, (5000, 8192), GQA, 1024, 4, name="prompt_window"),
        # whole prompts of a speech model: the most arithmetic
        _prompt(4, (7400, 8000), TTS, name="prompt_causal"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "positions", "axes", "prompt", "prompt"])
    seed = rng.randrange(1 << 30)
    heads = rng.choice([TINY, (8, 1, 64), TTS, MHA, GQA, (16, 2, 128)])
    step = rng.random() < 0.4
    if op == "plan":
        bs, hi = rng.choice([16, 64]), _log_int(rng, 16, 16384)
        new = 1 if step else _log_int(rng, 1, min(hi, 200))
        width = -(-hi // bs) + rng.choice([0, 1, _log_int(rng, 1, 300)])
        return _plan(_log_int(rng, 1, 500), (1 if step else max(1, new // 8), new), (new, hi), bs, width,
                     pad=rng.choice([0, 0, 1, 40]), shape_seed=seed)
    if op == "positions":
        hi = _log_int(rng, 8, 8192)
        new = (1, 1) if step else (max(1, hi // 3), hi)
        return _positions(_log_int(rng, 1, 128 if step else 8), new, (new[0], hi), _log_int(rng, 1, 60), shape_seed=seed)
    if op == "axes":
        new = 1 if step else _log_int(rng, 2, 6000)
        low = _log_int(rng, 1, new)
        B = _log_int(rng, 1, 128 if step else 4)
        return _axes(B, (low, new), (16, 4096) if step else (low, new), heads, rng.choice([16, 64]), rng.random() < 0.5,
                     rotary=rng.choice([heads[2], heads[2] // 2]), interleaved=rng.random() < 0.5,
                     cycled=rng.random() < 0.5, shape_seed=seed)
    hi = _log_int(rng, 1, 8000)
    B = max(1, min(_log_int(rng, 1, 64), 16000 // hi))
    window = rng.choice([0, 0, _log_int(rng, 1, 4096)])
    return _prompt(B, (max(1, _log_int(rng, 1, hi)), hi), heads, window, rng.choice([0, 1, 4, 37]) if window else 0,
                   shape_seed=seed)


def _lengths(case):
    """(new tokens, context) of each sequence; the longest is always among them."""
    rng = random.Random(case["shape_seed"])
    new, ctx = [], []
    for b in range(case["batch"]):
        n = case["new_max"] if b == 0 else _log_int(rng, case["new_min"], case["new_max"])
        if (case["new_min"], case["new_max"]) == (case["ctx_min"], case["ctx_max"]):
            c = n  # whole prompts
        else:
            c = max(n, case["ctx_max"] if b == 0 else _log_int(rng, case["ctx_min"], case["ctx_max"]))
        new.append(n)
        ctx.append(c)
    return new, ctx


def _rows_of(T):
    """Rows that the token arrays of a plan have: a few more than the batch needs."""
    return -(-T // 64) * 64


def work(case):
    new, ctx = _lengths(case)
    T, B = sum(new), len(new)
    if case["op"] == "plan":
        E, bs = B + case["pad"], case["block"]
        read = E * 8 + B * 8 + 4 * sum(-(-c // bs) for c in ctx)
        wrote = 4 * (E + 1 + 2 * E + E * case["width"] + 4 * _rows_of(T))
        return {"bytes": read + wrote, "flops": 4 * T + E * case["width"]}
    if case["op"] == "positions":
        return {"bytes": B * (12 + 4) + B * case["segments"] * 16 + 12 * T, "flops": 12 * T}
    hq, hkv, d = case["hq"], case["hkv"], case["dim"]
    if case["op"] == "axes":
        row = 2 * hkv * d * (1 if case["int8"] else 2)  # one token's K and V in the cache
        io = T * (hq * d * 4 + hkv * d * 6 + 12) + T * row
        back = T * row + T * 2 * hkv * d * 2 if case["int8"] else 0
        return {"bytes": io + back, "flops": 3 * T * (hq + hkv) * case["rotary"]}
    pairs = 0
    for n in new:
        w = case["window"] or n
        for p in range(n):
            lo = max(0, p - w + 1)
            pairs += p + 1 - lo + min(case["sinks"], lo)
    return {"bytes": T * (2 * hq + 2 * hkv) * d * 2, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _dev(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def _segments(rng, length, most):
    """Text and grids in turn over about the sequence's first `length` tokens, at most `most` segments."""
    segs, left = [], length
    while left > 0 and len(segs) < most - 1:
        n = min(left, int(rng.integers(1, max(2, length // most))))
        segs.append((n, 0, 0, 1))
        left -= n
        # an image, or a video of a few frames
        share = max(4, 2 * length // most)
        t = int(rng.integers(2, 9)) if rng.random() < 0.3 else 1
        h = int(rng.integers(1, max(2, math.isqrt(share // t) + 1)))
        w = max(1, min(share // (t * h), 2 * h))
        if t * h * w <= left and len(segs) < most - 1:
            segs.append((t, h, w, int(rng.integers(1, 4)) if t > 1 else 1))
            left -= t * h * w
    # what is left, up to a few tokens that a decode step has added since, is text
    if left > 3:
        segs.append((left - 3, 0, 0, 1))
    return segs


def _axis_of_pair(case):
    """Axis of each pair: sections of a quarter (time) and twice three eighths, or dealt out in turn."""
    half = case["rotary"] // 2
    side = 3 * half // 8
    if not case["cycled"]:
        return [0] * (half - 2 * side) + [1] * side + [2] * side
    return [j % 3 if j % 3 and j < 3 * side else 0 for j in range(half)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    new, ctx = _lengths(case)
    B, T = len(new), sum(new)
    s = dict(case=case, new=new, ctx_host=ctx, T=T, most=max(new))
    if case["op"] == "plan":
        _prepare_plan(s, rng)
    else:
        s["starts"], s["ctx"] = _dev(np.cumsum([0] + new)), _dev(ctx)
    if case["op"] in ("positions", "axes"):
        most = case.get("segments", 24)
        segs = [_segments(rng, c, most) for c in ctx]
        table = np.zeros((B, most, 4), np.int32)
        for b, x in enumerate(segs):
            table[b, :len(x)] = x
        s["segs_host"], s["segs"], s["nseg"] = segs, _dev(table), _dev([len(x) for x in segs])
    if case["op"] == "positions":
        s["out"] = torch.empty((3, T), dtype=torch.int32, device="cuda")
    if case["op"] in ("axes", "prompt"):
        hq, hkv, d = case["hq"], case["hkv"], case["dim"]
        # the three parts of one projection's output, as a model has them
        qkv = torch.randn((T, hq + 2 * hkv, d), generator=g, device="cuda", dtype=torch.bfloat16)
        qkv[:, hq:] *= 0.1 + 1.9 * torch.rand((2 * hkv, 1), generator=g, device="cuda").to(torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if case["op"] == "axes":
        _prepare_axes(s, rng, g)
    if own:
        s.update(_handles(s))
    return s


def _prepare_plan(s, rng):
    c = s["case"]
    B, E, bs, width = c["batch"], c["batch"] + c["pad"], c["block"], c["width"]
    slots_of = rng.permutation(B + 7)
    before = [x - n for x, n in zip(s["ctx_host"], s["new"])]
    held = [-(-x // bs) for x in before]
    # some sequences hold a block ahead
    held = [min(width, h + int(rng.random() < 0.1)) for h in held]
    need = [max(0, -(-x // bs) - h) for x, h in zip(s["ctx_host"], held)]
    N = sum(held) + sum(need) + 5
    ids = rng.permutation(N)
    tables = np.full((B + 7, width), -1, np.int32)
    lens, have = np.zeros(B + 7, np.int32), np.zeros(B + 7, np.int32)
    at = 0
    for b in range(B):
        sl = slots_of[b]
        tables[sl, :held[b]] = ids[at:at + held[b]]
        at += held[b]
        lens[sl], have[sl] = before[b], held[b]
    free, head = ids[at:], int(rng.integers(0, N))
    ring = np.full(N, -1, np.int32)
    ring[(head + np.arange(free.size)) % N] = free
    # the batch's entries: the sequences in order, entries without one among them
    place = np.sort(rng.permutation(E)[:B])
    slots, counts = np.full(E, -1, np.int32), np.zeros(E, np.int32)
    slots[place], counts[place] = slots_of[:B], s["new"]
    s.update(N=N, rows=_rows_of(s["T"]), tables=_dev(tables), lens=_dev(lens), held=_dev(have), ring=_dev(ring),
             state=_dev([head, free.size, 0, 0]), slots=_dev(slots), counts=_dev(counts))
    for name, shape in (("starts", E + 1), ("ctx", E), ("fill", E), ("out_tables", (E, width)), ("block_ids", s["rows"]),
                        ("offsets", s["rows"]), ("token_slots", s["rows"]), ("positions", s["rows"])):
        s[name] = torch.empty(shape, dtype=torch.int32, device="cuda")


def _prepare_axes(s, rng, g):
    c = s["case"]
    B, bs, hq, hkv, d, half = c["batch"], c["block"], c["hq"], c["hkv"], c["dim"], c["rotary"] // 2
    blocks = [-(-x // bs) for x in s["ctx_host"]]
    num_blocks, width = sum(blocks) + 3, max(blocks)
    ids = rng.permutation(num_blocks)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = ids[at:at + n]
        at += n
    s.update(num_blocks=num_blocks, tables=_dev(table), slots=_dev(rng.permutation(B)) if c["int8"] else None,
             inv_freq=_dev(10000.0 ** (-np.arange(half) / half), torch.float64), axis=_axis_of_pair(c),
             pos=_dev(_positions_of(s)))
    for name in "kv":
        rows = torch.randn((num_blocks, hkv, bs, d), generator=g, device="cuda", dtype=torch.bfloat16)
        if c["int8"]:
            s[name + "_tail"] = torch.randn((B, hkv, bs, d), generator=g, device="cuda", dtype=torch.bfloat16)
            s[name + "_pool"] = (rows.float() * 30).clamp(-127, 127).to(torch.int8)
        else:
            s[name + "_pool"] = rows
    if c["int8"]:
        s["scales"] = 0.01 + 0.02 * torch.rand((num_blocks, hkv, 2), generator=g, device="cuda")


def _handles(s):
    """What a program that uses the package keeps: descriptors, the layer's
    cache and the output buffers."""
    from paged_kv_cache_56_gb300 import pkv
    from paged_kv_cache_56_gb300.runtime import LayerCache
    c, h = s["case"], {}
    if c["op"] == "plan":
        h["pool"] = pkv.make_seq_pool(s["tables"], s["lens"], s["held"], s["ring"], s["state"], block_size=c["block"])
        h["plan"] = pkv.make_plan(s["starts"], s["out_tables"], s["ctx"], num_tokens=s["rows"], max_tokens=s["most"],
                                  fill_blocks=s["fill"], block_ids=s["block_ids"], offsets=s["offsets"],
                                  token_slots=s["token_slots"], positions=s["positions"])
        return h
    dummy = torch.zeros((c["batch"], 1 << 14), dtype=torch.int32, device="cuda")
    h["batch"] = pkv.make_batch(s["starts"], s.get("tables", dummy), s["ctx"], s.get("slots"), num_tokens=s["T"],
                                max_tokens=s["most"])
    if c["op"] == "positions":
        return h
    h["out"] = torch.empty((s["T"], c["hq"], c["dim"]), dtype=torch.bfloat16, device="cuda")
    if c["op"] == "prompt":
        h["layer"] = LayerCache(1, c["hq"], c["hkv"], c["dim"], 16, False, 0)
        return h
    lc = h["layer"] = LayerCache(s["num_blocks"], c["hq"], c["hkv"], c["dim"], c["block"], c["int8"], c["batch"])
    for name in ("k_pool", "v_pool", "scales", "k_tail", "v_tail"):
        if s.get(name) is not None:
            getattr(lc, name).copy_(s[name])
            h[name] = getattr(lc, name)
    h["rope"] = pkv.make_rope_axes(s["inv_freq"], s["axis"], positions=s["pos"], interleaved=c["interleaved"])
    h["k_out"] = torch.empty((s["T"], c["hkv"], c["dim"]), dtype=torch.bfloat16, device="cuda")
    if c["int8"]:
        h["rows"] = [torch.empty((s["T"], c["hkv"], c["dim"]), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    return h


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

_PLAN_OUT = ("starts", "ctx", "out_tables", "fill", "block_ids", "offsets", "token_slots", "positions")


def run(s):
    c = s["case"]
    if own:
        from paged_kv_cache_56_gb300 import pkv
        if c["op"] == "plan":
            pkv.pkv_plan_batch(s["pool"], s["slots"], s["plan"], s["counts"])
            return (*(s[x] for x in _PLAN_OUT), s["held"], s["state"][:2])
        if c["op"] == "positions":
            pkv.pkv_axis_positions(s["batch"], s["segs"], s["nseg"], s["out"])
            return s["out"]
        desc = s["layer"].desc
        if c["op"] == "prompt":
            pkv.pkv_prompt_attention(desc, s["batch"], s["q"], s["k"], s["v"], s["out"], c["window"], c["sinks"],
                                     c["dim"] ** -0.5)
            return s["out"]
        pkv.pkv_rope_append_axes(desc, s["batch"], s["rope"], s["q"], s["k"], s["v"], s["out"], s["k_out"])
        if not c["int8"]:
            return s["out"], s["k_out"], s["k_pool"], s["v_pool"]
        pkv.pkv_gather_kv(desc, s["batch"], *s["rows"])
        return (s["out"], s["k_out"], *s["rows"])
    return {"plan": _plain_plan, "positions": _plain_positions, "axes": _plain_axes, "prompt": _plain_prompt}[c["op"]](s)


def _plain_plan(s):
    c = s["case"]
    bs, width, N, rows = c["block"], c["width"], s["N"], s["rows"]
    there = s["slots"] >= 0
    slot = s["slots"].clamp(min=0).long()
    n = torch.where(there, s["counts"], 0).long()
    before = torch.where(there, s["lens"][slot], 0).long()
    held = torch.where(there, s["held"][slot], 0).long()
    end = before + n
    need = (-(-end // bs) - held).clamp(min=0)
    upto = need.cumsum(0)
    head, total = s["state"][0].long(), upto[-1]
    # the new blocks: entry and index of each (as many as the rows can need at most)
    i = torch.arange(rows + n.numel(), device="cuda")
    b = torch.searchsorted(upto, i, right=True)
    real = b < n.numel()
    b = b.clamp(max=n.numel() - 1)
    col = held[b] + i - (upto - need)[b]
    fresh = s["ring"][(head + i) % N]
    at = torch.where(real, slot[b] * width + col, s["tables"].numel())
    flat = torch.cat([s["tables"].flatten(), s["tables"].new_zeros(1)])
    flat.scatter_(0, at, fresh)
    s["tables"].copy_(flat[:-1].view_as(s["tables"]))
    s["held"].scatter_add_(0, torch.where(there, slot, 0), torch.where(there, need, 0).to(torch.int32))
    s["state"][0] = (head + total) % N
    s["state"][1] -= total
    have = held + need
    out = torch.where(torch.arange(width, device="cuda") < have[:, None], s["tables"][slot], -1)
    starts = torch.cat([n.new_zeros(1), n.cumsum(0)])
    # the rows
    row = torch.arange(rows, device="cuda")
    e = torch.searchsorted(starts[1:].contiguous(), row, right=True)
    real = e < n.numel()
    e = e.clamp(max=n.numel() - 1)
    pos = before[e] + row - starts[e]
    block = out[e, (pos // bs).clamp(0, width - 1)]
    result = [starts, end, out, torch.where((n > 0) & (end % bs == 0), out[torch.arange(n.numel(), device="cuda"), (end - 1).clamp(min=0) // bs], -1),
              torch.where(real, block, -1), torch.where(real, pos % bs, 0), torch.where(real, s["slots"][e], -1),
              torch.where(real, pos, 0)]
    return (*(x.to(torch.int32) for x in result), s["held"], s["state"][:2])


def _rows(s):
    """Sequence and token of every row of the batch."""
    n = (s["starts"][1:] - s["starts"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n, output_size=s["T"])
    tok = (s["ctx"].long() - n - s["starts"][:-1].long())[seq] + torch.arange(s["T"], device="cuda")
    return seq, tok


def _plain_positions(s):
    t, h, w, step = s["segs"].long().unbind(-1)
    text = h == 0
    live = torch.arange(t.shape[1], device="cuda") < s["nseg"][:, None]
    tokens = torch.where(live, torch.where(text, t, t * h * w), 0)
    moves = torch.where(text, t, torch.maximum((t - 1) * step, torch.maximum(h - 1, w - 1)) + 1)
    moves = torch.where(live, moves, 0)
    end, base = tokens.cumsum(1), moves.cumsum(1)
    seq, tok = _rows(s)
    k = (tok[:, None] >= end[seq]).sum(1)                 # segments that end before the token
    behind = k == t.shape[1]
    k = k.clamp(max=t.shape[1] - 1)
    first, at = (end - tokens)[seq, k], (base - moves)[seq, k]
    first, at = torch.where(behind, end[seq, -1], first), torch.where(behind, base[seq, -1], at)
    i = tok - first
    plain = text[seq, k] | behind | ~live[seq, k]
    ww, hh = w[seq, k].clamp(min=1), h[seq, k].clamp(min=1)
    grid = torch.stack([i // (hh * ww) * step[seq, k], i // ww % hh, i % ww])
    return (at + torch.where(plain, i, grid)).to(torch.int32)


def _turn(x, cos, sin, interleaved):
    """x [T, H, d] fp32, its first 2 * cos.shape[1] elements turned."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    u, w = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, w], dim=-1).flatten(-2) if interleaved else torch.cat([u, w], dim=-1)
    return torch.cat([y, x[..., 2 * half:]], dim=-1).to(torch.bfloat16)


def _plain_axes(s):
    c, bs = s["case"], s["case"]["block"]
    seq, tok = _rows(s)
    axis = torch.tensor(s["axis"], device="cuda")
    angle = s["pos"][axis].double().T * s["inv_freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    out = _turn(s["q"].float(), cos, sin, c["interleaved"])
    rows = {"k": _turn(s["k"].float(), cos, sin, c["interleaved"]), "v": s["v"]}
    if not c["int8"]:
        block = s["tables"][seq, tok // bs].long()
        s["k_pool"][block, :, tok % bs] = rows["k"]
        s["v_pool"][block, :, tok % bs] = rows["v"]
        return out, rows["k"], s["k_pool"], s["v_pool"]
    # every block that the new tokens reach: its rows, old and new
    n, ctx = (s["starts"][1:] - s["starts"][:-1]).long(), s["ctx"].long()
    begin = (ctx - n) // bs
    count = (ctx - 1) // bs - begin + 1
    total = sum((x - 1) // bs - (x - m) // bs + 1 for m, x in zip(s["new"], s["ctx_host"]))
    b = torch.repeat_interleave(torch.arange(c["batch"], device="cuda"), count, output_size=total)
    last = count.cumsum(0) - 1
    blk = torch.arange(total, device="cuda") - (last - count + 1)[b] + begin[b]
    t = blk[:, None] * bs + torch.arange(bs, device="cuda")
    fresh = ((t >= (ctx - n)[b][:, None]) & (t < ctx[b][:, None]))[:, None, :, None]
    row = (t - (ctx - n - s["starts"][:-1].long())[b][:, None]).clamp(0, s["T"] - 1)
    ids, slots = s["tables"][b, blk].long(), s["slots"].long()
    full = ((blk + 1) * bs <= ctx[b])[:, None, None, None]
    back = []
    for kv, name in enumerate("kv"):
        x = torch.where(fresh, rows[name][row].transpose(1, 2), s[name + "_tail"][slots[b]])
        y = x.float()
        top = y.abs().amax(dim=(2, 3), keepdim=True)
        scale = torch.where(top < 1e-6, torch.ones_like(top), top / 127)
        code = torch.round(y / scale).clamp(-127, 127).to(torch.int8)
        s[name + "_pool"][ids] = torch.where(full, code, s[name + "_pool"][ids])
        s["scales"][ids, :, kv] = torch.where(full, scale, s["scales"][ids, :, kv, None, None])[:, :, 0, 0]
        s[name + "_tail"][slots] = torch.where(full[last], s[name + "_tail"][slots], x[last])
        # the rows read back, dequantized
        at = s["tables"][seq, tok // bs].long()
        z = s[name + "_pool"][at, :, tok % bs].float() * s["scales"][at, :, kv].unsqueeze(-1)
        tail = s[name + "_tail"][slots[seq], :, tok % bs].float()
        back.append(torch.where((tok >= ctx[seq] // bs * bs)[..., None, None], tail, z).to(torch.bfloat16))
    return out, rows["k"], *back


def _plain_prompt(s):
    c = s["case"]
    hq, hkv, d, window, sinks = c["hq"], c["hkv"], c["dim"], c["window"], c["sinks"]
    out, at = [], 0
    for n in s["new"]:
        q, k, v = (s[x][at:at + n].float().transpose(0, 1) for x in "qkv")
        at += n
        i = torch.arange(n, device="cuda")
        hide = i > i[:, None]
        if window > 0:
            hide |= (i[:, None] - i >= window) & (i >= sinks)
        score = (q.reshape(hkv, -1, d) @ k.transpose(1, 2)).mul_(d ** -0.5).view(hq, n, n)
        score.masked_fill_(hide, -math.inf)
        score.sub_(score.amax(dim=-1, keepdim=True)).exp_()
        total = score.sum(dim=-1, keepdim=True)
        y = (score.view(hkv, -1, n) @ v).view(hq, n, d) / total
        out.append(y.transpose(0, 1).to(torch.bfloat16))
    return torch.cat(out)


# ---------------------------------------------------------------------------
# In 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _positions_of(s):
    """[3, T] of the batch's tokens, segment by segment on the host."""
    parts = []
    for n, ctx, segs in zip(s["new"], s["ctx_host"], s["segs_host"]):
        rows, base = [], 0
        for t, h, w, step in segs:
            if h == 0:
                part = np.tile(np.arange(t), (3, 1))
            else:
                i, j, k = np.meshgrid(np.arange(t) * step, np.arange(h), np.arange(w), indexing="ij")
                part = np.stack([i.ravel(), j.ravel(), k.ravel()])
            rows.append(base + part)
            base += int(part.max()) + 1
        have = sum(r.shape[1] for r in rows)
        if have < ctx:
            rows.append(np.tile(base + np.arange(ctx - have), (3, 1)))
        parts.append(np.concatenate(rows, axis=1)[:, ctx - n:ctx])
    return np.concatenate(parts, axis=1)


def _exact_plan(s):
    c, bs = s["case"], s["case"]["block"]
    tables, lens, held, ring = (s[x].cpu().numpy().copy() for x in ("tables", "lens", "held", "ring"))
    head, free = s["state"][:2].tolist()
    starts, ctx, fill, ids, off, slot, pos = [0], [], [], [], [], [], []
    out = np.full((s["slots"].numel(), c["width"]), -1)
    for e, (sl, n) in enumerate(zip(s["slots"].tolist(), s["counts"].tolist())):
        if sl < 0:
            starts.append(starts[-1])
            ctx.append(0)
            fill.append(-1)
            continue
        while held[sl] * bs < lens[sl] + n:
            tables[sl, held[sl]] = ring[head]
            held[sl] += 1
            head, free = (head + 1) % s["N"], free - 1
        out[e, :held[sl]] = tables[sl, :held[sl]]
        for p in range(lens[sl], lens[sl] + n):
            ids.append(out[e, p // bs])
            off.append(p % bs)
            slot.append(sl)
            pos.append(p)
        starts.append(starts[-1] + n)
        ctx.append(lens[sl] + n)
        fill.append(out[e, ctx[-1] // bs - 1] if n and ctx[-1] % bs == 0 else -1)
    rest = s["rows"] - len(ids)
    return tuple(_dev(x) for x in (starts, ctx, out, fill, ids + [-1] * rest, off + [0] * rest, slot + [-1] * rest,
                                   pos + [0] * rest, held, [head, free]))


def _exact_turn(x, s):
    c = s["case"]
    axis = torch.tensor(s["axis"], device="cuda")
    a = s["pos"].double()[axis].T * s["inv_freq"]
    z = torch.polar(torch.ones_like(a), a)[:, None]
    y = x.double().clone()
    half = c["rotary"] // 2
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
    turned = torch.complex(y[:, :, first], y[:, :, second]) * z
    y[:, :, first], y[:, :, second] = turned.real, turned.imag
    return y


def _exact_axes(s):
    c, bs = s["case"], s["case"]["block"]
    rows = {"k": _exact_turn(s["k"], s), "v": s["v"].double()}
    result = [_exact_turn(s["q"], s), rows["k"]]
    for name in "kv":
        pool = s[name + "_pool"].double() if not c["int8"] else None
        back, at = [], 0
        for b, (n, ctx) in enumerate(zip(s["new"], s["ctx_host"])):
            x = rows[name][at:at + n]
            at += n
            begin = (ctx - n) // bs * bs
            if not c["int8"]:
                t = torch.arange(ctx - n, ctx, device="cuda")
                pool[s["tables"][b, t // bs].long(), :, t % bs] = x
                continue
            # the cache holds rows rounded to bf16; a block that is full is then quantized
            x = x.to(torch.bfloat16).double()
            old = s[name + "_tail"][int(s["slots"][b]), :, :ctx - n - begin].double().transpose(0, 1)
            x = torch.cat([old, x])
            whole = x.shape[0] // bs * bs
            y = x[:whole].view(-1, bs, c["hkv"], c["dim"])
            top = y.abs().amax(dim=(1, 3), keepdim=True)
            scale = torch.where(top < 1e-6, torch.ones_like(top), top / 127)
            y = torch.round(y / scale).clamp(-127, 127) * scale
            back.append(torch.cat([y.reshape(whole, c["hkv"], c["dim"]), x[whole:]])[ctx - n - begin:])
        result.append(torch.cat(back) if c["int8"] else pool)
    return tuple(result)


def _exact_prompt(s):
    c = s["case"]
    G, window, sinks = c["hq"] // c["hkv"], c["window"], c["sinks"]
    out, at = [], 0
    for n in s["new"]:
        k, v = s["k"][at:at + n].double(), s["v"][at:at + n].double()
        for i in range(0, n, 512):
            m = min(512, n - i)
            p = torch.arange(i, i + m, device="cuda")[:, None]
            t = torch.arange(i + m, device="cuda")
            if window > 0:  # leave out what none of these tokens sees
                t = t[(t < sinks) | (t > i - window)]
            hide = t > p
            if window > 0:
                hide |= (p - t >= window) & (t >= sinks)
            q = s["q"][at + i:at + i + m].double().view(m, c["hkv"], G, c["dim"])
            logit = torch.einsum("mhgd,thd->hgmt", q, k[t]) / math.sqrt(c["dim"])
            logit[:, :, hide] = -math.inf
            weight = torch.exp(logit - torch.logsumexp(logit, dim=-1, keepdim=True))
            out.append(torch.einsum("hgmt,thd->mhgd", weight, v[t]).reshape(m, c["hq"], c["dim"]))
        at += n
    return torch.cat(out)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s)
    if case["op"] == "positions":
        return _dev(_positions_of(s))
    return _exact_axes(s) if case["op"] == "axes" else _exact_prompt(s)
