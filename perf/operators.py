"""The chunk operators of the paged cache, as they are called and in plain torch.

A batch holds B sequences; sequence b brings n_b new tokens (one in a decode
step, a few drafted ones, a chunk of a prompt or a whole prompt), its rows
starts[b] .. starts[b+1]-1 of the token arrays, which are tokens
ctx_b - n_b .. ctx_b - 1 of its context. Three operators work on such a batch:

  rope    the rotary turn of q and k and the write of k, v into the cache
          (an INT8 cache quantizes each block that fills: case key "int8");
  window  attention of the new tokens over the cache, causal, each token
          seeing the last `window` tokens (0: all) and the first `sinks`;
  gather  rows of the cache read back, dequantized, in token order.

`own` False computes them with elementary torch operations in 32 bits (angles
in 64), `own` True makes the calls of this package.
"""

import math
import random

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _case(op, B, new, ctx, heads, bs, int8, **kw):
    """new, ctx: (smallest, largest) tokens brought and context after them."""
    hq, hkv, d = heads
    c = dict(op=op, batch=B, new_min=new[0], new_max=new[1], ctx_min=ctx[0], ctx_max=ctx[1], hq=hq, hkv=hkv, dim=d,
             block=bs, int8=int8, window=0, sinks=0, rotary=d, interleaved=False, stretch=1.0, far=0, fp32=False,
             shape_seed=1)
    c.update(kw)
    return c


def listed():
    tiny, tts, mha, gqa = (4, 2, 64), (16, 8, 128), (32, 32, 128), (32, 8, 128)
    return [
        # one decode step of a very small model: what a call costs in latency
        _case("window", 4, (1, 1), (1, 100), tiny, 16, False, window=32, sinks=4, name="window_step_tiny"),
        # continuous batching with a windowed model: one token each, INT8 cache,
        # contexts far longer than the window
        _case("window", 64, (1, 1), (1000, 16384), gqa, 16, True, window=2048, sinks=4, name="window_step_int8"),
        # drafted tokens checked against the whole context in one call
        _case("window", 16, (2, 6), (6000, 8000), tts, 16, False, name="draft_step_bf16"),
        # prompts of a windowed model
        _case("window", 2, (5000, 8192), (5000, 8192), gqa, 16, False, window=1024, sinks=4, name="window_prompt_bf16"),
        # whole prompts of a speech model, no window: the most arithmetic
        _case("window", 4, (7400, 8000), (7400, 8000), tts, 16, False, name="causal_prompt_bf16"),
        # chunks of long prompts over an INT8 cache that is already long
        _case("window", 8, (100, 512), (9001, 32768), gqa, 64, True, window=4096, sinks=64, name="window_chunk_int8"),
        # one token each for a full batch, INT8 cache: written, and the row read back
        _case("rope", 128, (1, 1), (16, 4096), gqa, 16, True, name="rope_step_int8"),
        # prompts into a bf16 cache; half of each head turns, pairs interleaved,
        # frequencies stretched for long contexts, positions far out
        _case("rope", 4, (7000, 8000), (7000, 8000), tts, 16, False, rotary=64, interleaved=True, stretch=8.0,
              far=1000000, name="rope_prompt_bf16"),
        # ragged prompts quantized as they are written, and read back
        _case("rope", 16, (16, 4096), (16, 4096), gqa, 16, True, name="rope_prompt_int8"),
        # a few short contexts read back in fp32
        _case("gather", 4, (1, 100), (1, 100), tiny, 16, False, fp32=True, name="gather_tiny"),
        # long contexts read back from an INT8 cache (moved to another engine)
        _case("gather", 8, (30000, 32768), (30000, 32768), gqa, 64, True, name="gather_long_int8"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "rope", "gather"])
    heads = rng.choice([(4, 2, 64), (8, 1, 64), (16, 8, 128), (32, 32, 128), (32, 8, 128), (16, 2, 128)])
    bs, int8 = rng.choice([16, 64]), rng.random() < 0.5
    seed = rng.randrange(1 << 30)
    kind = rng.choice(["step", "draft", "chunk", "prompt"])
    top = {"step": 1, "draft": 9, "chunk": 700, "prompt": 6000}[kind]
    new_hi = 1 if kind == "step" else _log_int(rng, 2, top)
    new_lo = _log_int(rng, 1, new_hi)
    B = _log_int(rng, 1, {"step": 128, "draft": 32, "chunk": 8, "prompt": 2}[kind])
    if op == "gather":
        hi = _log_int(rng, 8, 16000)
        return _case("gather", min(B, 16), (max(1, hi // 3), hi), (max(1, hi // 3), hi), heads, bs, int8,
                     fp32=rng.random() < 0.5, shape_seed=seed)
    if op == "rope":
        far = rng.choice([0, 0, 100000])
        turn = rng.choice([heads[2], heads[2] // 2, heads[2] // 4])
        # whole prompts (a step where kind == "step"): a cache that has just been begun
        ctx = (new_lo, new_hi) if kind != "step" else (16, 4096)
        return _case("rope", B, (new_lo, new_hi), ctx, heads, bs, int8, rotary=turn, interleaved=rng.random() < 0.5,
                     stretch=rng.choice([1.0, 4.0]), far=far, shape_seed=seed)
    before = 0 if kind == "prompt" else _log_int(rng, 1, 12000)
    window = rng.choice([0, _log_int(rng, 1, 4096)])
    return _case("window", B, (new_lo, new_hi), (new_lo + before // 3, new_hi + before), heads, bs, int8,
                 window=window, sinks=rng.choice([0, 1, 4, 37]) if window else 0, shape_seed=seed)


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


def _visible(n, c, window, sinks):
    """(keys that some token of the sequence sees, pairs of a token and a key it sees)."""
    pairs = 0
    for p in range(c - n, c):
        lo = 0 if window <= 0 else max(0, p - window + 1)
        pairs += p + 1 - lo + min(sinks, lo)
    lo = 0 if window <= 0 else max(0, c - n - window + 1)
    return c - lo + min(sinks, lo), pairs


def work(case):
    new, ctx = _lengths(case)
    hq, hkv, d, T = case["hq"], case["hkv"], case["dim"], sum(new)
    row = 2 * hkv * d * (1 if case["int8"] else 2)  # one token's K and V in the cache
    if case["op"] == "window":
        keys = pairs = 0
        for n, c in zip(new, ctx):
            k, p = _visible(n, c, case["window"], case["sinks"])
            keys, pairs = keys + k, pairs + p
        return {"bytes": keys * row + T * hq * d * 4, "flops": 4 * d * hq * pairs}
    if case["op"] == "rope":
        io = T * (hq * d * 4 + 2 * hkv * d * 2) + T * row  # q in and out, k and v in, the cache written
        back = T * row + T * 2 * hkv * d * 2 if case["int8"] else 0
        return {"bytes": io + back, "flops": 3 * T * (hq + hkv) * case["rotary"]}
    return {"bytes": T * row + T * 2 * hkv * d * (4 if case["fp32"] else 2), "flops": T * 2 * hkv * d}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _frequencies(case):
    """fp64 radians a position of each pair, and the factor on the turned part:
    with a stretch, long wavelengths are interpolated and short ones kept."""
    half = case["rotary"] // 2
    f = 10000.0 ** (-np.arange(half, dtype=np.float64) / half)
    if case["stretch"] <= 1:
        return f, 1.0
    turns = 4096 * f / (2 * math.pi)
    keep = np.clip((turns - 1) / 31, 0, 1)
    return f * keep + f / case["stretch"] * (1 - keep), 0.1 * math.log(case["stretch"]) + 1


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    order = np.random.default_rng(seed)
    new, ctx = _lengths(case)
    B, T, bs = case["batch"], sum(new), case["block"]
    hq, hkv, d = case["hq"], case["hkv"], case["dim"]

    def dev(a, dtype=torch.int32):
        return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    blocks = [-(-c // bs) for c in ctx]
    num_blocks, width = sum(blocks) + 3, max(blocks)
    ids = order.permutation(num_blocks)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = ids[at:at + n]
        at += n
    # heads of different magnitudes, as attention layers have them
    spread = 0.1 + 1.9 * torch.rand((2, hkv, 1, 1), generator=g, device="cuda")
    s = dict(case=case, new=new, ctx_host=ctx, T=T, num_blocks=num_blocks, starts=dev(np.cumsum([0] + new)), ctx=dev(ctx),
             tables=dev(table), slots=dev(order.permutation(B)) if case["int8"] else None, keys=0)
    for i, name in enumerate("kv"):
        rows = normal(num_blocks, hkv, bs, d)
        if case["int8"]:
            s[name + "_tail"] = (normal(B, hkv, bs, d) * spread[i]).to(torch.bfloat16)
            top = rows.abs().amax(dim=(2, 3), keepdim=True).float()
            s[name + "_pool"] = torch.round(rows.float() * (127 / top)).to(torch.int8)
            s[name + "_scale"] = top[:, :, 0, 0] * spread[i, :, 0, 0] / 127
        else:
            s[name + "_pool"] = (rows * spread[i]).to(torch.bfloat16)
    if case["int8"]:
        s["scales"] = torch.stack([s.pop("k_scale"), s.pop("v_scale")], dim=2).contiguous()
    if case["op"] != "gather":
        # the three parts of one projection's output, as a model has them
        qkv = normal(T, (hq + 2 * hkv) * d).view(T, hq + 2 * hkv, d)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if case["op"] == "window":
        s["keys"] = max(c - (max(case["sinks"], c - n - case["window"] + 1) if case["window"] > 0 else 0)
                        for n, c in zip(new, ctx))
    if case["op"] == "rope":
        f, s["factor"] = _frequencies(case)
        s["inv_freq"] = dev(f, torch.float64)
        pos = np.concatenate([np.arange(c - n, c) for n, c in zip(new, ctx)])
        s["positions"] = dev(pos + case["far"]) if case["far"] else None
    if own:
        s.update(_handles(s))
    return s


def _handles(s):
    """What a program that uses the package keeps: the layer's cache, the batch
    and rotary descriptors, the workspace and the output buffers."""
    from paged_kv_cache_56_gb300 import pkv
    from paged_kv_cache_56_gb300.runtime import LayerCache
    c = s["case"]
    lc = LayerCache(s["num_blocks"], c["hq"], c["hkv"], c["dim"], c["block"], c["int8"], c["batch"])
    for name in ("k_pool", "v_pool", "scales", "k_tail", "v_tail"):
        if s.get(name) is not None:
            getattr(lc, name).copy_(s[name])
            s[name] = getattr(lc, name)
    batch = pkv.make_batch(s["starts"], s["tables"], s["ctx"], s["slots"], num_tokens=s["T"], max_tokens=max(s["new"]))
    h = dict(layer=lc, batch=batch)
    if c["op"] == "window":
        h["out"] = torch.empty((s["T"], c["hq"], c["dim"]), dtype=torch.bfloat16, device="cuda")
        h["split"] = pkv.pkv_window_split_tokens(lc.desc, batch, c["window"], c["sinks"])
        n = pkv.pkv_window_ws_bytes(lc.desc, batch, c["window"], c["sinks"], h["split"])
        h["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None
    if c["op"] == "rope":
        h["rope"] = pkv.make_rope(s["inv_freq"], interleaved=c["interleaved"], scale=s["factor"], positions=s["positions"])
        h["out"] = torch.empty((s["T"], c["hq"], c["dim"]), dtype=torch.bfloat16, device="cuda")
    if c["op"] == "gather" or (c["op"] == "rope" and c["int8"]):
        t = torch.float32 if c["fp32"] else torch.bfloat16
        h["rows"] = [torch.empty((s["T"], c["hkv"], c["dim"]), dtype=t, device="cuda") for _ in range(2)]
    return h


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        from paged_kv_cache_56_gb300 import pkv
        desc, batch = s["layer"].desc, s["batch"]
        if c["op"] == "window":
            pkv.pkv_window_attention(desc, batch, s["q"], s["out"], c["window"], c["sinks"], c["dim"] ** -0.5,
                                     s["split"], s["ws"])
            return s["out"]
        if c["op"] == "rope":
            pkv.pkv_rope_append(desc, batch, s["rope"], s["q"], s["k"], s["v"], s["out"])
            if not c["int8"]:
                return s["out"], s["k_pool"], s["v_pool"]
        pkv.pkv_gather_kv(desc, batch, *s["rows"])
        return tuple(s["rows"]) if c["op"] == "gather" else (s["out"], *s["rows"])
    if c["op"] == "window":
        return _plain_window(s)
    if c["op"] == "rope":
        out = _plain_rope(s)
        return (out, *_plain_gather(s)) if c["int8"] else (out, s["k_pool"], s["v_pool"])
    return _plain_gather(s)


def _rows(s):
    """Sequence and token of every row of the batch."""
    n = (s["starts"][1:] - s["starts"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n, output_size=s["T"])
    tok = (s["ctx"].long() - n - s["starts"][:-1].long())[seq] + torch.arange(s["T"], device="cuda")
    return seq, tok


def _cached(s, name, seq, tok):
    """Tokens `tok` of sequences `seq` from the K or V cache, fp32 [..., hkv, d]."""
    bs, kv = s["case"]["block"], "kv".index(name)
    block, off = s["tables"][seq, tok // bs].long(), tok % bs
    x = s[name + "_pool"][block, :, off].float()
    if not s["case"]["int8"]:
        return x
    x = x * s["scales"][block, :, kv].unsqueeze(-1)
    tail = s[name + "_tail"][s["slots"][seq].long(), :, off].float()
    return torch.where((tok >= s["ctx"][seq] // bs * bs)[..., None, None], tail, x)


def _plain_gather(s):
    t = torch.float32 if s["case"]["fp32"] else torch.bfloat16
    return tuple(_cached(s, name, *_rows(s)).to(t) for name in "kv")


def _plain_window(s):
    c = s["case"]
    B, hq, hkv, d, window, sinks = c["batch"], c["hq"], c["hkv"], c["dim"], c["window"], c["sinks"]
    G, most, ctx = hq // hkv, max(s["new"]), s["ctx"].long()
    seq, tok = _rows(s)
    n = (s["starts"][1:] - s["starts"][:-1]).long()
    # the keys that a sequence's tokens can see: the sinks, then one stretch up to its end
    lo = (ctx - n - window + 1).clamp(min=sinks) if window > 0 else torch.zeros_like(ctx)
    first = sinks if window > 0 else 0
    j = torch.arange(first + s["keys"], device="cuda")
    key = torch.where(j < first, j, lo[:, None] + j - first)
    there = key < ctx[:, None]
    key = key.minimum(ctx[:, None] - 1)
    every = torch.arange(B, device="cuda")[:, None].expand_as(key)
    k, v = (_cached(s, name, every, key).permute(0, 2, 1, 3) for name in "kv")
    local = torch.arange(s["T"], device="cuda") - s["starts"].long()[seq]
    q = torch.zeros((B, most, hq, d), device="cuda")
    q[seq, local] = s["q"].float()
    q = q.view(B, most, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * most, d)
    score = (q @ k.transpose(2, 3)).mul_(d ** -0.5).view(B, hkv, G, most, -1)
    at = (ctx - n)[:, None, None] + torch.arange(most, device="cuda")[:, None]
    see = there[:, None] & (key[:, None] <= at)
    if window > 0:
        see &= (at - key[:, None] < window) | (key[:, None] < sinks)
    score.masked_fill_(~see[:, None, None], -math.inf)
    score.sub_(score.amax(dim=-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = score.sum(dim=-1, keepdim=True)
    out = (score.view(B, hkv, G * most, -1) @ v).view(B, hkv, G, most, d) / total
    return out.permute(0, 3, 1, 2, 4).reshape(B, most, hq, d)[seq, local].to(torch.bfloat16)


def _turn(x, cos, sin, interleaved):
    """x [T, H, d] fp32, its first 2 * cos.shape[1] elements turned."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    u, w = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, w], dim=-1).flatten(-2) if interleaved else torch.cat([u, w], dim=-1)
    return torch.cat([y, x[..., 2 * half:]], dim=-1).to(torch.bfloat16)


def _plain_rope(s):
    c = s["case"]
    bs = c["block"]
    seq, tok = _rows(s)
    pos = s["positions"] if s["positions"] is not None else tok
    angle = pos.double()[:, None] * s["inv_freq"]
    cos, sin = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
    out = _turn(s["q"].float(), cos, sin, c["interleaved"])
    rows = {"k": _turn(s["k"].float(), cos, sin, c["interleaved"]), "v": s["v"]}
    if not c["int8"]:
        block = s["tables"][seq, tok // bs].long()
        s["k_pool"][block, :, tok % bs] = rows["k"]
        s["v_pool"][block, :, tok % bs] = rows["v"]
        return out
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
    for kv, name in enumerate("kv"):
        x = torch.where(fresh, rows[name][row].transpose(1, 2), s[name + "_tail"][slots[b]])
        y = x.float()
        top = y.abs().amax(dim=(2, 3), keepdim=True)
        scale = torch.where(top < 1e-6, torch.ones_like(top), top / 127)
        code = torch.round(y / scale).clamp(-127, 127).to(torch.int8)
        s[name + "_pool"][ids] = torch.where(full, code, s[name + "_pool"][ids])
        s["scales"][ids, :, kv] = torch.where(full, scale, s["scales"][ids, :, kv, None, None])[:, :, 0, 0]
        s[name + "_tail"][slots] = torch.where(full[last], s[name + "_tail"][slots], x[last])
    return out


# ---------------------------------------------------------------------------
# In 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _history(s, name, b, upto):
    """Tokens 0 .. upto-1 of sequence b, fp64 [upto, hkv, d], block by block of its table."""
    c, bs = s["case"], s["case"]["block"]
    ids = s["tables"][b, :-(-upto // bs)].long()
    x = s[name + "_pool"].index_select(0, ids).double()
    if c["int8"]:
        x = x * s["scales"].index_select(0, ids)[:, :, "kv".index(name), None, None].double()
        if s["ctx_host"][b] // bs < ids.numel():
            x[-1] = s[name + "_tail"][int(s["slots"][b])].double()
    return x.transpose(1, 2).reshape(-1, c["hkv"], c["dim"])[:upto]


def _exact_window(s):
    c = s["case"]
    G, window, sinks = c["hq"] // c["hkv"], c["window"], c["sinks"]
    out, at = [], 0
    for b, (n, ctx) in enumerate(zip(s["new"], s["ctx_host"])):
        k, v = _history(s, "k", b, ctx), _history(s, "v", b, ctx)
        for i in range(0, n, 512):
            m = min(512, n - i)
            p = torch.arange(ctx - n + i, ctx - n + i + m, device="cuda")[:, None]
            t = torch.arange(int(p[-1]) + 1, device="cuda")
            if window > 0:  # leave out what none of these tokens sees
                t = t[(t < sinks) | (t > int(p[0]) - window)]
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


def _exact_turn(x, s):
    c, rows = s["case"], []
    at = 0
    for n, ctx in zip(s["new"], s["ctx_host"]):
        p = torch.arange(ctx - n, ctx, device="cuda", dtype=torch.float64) + c["far"]
        z = torch.polar(torch.full_like(p[:, None] * s["inv_freq"], s["factor"]), p[:, None] * s["inv_freq"])
        y = x[at:at + n].double().clone()
        half = c["rotary"] // 2
        i = torch.arange(half, device="cuda")
        first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        turned = torch.complex(y[:, :, first], y[:, :, second]) * z[:, None]
        y[:, :, first], y[:, :, second] = turned.real, turned.imag
        rows.append(y)
        at += n
    return torch.cat(rows)


def _exact_rope(s):
    c, bs = s["case"], s["case"]["block"]
    rows = {"k": _exact_turn(s["k"], s), "v": s["v"].double()}
    result = [_exact_turn(s["q"], s)]
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


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "window":
        return _exact_window(s)
    if case["op"] == "rope":
        return _exact_rope(s)
    return tuple(torch.cat([_history(s, name, b, c)[c - n:] for b, (n, c) in enumerate(zip(s["new"], s["ctx_host"]))])
                 for name in "kv")
