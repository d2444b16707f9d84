"""A batch over one layer's cache with known contents, and the chunk operators
from their definitions in fp64 (CPU, plain loops over sequences).

What must not be read is poisoned: rows behind a context, blocks that no
sequence holds and, where asked, blocks before a window hold NaN (INT8: NaN
scales), and table entries that must not be looked up are -1."""

from __future__ import annotations

import math

import numpy as np
import torch

from oracle.quantize import quantize_block
from paged_kv_cache_56_gb300 import pkv
from paged_kv_cache_56_gb300.runtime import LayerCache

NAN = float("nan")


def bf16(x):
    return torch.as_tensor(np.asarray(x)).to(torch.bfloat16)


def quantize_heads(x):
    """Codes and scales of one block's rows [hkv, bs, d], head by head."""
    parts = [quantize_block(h) for h in x.float().numpy()]
    return np.stack([q for q, _ in parts]), np.array([sc for _, sc in parts], np.float32)


class Setup:
    """Sequences of contexts `ctx` of which the last `new` tokens are new. The
    cache holds tokens 0 .. filled-1 of each (filled: ctx, or ctx - new for a
    test that appends)."""

    def __init__(self, seed, new, ctx, heads, bs, int8, appended=True, kv_mult=1.0, hidden=None, spare_slots=1):
        g = torch.Generator().manual_seed(seed)
        self.new, self.ctx, self.bs, self.int8 = list(new), list(ctx), bs, int8
        self.hq, self.hkv, self.d = heads
        self.B, self.T = len(new), sum(new)
        self.G = self.hq // self.hkv
        blocks = [-(-c // bs) for c in ctx]
        self.num_blocks = sum(blocks) + 3
        self.width = max(max(blocks), 1) + 1
        ids = torch.randperm(self.num_blocks, generator=g).tolist()
        self.table = np.full((self.B, self.width), -1, np.int32)
        for b, n in enumerate(blocks):
            self.table[b, :n] = [ids.pop() for _ in range(n)]
        self.starts = np.cumsum([0] + self.new).astype(np.int32)
        self.slots = torch.randperm(self.B + spare_slots, generator=g)[:self.B].numpy().astype(np.int32)
        self.lc = LayerCache(self.num_blocks, self.hq, self.hkv, self.d, bs, int8, self.B + spare_slots)

        def normal(*shape):
            return torch.randn(shape, generator=g)

        self.rows = {n: [bf16(normal(c, self.hkv, self.d) * kv_mult) for c in ctx] for n in "kv"}
        self.q = bf16(normal(self.T, self.hq, self.d))
        self.held = [c if appended else c - n for n, c in zip(new, ctx)]
        self.values = {n: [] for n in "kv"}  # fp64 [held, hkv, d]: what the cache stands for
        self.codes = {}
        for kv, n in enumerate("kv"):
            pool = torch.full((self.num_blocks, self.hkv, bs, self.d), 127 if int8 else NAN,
                              dtype=torch.int8 if int8 else torch.bfloat16)
            tail = torch.full((self.B + spare_slots, self.hkv, bs, self.d), NAN, dtype=torch.bfloat16)
            scales = torch.full((self.num_blocks, self.hkv), NAN)
            for b in range(self.B):
                h = self.held[b]
                val = self.rows[n][b][:h].double().numpy().copy()
                for i in range(-(-h // bs)):
                    lo, hi = i * bs, min(h, (i + 1) * bs)
                    x = self.rows[n][b][lo:hi].transpose(0, 1)  # [hkv, rows, d]
                    if not int8:
                        pool[self.table[b, i], :, :hi - lo] = x
                    elif hi - lo < bs:
                        tail[self.slots[b], :, :hi - lo] = x
                    else:
                        code, sc = quantize_heads(x)
                        pool[self.table[b, i]] = torch.as_tensor(code)
                        scales[self.table[b, i]] = torch.as_tensor(sc)
                        val[lo:hi] = (code.astype(np.float64) * sc.astype(np.float64)[:, None, None]).transpose(1, 0, 2)
                self.values[n].append(val)
            getattr(self.lc, n + "_pool").copy_(pool)
            if int8:
                getattr(self.lc, n + "_tail").copy_(tail)
                self.lc.scales[:, :, kv].copy_(scales)
        if hidden:  # hide(b, block) -> True: the block must not be looked up
            for b in range(self.B):
                for i in range(blocks[b]):
                    if hidden(b, i):
                        old = int(self.table[b, i])
                        self.table[b, i] = -1
                        if int8:
                            self.lc.scales[old] = NAN
                        else:
                            self.lc.k_pool[old] = NAN
                            self.lc.v_pool[old] = NAN
        dev = lambda a: torch.as_tensor(np.asarray(a, np.int32)).cuda()  # noqa: E731
        self.d_starts, self.d_table, self.d_ctx, self.d_slots = dev(self.starts), dev(self.table), dev(ctx), dev(self.slots)
        self.batch = pkv.make_batch(self.d_starts, self.d_table, self.d_ctx, self.d_slots if int8 else None,
                                    num_tokens=self.T, max_tokens=max(self.new + [0]))

    def new_rows(self, name):
        """The new tokens' rows [T, hkv, d] bf16."""
        parts = [r[c - n:] for r, n, c in zip(self.rows[name], self.new, self.ctx)]
        return torch.cat(parts) if parts else torch.zeros((0, self.hkv, self.d), dtype=torch.bfloat16)

    def error_bits(self):
        return self.lc.error_bits()


def attention(s: Setup, window, sinks, sm_scale=None, values=None):
    """(output, sum of weights times |v|) fp64 [T, hq, d] from the definition.

    INT8: a weight times its block's V scale is held in f16, in units in which a
    weight of 1 times the largest V scale of the tile's blocks is at least 2^14
    (the decode kernel's range design). Its rounding is then at most half of
    f16's smallest step, 2^-25, where it is below f16's normal range: 2^-39 of
    the largest V scale for each token, times a code of at most 127, over a sum
    of weights of at least 1. With 2^-8 of the magnitude allowed, 2^-30 of the
    largest |v| of the head for each token holds that and is added to it."""
    sm_scale = 1 / math.sqrt(s.d) if sm_scale is None else sm_scale
    out = np.zeros((s.T, s.hq, s.d))
    mag = np.zeros_like(out)
    q = s.q.double().numpy()
    for b in range(s.B):
        k, v = (s.values[n][b] if values is None else values[n][b] for n in "kv")
        for i in range(s.new[b]):
            p = s.ctx[b] - s.new[b] + i
            t = np.arange(p + 1)
            if window > 0:
                t = t[(p - t < window) | (t < sinks)]
            row = s.starts[b] + i
            kk, vv = k[t], v[t]                                  # [n, hkv, d]
            qq = q[row].reshape(s.hkv, s.G, s.d)
            x = np.einsum("hgd,thd->hgt", qq, kk) * sm_scale
            w = np.exp(x - x.max(axis=-1, keepdims=True))
            w /= w.sum(axis=-1, keepdims=True)
            out[row] = np.einsum("hgt,thd->hgd", w, vv).reshape(s.hq, s.d)
            mag[row] = np.einsum("hgt,thd->hgd", w, np.abs(vv)).reshape(s.hq, s.d)
            if s.int8:
                top = np.abs(v).max(axis=(0, 2))  # [hkv]
                mag[row] += np.repeat(top, s.G)[:, None] * (t.size * 2.0 ** -30)
    return out, mag


def assert_attention(got, ref, mag, what=""):
    """The result is rounded to bf16 (half a step: 2^-8 of it) and each weight to
    bf16 at worst before it meets V (2^-8 of what it adds to); scores, exponentials
    and sums are fp32: an error of a score of size up to 2^6 is 2^-18 and so is
    the relative error of its weight -- 2^-12 of the magnitude holds all of it."""
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all(), f"{what}: {np.argwhere(~np.isfinite(got))[:3].tolist()} not finite"
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * mag + 1e-30
    bad = np.abs(got - ref) > tol
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; first at {i}: {got[i]!r} against {ref[i]!r}, "
                             f"tolerance {tol[i]!r}")


def turned(x, pos, inv_freq, interleaved, scale):
    """Rows x [T, H, d] (bf16) turned, fp64."""
    y = x.double().numpy().copy()
    half = len(inv_freq)
    a = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = (np.cos(a) * scale)[:, None], (np.sin(a) * scale)[:, None]
    i = np.arange(half)
    f, g = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    u, w = y[:, :, f].copy(), y[:, :, g].copy()
    y[:, :, f], y[:, :, g] = u * c - w * s, w * c + u * s
    return y
