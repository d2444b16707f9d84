"""Calls of the GPU plans, axis positions, multi-axis append and prompt attention
that cannot be right are refused before any launch; descriptor layouts."""

import ctypes
import math
import os
import re

import pytest
import torch

from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv
from test_chunk_host import INT8, batch, desc, ref

BAD = pkv.PKV_ERR_INVALID


@pytest.fixture(scope="module")
def L():
    return ensure_built()


def pool(**kw):
    d = dict(tables=16, lens=16, held=16, ring=16, state=16, err_word=None, max_slots=4, max_blocks=8, num_blocks=20,
             block_size=16, int8=0)
    d.update(kw)
    return pkv.SeqPool(**d)


def plan(**kw):
    d = dict(token_starts=16, block_tables=16, ctx_lens=16, fill_blocks=None, block_ids=None, offsets=None, token_slots=None,
             positions=None, num_tokens=8, max_tokens=4)
    d.update(kw)
    return pkv.PlanDesc(**d)


def calls(L, p="p", slots=16, B=2, o="o"):
    p, o = pool() if p == "p" else p, plan() if o == "o" else o
    return (L.pkv_plan_batch(ref(p), slots, None, B, ref(o), None), L.pkv_commit_batch(ref(p), slots, None, B, ref(o), None),
            L.pkv_release_batch(ref(p), slots, B, None))


@pytest.mark.parametrize("p,code", [
    (None, BAD), (pool(tables=None), BAD), (pool(lens=None), BAD), (pool(held=None), BAD), (pool(ring=None), BAD),
    (pool(state=None), BAD), (pool(tables=18), BAD), (pool(lens=18), BAD), (pool(held=17), BAD), (pool(ring=18), BAD),
    (pool(state=18), BAD), (pool(err_word=18), BAD), (pool(max_slots=0), BAD), (pool(max_blocks=0), BAD),
    (pool(num_blocks=0), BAD), (pool(max_blocks=1 << 27), BAD), (pool(block_size=32), pkv.PKV_ERR_UNSUPPORTED),
    (pool(max_slots=65537), pkv.PKV_ERR_UNSUPPORTED),
])
def test_pools_are_checked(L, p, code):
    assert calls(L, p) == (code,) * 3


def test_plan_arguments(L):
    assert calls(L, B=-1) == (BAD,) * 3 and calls(L, B=65536) == (BAD,) * 3
    assert calls(L, slots=None) == (BAD,) * 3 and calls(L, slots=18) == (BAD,) * 3
    assert calls(L, B=0, slots=None) == (pkv.PKV_OK,) * 3
    assert calls(L, o=None)[:2] == (BAD,) * 2
    for kw in (dict(token_starts=None), dict(ctx_lens=None), dict(token_starts=18), dict(ctx_lens=18)):
        assert calls(L, o=plan(**kw))[:2] == (BAD,) * 2
    for kw in (dict(block_tables=None), dict(block_tables=18), dict(fill_blocks=18), dict(block_ids=18), dict(offsets=18),
               dict(token_slots=18), dict(positions=18), dict(num_tokens=-1), dict(max_tokens=-1), dict(max_tokens=9),
               dict(num_tokens=0x7FFF0000)):
        assert calls(L, o=plan(**kw))[0] == BAD
    assert L.pkv_plan_batch(ref(pool()), 16, 18, 2, ref(plan()), None) == BAD
    assert L.pkv_commit_batch(ref(pool()), 16, 18, 2, ref(plan()), None) == BAD


def positions(L, b="b", segs=16, num=16, R=2, S=3, rows=None, out=16, stride=8, err=None):
    return L.pkv_axis_positions(ref(batch() if b == "b" else b), segs, num, R, S, rows, out, stride, err, None)


def test_position_arguments(L):
    for b in (None, batch(B=-1), batch(B=65536), batch(num_tokens=-1), batch(max_tokens=-1), batch(max_tokens=9),
              batch(token_starts=None), batch(ctx_lens=None), batch(ctx_lens=18)):
        assert positions(L, b) == BAD
    for kw in (dict(segs=None), dict(segs=8), dict(num=None), dict(num=18), dict(R=-1), dict(S=-1), dict(R=0), dict(R=1),
               dict(rows=18), dict(out=None), dict(out=18), dict(stride=7), dict(err=18)):
        assert positions(L, **kw) == BAD, kw
    assert positions(L, batch(B=0), num=None) == pkv.PKV_OK and positions(L, batch(num_tokens=0, max_tokens=0)) == pkv.PKV_OK


def axes(L, c="d", b="b", r=None, q=16, qs=512, k=16, ks=256, v=16, vs=256, o=32, os_=512, ko=None, kos=256):
    c, b = desc() if c == "d" else c, batch() if b == "b" else b
    return L.pkv_rope_append_axes(ref(c), ref(b), ref(r), q, qs, k, ks, v, vs, o, os_, ko, kos, None)


def test_multi_axis_append_arguments(L):
    def r(pairs=(), **kw):
        d = dict(inv_freq=16, positions=None, axis_stride=8, num_axes=3, rotary_dim=64, interleaved=0, scale=1.0)
        d.update(kw)
        return pkv.RopeAxesDesc(**d, pair_axis=(ctypes.c_uint8 * 64)(*pairs))
    assert axes(L, None) == BAD and axes(L, b=None) == BAD and axes(L, desc(**INT8)) == BAD
    assert axes(L, r=r(rotary_dim=24)) == pkv.PKV_ERR_UNSUPPORTED
    assert axes(L, r=r(rotary_dim=144)) == BAD and axes(L, r=r(rotary_dim=-16)) == BAD
    assert axes(L, r=r(inv_freq=None)) == BAD and axes(L, r=r(inv_freq=12)) == BAD
    assert axes(L, r=r(positions=18)) == BAD and axes(L, r=r(scale=math.nan)) == BAD
    assert axes(L, r=r(num_axes=0)) == BAD and axes(L, r=r(num_axes=5)) == BAD
    assert axes(L, r=r([0, 1, 2, 3])) == BAD                     # a pair on an axis that there is not
    assert axes(L, r=r(positions=16, axis_stride=7)) == BAD
    assert axes(L, k=None) == BAD and axes(L, v=None) == BAD and axes(L, k=24) == BAD and axes(L, o=None) == BAD
    assert axes(L, ks=255) == BAD and axes(L, vs=128) == BAD and axes(L, qs=504) == BAD and axes(L, os_=516) == BAD
    assert axes(L, ko=24) == BAD and axes(L, ko=48, kos=248) == BAD and axes(L, ko=48, kos=260) == BAD
    assert axes(L, q=16, o=16, os_=1024) == BAD and axes(L, k=48, ko=48, kos=512) == BAD  # in place with another stride
    assert axes(L, b=batch(B=0)) == pkv.PKV_OK


def prompt(L, c="d", b="b", q=16, qs=512, k=32, ks=256, v=48, vs=256, w=8, s=2, scale=0.1, o=64, os_=512):
    c, b = desc() if c == "d" else c, batch() if b == "b" else b
    return L.pkv_prompt_attention(ref(c), ref(b), q, qs, k, ks, v, vs, w, s, scale, o, os_, None)


def test_prompt_arguments(L):
    assert prompt(L, None) == BAD and prompt(L, b=None) == BAD and prompt(L, desc(head_dim=96)) == pkv.PKV_ERR_UNSUPPORTED
    assert prompt(L, desc(num_q_heads=6)) == pkv.PKV_ERR_UNSUPPORTED
    for kw in (dict(w=-1), dict(s=-1), dict(scale=math.nan), dict(scale=math.inf), dict(scale=-0.5), dict(q=None), dict(k=None),
               dict(v=None), dict(o=None), dict(q=24), dict(k=24), dict(v=24), dict(o=24), dict(qs=504), dict(ks=248),
               dict(vs=248), dict(os_=504), dict(qs=516), dict(ks=260), dict(vs=260), dict(os_=516),
               dict(q=64, o=64, os_=1024)):
        assert prompt(L, **kw) == BAD, kw
    huge = batch(num_tokens=(1 << 25) + 1, max_tokens=(1 << 25) + 1)
    assert prompt(L, b=huge) == pkv.PKV_ERR_UNSUPPORTED
    assert prompt(L, b=batch(B=0)) == pkv.PKV_OK and prompt(L, b=batch(num_tokens=0, max_tokens=0)) == pkv.PKV_OK


def test_layouts_match_the_header():
    assert ctypes.sizeof(pkv.SeqPool) == 6 * 8 + 5 * 4 + 4  # (padded)
    assert ctypes.sizeof(pkv.PlanDesc) == 8 * 8 + 2 * 4
    assert ctypes.sizeof(pkv.RopeAxesDesc) == 3 * 8 + 4 * 4 + 64
    src = open(os.path.join(os.path.dirname(pkv.__file__), "..", "include", "pkv.h")).read()
    for name in ("PKV_DEVERR_OOM", "PKV_DEVERR_SEGMENT", "PKV_DEVERR_BATCH"):
        assert int(re.search(rf"#define\s+{name}\s+(\d+)", src).group(1)) == getattr(pkv, name)


def test_binding_checks():
    i = torch.zeros(8, dtype=torch.int32)
    f = torch.zeros(4, dtype=torch.float64)
    for call in (lambda: pkv.make_seq_pool(i, i, i, i, i, block_size=16),
                 lambda: pkv.make_seq_pool(i.view(2, 4), i, i, i, i, block_size=16),     # not on a GPU
                 lambda: pkv.make_plan(i, i, i, num_tokens=4, max_tokens=4),
                 lambda: pkv.make_plan(i, i.view(2, 4), i[:2], num_tokens=4, max_tokens=4),
                 lambda: pkv.make_rope_axes(f, [0, 1, 2]), lambda: pkv.make_rope_axes(f, [0, 1, 2, -1]),
                 lambda: pkv.make_rope_axes(f, [0, 1, 2, 0]),
                 lambda: pkv.make_rope_axes(torch.zeros(65, dtype=torch.float64), [0] * 65),
                 lambda: pkv.pkv_axis_positions(batch(), i, i, i)):
        with pytest.raises(ValueError):
            call()
    p, o = pool(), plan()
    p.device = o.device = torch.device("cuda", 0)
    o.B, o.width = 2, 8
    for slots in (i[:3], i[:2]):  # a plan for another batch; not on the pool's device
        for call in (pkv.pkv_plan_batch, pkv.pkv_commit_batch):
            with pytest.raises(ValueError):
                call(p, slots, o)
    with pytest.raises(ValueError):
        pkv.pkv_release_batch(p, i)
    o.width = 7
    with pytest.raises(ValueError, match="blocks"):
        pkv.pkv_plan_batch(p, i[:2], o)
