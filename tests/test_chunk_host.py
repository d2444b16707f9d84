"""The chunk operators on the host: refusals that come before any CUDA call,
descriptor layouts, the binding's checks, chunk plans and rotary frequencies,
and the kernels' integer steps restated."""

import ctypes
import math
import random
import re
import os
from fractions import Fraction

import numpy as np
import pytest
import torch

from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv
from paged_kv_cache_56_gb300.runtime import PagedKVCache, rope_frequencies

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_56_gb300", "csrc")


@pytest.fixture(scope="module")
def L():
    return ensure_built()


def desc(**kw):
    d = dict(k_pool=16, v_pool=32, scales=None, k_tail=None, v_tail=None, num_blocks=4, num_q_heads=4,
             num_kv_heads=2, head_dim=128, block_size=16, max_slots=0, dtype=pkv.PKV_DTYPE_BF16, err_word=None)
    d.update(kw)
    return pkv.CacheDesc(**d)


def batch(**kw):
    d = dict(token_starts=16, block_tables=16, ctx_lens=16, slots=None, B=2, max_blocks=4, num_tokens=8, max_tokens=4)
    d.update(kw)
    return pkv.BatchDesc(**d)


def ref(x):
    return None if x is None else ctypes.byref(x)


def rope(L, c="d", b="b", r=None, q=16, qs=512, k=16, ks=256, v=16, vs=256, o=32, os_=512):
    c, b = desc() if c == "d" else c, batch() if b == "b" else b
    return L.pkv_rope_append(ref(c), ref(b), ref(r), q, qs, k, ks, v, vs, o, os_, None)


def window(L, c="d", b="b", q=16, qs=512, w=8, s=2, scale=0.1, split=0, ws=None, n=0, o=32, os_=512):
    c, b = desc() if c == "d" else c, batch() if b == "b" else b
    return L.pkv_window_attention(ref(c), ref(b), q, qs, w, s, scale, split, ws, n, o, os_, None)


def gather(L, c="d", b="b", first=None, k=16, v=16, s=256, t=0):
    c, b = desc() if c == "d" else c, batch() if b == "b" else b
    return L.pkv_gather_kv(ref(c), ref(b), first, k, v, s, t, None)


INT8 = dict(dtype=pkv.PKV_DTYPE_INT8, scales=16, k_tail=16, v_tail=16, max_slots=2)


@pytest.mark.parametrize("call", [rope, window, gather])
@pytest.mark.parametrize("c,b,code", [
    (None, "b", pkv.PKV_ERR_INVALID), ("d", None, pkv.PKV_ERR_INVALID),
    (desc(head_dim=96), "b", pkv.PKV_ERR_UNSUPPORTED), (desc(block_size=32), "b", pkv.PKV_ERR_UNSUPPORTED),
    (desc(num_q_heads=6, num_kv_heads=2), "b", pkv.PKV_ERR_UNSUPPORTED), (desc(k_pool=24), "b", pkv.PKV_ERR_INVALID),
    ("d", batch(B=-1), pkv.PKV_ERR_INVALID), ("d", batch(num_tokens=-1), pkv.PKV_ERR_INVALID),
    ("d", batch(max_tokens=-1), pkv.PKV_ERR_INVALID), ("d", batch(max_tokens=9), pkv.PKV_ERR_INVALID),
    ("d", batch(B=70000), pkv.PKV_ERR_INVALID), ("d", batch(max_blocks=0), pkv.PKV_ERR_INVALID),
    ("d", batch(max_blocks=1 << 27), pkv.PKV_ERR_INVALID),  # 2^31 tokens
    ("d", batch(token_starts=None), pkv.PKV_ERR_INVALID), ("d", batch(block_tables=None), pkv.PKV_ERR_INVALID),
    ("d", batch(ctx_lens=None), pkv.PKV_ERR_INVALID), ("d", batch(ctx_lens=18), pkv.PKV_ERR_INVALID),
    (desc(**INT8), "b", pkv.PKV_ERR_INVALID),               # INT8 without slots
    ("d", batch(B=0), pkv.PKV_OK), ("d", batch(num_tokens=0, max_tokens=0), pkv.PKV_OK),
])
def test_descriptors_are_checked(L, call, c, b, code):
    assert call(L, c, b) == code


def test_rope_append_arguments(L):
    bad = pkv.PKV_ERR_INVALID
    r = lambda **kw: pkv.RopeDesc(**{**dict(inv_freq=16, positions=None, rotary_dim=64, interleaved=0, scale=1.0), **kw})  # noqa: E731
    assert rope(L, r=r(rotary_dim=24)) == pkv.PKV_ERR_UNSUPPORTED
    assert rope(L, r=r(rotary_dim=144)) == bad and rope(L, r=r(rotary_dim=-16)) == bad
    assert rope(L, r=r(inv_freq=None)) == bad and rope(L, r=r(inv_freq=12)) == bad
    assert rope(L, r=r(positions=18)) == bad and rope(L, r=r(scale=math.nan)) == bad
    assert rope(L, k=None) == bad and rope(L, v=None) == bad and rope(L, k=24) == bad
    assert rope(L, o=None) == bad and rope(L, q=24) == bad
    assert rope(L, ks=255) == bad and rope(L, ks=260) == bad and rope(L, vs=128) == bad
    assert rope(L, qs=504) == bad and rope(L, os_=516) == bad
    assert rope(L, q=16, o=16, qs=512, os_=1024) == bad  # in place with another stride


def test_window_arguments(L):
    bad = pkv.PKV_ERR_INVALID
    assert window(L, w=-1) == bad and window(L, s=-1) == bad and window(L, split=-16) == bad and window(L, split=24) == bad
    for scale in (math.nan, math.inf, -0.5):
        assert window(L, scale=scale) == bad
    assert window(L, q=None) == bad and window(L, o=None) == bad and window(L, q=24) == bad and window(L, o=40) == bad
    assert window(L, qs=504) == bad and window(L, os_=508) == bad
    assert L.pkv_window_split_tokens(ref(desc()), ref(batch()), -1, 0) == bad
    assert L.pkv_window_split_tokens(None, ref(batch()), 0, 0) == bad
    assert L.pkv_window_split_tokens(ref(desc()), ref(batch(B=0)), 0, 0) == 0
    assert L.pkv_window_ws_bytes(ref(desc()), ref(batch(B=0)), 0, 0, 16) == 0
    assert L.pkv_window_ws_bytes(None, None, 0, 0, 16) == 0


def test_gather_arguments(L):
    bad = pkv.PKV_ERR_INVALID
    assert gather(L, k=None) == bad and gather(L, v=24) == bad and gather(L, t=2) == bad
    assert gather(L, s=255) == bad and gather(L, s=260) == bad and gather(L, s=258, t=1) == bad and gather(L, first=18) == bad


def test_descriptor_layouts_match_the_header():
    assert ctypes.sizeof(pkv.BatchDesc) == 4 * 8 + 4 * 4
    assert ctypes.sizeof(pkv.RopeDesc) == 2 * 8 + 2 * 4 + 4 + 4  # (padded)
    src = open(os.path.join(CSRC, "..", "..", "include", "pkv.h")).read()
    for name in ("PKV_OUT_BF16", "PKV_OUT_FP32"):
        assert int(re.search(rf"#define\s+{name}\s+(\d+)", src).group(1)) == getattr(pkv, name)


def test_binding_checks():
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.make_batch(i, torch.zeros((2, 4), dtype=torch.int32), i[:2], num_tokens=2, max_tokens=1)
    with pytest.raises(ValueError):
        pkv.make_batch(i, i, i[:2], num_tokens=2, max_tokens=1)
    with pytest.raises(ValueError):
        pkv.make_rope(torch.zeros(32, dtype=torch.float64))
    b = batch()
    b.device, b.keep = torch.device("cuda", 0), None
    q = torch.zeros((8, 4, 128), dtype=torch.bfloat16)
    for call in (lambda: pkv.pkv_window_attention(desc(), b, q, q, 0, 0, 0.1),
                 lambda: pkv.pkv_rope_append(desc(), b, None, q, q[:, :2], q[:, :2]),
                 lambda: pkv.pkv_gather_kv(desc(), b, q[:, :2], q[:, :2]),
                 lambda: pkv.pkv_gather_kv(desc(), b, q[:, :2].half(), q[:, :2].half())):
        with pytest.raises(ValueError):
            call()
    b.device = torch.device("cpu")  # shapes, strides and types of rows
    for x in (q.float(), q[:4], q[:, :3], q[..., :64], q.transpose(0, 1), torch.zeros((8, 4, 256), dtype=torch.bfloat16)[..., ::2]):
        with pytest.raises(ValueError):
            pkv._rows(x, "q", b, 4, 128)
    assert pkv._rows(q, "q", b, 4, 128)[1] == 512
    wide = torch.zeros((8, 9, 128), dtype=torch.bfloat16)
    assert pkv._rows(wide[:, 2:6], "q", b, 4, 128) == (wide.data_ptr() + 2 * 256, 9 * 128)
    b.num_tokens = 1
    assert pkv._rows(q[:1], "q", b, 4, 128)[1] == 512


# ---------------------------------------------------------------------------
# Plans
# ---------------------------------------------------------------------------

def make_cache(L, blocks=16, bs=16, int8=False, **kw):
    return PagedKVCache(1, blocks, 4, 2, 64, bs, int8, max_slots=4, max_blocks_per_seq=8, device="cpu", **kw)


def test_plan_chunk_grows_block_lists(L):
    c = make_cache(L)
    for r in (1, 2, 3):
        c.add_sequence(r)
    p = c.plan_chunk([1, 2, 3], [20, 0, 16])
    assert p.starts.tolist() == [0, 20, 20, 36] and p.ctx_lens.tolist() == [20, 0, 16]
    assert [len(c.table(r)) for r in (1, 2, 3)] == [2, 0, 1]
    c.commit_chunk([1, 2, 3], [20, 0, 16])
    p = c.plan_chunk([3, 1], [1, 12])
    assert p.ctx_lens.tolist() == [17, 32] and [len(c.table(r)) for r in (1, 3)] == [2, 2]
    assert p.tables[0, :2].tolist() == c.table(3) and p.tables[1, :2].tolist() == c.table(1)
    c.close()


def test_plan_chunk_is_all_or_nothing(L):
    c = make_cache(L, blocks=5)
    c.add_sequence(1)
    c.add_sequence(2)
    with pytest.raises(pkv.PkvError) as e:
        c.plan_chunk([1, 2], [48, 48])
    assert e.value.code == pkv.PKV_ERR_OOM and c.table(1) == [] and c.table(2) == [] and pkv.pkv_num_free(c.alloc) == 5
    for counts in ([1], [-1, 2], [200, 1]):
        with pytest.raises(ValueError):
            c.plan_chunk([1, 2], counts)
    with pytest.raises(ValueError):
        c.plan_chunk([1, 1], [1, 1])
    c.close()


def test_plan_chunk_copies_a_shared_block_before_writing(L):
    c = make_cache(L)
    c.add_sequence(1)
    c.plan_chunk([1], [20])
    c.commit_chunk([1], [20])
    c.fork(1, 2)
    t = c.table(1)
    p = c.plan_chunk([1, 2], [3, 40])
    assert len(p.cow) == 1 and c.table(1)[0] == t[0] == c.table(2)[0] and c.table(1)[1] != c.table(2)[1]
    c.commit_chunk([1, 2], [3, 40])
    assert not c.plan_chunk([1, 2], [1, 1]).cow
    c.close()


def test_rope_frequencies():
    f, a = rope_frequencies(64, 10000.0)
    assert a == 1.0 and np.allclose(f, [10000.0 ** (-2 * j / 64) for j in range(32)], rtol=1e-15)
    g, a = rope_frequencies(64, 10000.0, stretch=4)
    assert a == 1.0 and np.array_equal(g, f / 4)
    g, a = rope_frequencies(64, 10000.0, stretch=4, trained=4096)
    turns = 4096 * f / (2 * math.pi)
    assert math.isclose(a, 0.1 * math.log(4) + 1)
    assert np.array_equal(g[turns >= 32], f[turns >= 32]) and np.allclose(g[turns <= 1], f[turns <= 1] / 4)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (g[mid] < f[mid]).all() and (g[mid] > f[mid] / 4).all()
    for bad in (dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=64, stretch=0.5),
                dict(rotary_dim=64, short_turns=1, long_turns=1)):
        with pytest.raises(ValueError):
            rope_frequencies(**bad)


# ---------------------------------------------------------------------------
# The kernels' integer steps, restated
# ---------------------------------------------------------------------------

TWO_PI = 2 * Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286, 10 ** 75)


def turns_of(f):
    """turns_of() of the rotary kernel in Python integers."""
    bits = int(np.float64(f).view(np.uint64))
    e = (bits >> 52) & 0x7FF
    if e == 0:
        return 0
    m = ((bits << 11) | 1 << 63) & (1 << 64) - 1
    prod, right = m * 0x28BE60DB9391054A, 1086 - e
    u = (prod >> right if right >= 0 else prod << -right) & (1 << 64) - 1 if right < 128 else 0
    return (1 << 64) - u & (1 << 64) - 1 if bits >> 63 else u


def test_frequency_in_turns():
    rng = random.Random(5)
    values = [1.0, 0.5, 1e-4, 10000.0 ** -0.984375, 3.25, 100.0, 0.0, -1.0, 2.0 ** -60]
    values += [math.exp(rng.uniform(math.log(1e-7), math.log(2.0))) for _ in range(200)]
    for f in values:
        want = Fraction(np.float64(f).item()) / TWO_PI
        diff = (Fraction(turns_of(f), 2 ** 64) - want) % 1
        diff = min(diff, 1 - diff)
        # 1 / 2 pi is cut to 64 bits (2^-64 for each radian), the result to 2^-64
        assert diff <= Fraction(1, 2 ** 63) * (1 + Fraction(abs(f))), f
        for pos in (1, 12345, 10 ** 6, 2 ** 31 - 1):  # 32 bits of the angle
            top = (turns_of(f) * pos % 2 ** 64) >> 32
            d = (Fraction(top, 2 ** 32) - want * pos) % 1
            assert min(d, 1 - d) <= Fraction(1, 2 ** 32) + Fraction(pos, 2 ** 63) * (1 + Fraction(abs(f)))


def key_tiles(p_first, p_last, window, sinks, unit):
    lo = max(0, p_first - window + 1)
    s = min(sinks, lo)
    lo_t, ns = lo // unit, -(-s // unit)
    if ns >= lo_t and s > 0:
        ns = lo_t = 0
    n = ns + p_last // unit - lo_t + 1
    return [k if k < ns else k - ns + lo_t for k in range(n)]


def test_key_tiles_are_the_visible_ones():
    rng = random.Random(7)
    for _ in range(3000):
        unit = rng.choice([16, 64])
        a = rng.randrange(0, 700)
        b = a + rng.randrange(0, 130)
        window, sinks = rng.choice([0x7FFFFFFF, rng.randrange(1, 400)]), rng.randrange(0, 200)
        sinks = 0 if window == 0x7FFFFFFF else sinks
        got = key_tiles(a, b, window, sinks, unit)
        seen = {t // unit for p in range(a, b + 1) for t in range(p + 1) if p - t < window or t < sinks}
        assert got == sorted(set(got)) and seen <= set(got)
        # no more than the sinks' units and one stretch up to the end
        assert set(got) <= {t // unit for t in range(sinks)} | set(range(max(0, a - window + 1) // unit, b // unit + 1))


def test_converted_tile_is_whole_and_without_bank_conflicts():
    """Where the INT8 loader's threads store a tile's 16-byte pieces (128-byte rows in slabs, chunks swizzled by row)."""
    for d in (64, 128):
        cpr = d // 16
        step = 128 // cpr
        seen = {}
        for k in range(128 * cpr // 128):
            for half in range(2):
                for warp in range(4):
                    phases = [[], [], [], []]
                    for lane in range(32):
                        c = (lane & 3) + ((lane >> 3) & 1) * 4 if d == 128 else lane & 3
                        row0 = warp * (32 // cpr) + (((lane >> 2) & 1) + (lane >> 4) * 2 if d == 128 else lane >> 2)
                        ca, sw = (2 * c) % 8 + half, row0 & 7
                        at = (c // 4) * 16384 + row0 * 128 + ((ca ^ sw) << 4) + k * step * 128
                        row, dim = row0 + k * step, c * 16 + half * 8
                        assert at == (dim // 64) * 16384 + row * 128 + ((((dim % 64) // 8) ^ (row & 7)) << 4)
                        assert (row, dim) not in seen
                        seen[row, dim] = at
                        phases[lane // 8].append(at % 128)
                    assert all(len(set(p)) == 8 for p in phases)  # eight threads, all 32 banks
        assert len(seen) == 128 * d // 8


def test_int8_codes_as_bf16():
    """(0x4300 | m) - (0x4300 | s << 7) in bf16 is the code of bits s:m."""
    def bf16(bits):
        return torch.tensor([bits << 16], dtype=torch.int32).view(torch.float32).item()
    for x in range(-128, 128):
        byte = x & 0xFF
        t = 0x4300 | byte
        assert bf16(t & 0xFF7F) - bf16(t & 0xFF80) == x


def test_division_steps_of_the_quantizer():
    """The rotary append's quotient: x * inv, corrected twice by fused multiply-adds, equals the rounded quotient for
    every pair of significands (fp32 emulated exactly in integers)."""
    def rn(v):  # Fraction -> nearest fp32 (ties to even), as a Fraction
        if v == 0:
            return Fraction(0)
        s, v = (-1, -v) if v < 0 else (1, v)
        e = v.numerator.bit_length() - v.denominator.bit_length()
        e -= Fraction(2) ** e > v
        unit = Fraction(2) ** (e - 23)
        n, r = divmod(v, unit)
        n += r * 2 > unit or (r * 2 == unit and n % 2 == 1)
        return s * n * unit
    rng = random.Random(3)
    for top in list(range(128, 256, 9)) + [128, 129, 255]:
        scale = rn(Fraction(top) / 127)
        inv = rn(1 / scale)
        for x in [rng.randrange(128, top + 1) if top > 128 else 128 for _ in range(25)]:
            for e in (0, -1, -3, -7):
                f = Fraction(x) * Fraction(2) ** e
                q = rn(f * inv)
                for _ in range(2):
                    q = rn(rn(f - q * scale) * inv + q)
                assert q == rn(f / scale)


def test_everything_of_a_call_is_on_one_device():
    b = batch()
    b.device, b.keep = torch.device("cpu"), None
    q = torch.zeros((8, 4, 128), dtype=torch.bfloat16)
    r = pkv.RopeDesc()
    r.device, r.num_positions = torch.device("cuda", 1), None
    for call in (lambda: pkv.pkv_rope_append(desc(), b, r, None, q[:, :2], q[:, :2]),
                 lambda: pkv.pkv_gather_kv(desc(), b, q[:, :2], q[:, :2], torch.zeros(2, dtype=torch.int32, device="meta")),
                 lambda: pkv.pkv_window_attention(desc(), b, q, q, 0, 0, 0.1, 0, torch.zeros(8, device="meta"))):
        with pytest.raises(ValueError):
            call()
