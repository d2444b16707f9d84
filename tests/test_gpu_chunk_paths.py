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
