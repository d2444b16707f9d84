"""Windowed attention after a wait that ran out (the library's test hook leaves
one copy unissued): the call reports it and returns, and the next one on the same
workspace is right."""

import pytest
import torch

from chunk_ref import Setup, assert_attention, attention
from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv

pytestmark = pytest.mark.gpu

COUNTERS = 16384 * 4  # bytes of arrival counters in front of a workspace


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("new,ctx,heads,split", [
    ([1, 3], [700, 900], (4, 2, 64), 0),           # few rows, whole
    ([1, 3], [700, 900], (4, 2, 64), 64),          # ... in splits
    ([40], [300], (8, 2, 128), 0),                 # many rows, whole
    ([300], [3000], (16, 8, 64), 256),             # ... 24 row tiles in 12 splits: two for each SM
    ([300], [1500], (8, 2, 128), 128),
])
def test_the_call_after_a_wait_that_ran_out_is_right(new, ctx, heads, split, int8):
    s = Setup(17, new, ctx, heads, 16, int8)
    desc, scale = s.lc.desc, s.d ** -0.5
    n = pkv.pkv_window_ws_bytes(desc, s.batch, 0, 0, split)
    assert (n > 0) == (split > 0)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None
    q, out = s.q.cuda(), torch.empty((s.T, s.hq, s.d), dtype=torch.bfloat16, device="cuda")
    pkv.pkv_debug_skip_copy(0)
    try:
        pkv.pkv_window_attention(desc, s.batch, q, out, 0, 0, scale, split, ws)
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_sync_status([desc])
        assert e.value.code == pkv.PKV_ERR_DEVICE_TIMEOUT
    finally:
        pkv.pkv_debug_skip_copy(-1)
    assert ws is None or not ws[:COUNTERS].any()
    ref, mag = attention(s, 0, 0)
    for _ in range(2):
        out.fill_(7.0)
        pkv.pkv_window_attention(desc, s.batch, q, out, 0, 0, scale, split, ws)
        assert pkv.pkv_sync_status([desc]) == 0
        assert_attention(out, ref, mag)
    assert ws is None or not ws[:COUNTERS].any()
