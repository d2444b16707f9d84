"""Plans that need just the free blocks there are, or one more, with entries read once and twice."""

import pytest

from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv
from plan_ref import DevicePoolOf, PoolModel, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("B", [4, 511, 512, 513, 700, 1030])
@pytest.mark.parametrize("short", [0, 1])
def test_as_many_blocks_as_are_free_and_one_more(B, short):
    """17 tokens each take two blocks, 60 more take three: all are taken where they just fit, none where one
    is missing; then all again by a batch that needs one less."""
    N = 5 * B - short
    m = PoolModel(B + 2, 6, N, 16)
    g = DevicePoolOf(m, B, 60 * B, 60, head=N - 3)
    slots = list(range(B, 0, -1))

    def go(counts, bits):
        want = m.plan(slots, counts, 60 * B, 60)
        pkv.pkv_plan_batch(g.pool, dev(slots), g.plan_desc, dev(counts))
        assert g.error() == bits
        if bits:
            assert want == bits
            g.check_empty_plan()
        else:
            g.check_plan(want)
        g.check_state()
        pkv.pkv_commit_batch(g.pool, dev(slots), g.plan_desc)
        if not bits:
            m.commit(slots, counts, counts)
        assert g.error() == 0
        g.check_state()

    go([17] * B, 0)
    assert len(m.free) == 3 * B - short
    go([60] * B, pkv.PKV_DEVERR_OOM if short else 0)
    if short:
        go([60] * (B - 1) + [44], 0)
    assert not m.free
    go([3] * B, 0)  # 80 tokens fill their five blocks, 64 four
    go([0] * (B - 1) + [16], pkv.PKV_DEVERR_OOM)  # one more
    go([0] * B, 0)
