"""Axis positions where a sequence's list of segments goes on behind what its first
new tokens need, and segments that cannot be."""

import numpy as np
import pytest

from libpkv import ensure_built
from paged_kv_cache_56_gb300 import pkv
from plan_ref import dev
from test_gpu_axes import make, positions_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("at", [0, 250, 255, 256, 400, 511, 512, 599])
@pytest.mark.parametrize("bad", [(-1, 0, 0, 1), (1, 2, 0, 1), (2, 2, 2, -1)])
def test_bad_segments_far_behind_the_first_tokens_are_reported(at, bad):
    """600 segments of seven tokens: the first 1024 tokens end in the first 256 of them, the bad one stands anywhere."""
    segs = [(7, 0, 0, 1) if i % 2 else (1, 1, 7, 1) for i in range(600)]
    good = segs[:at] + segs[at + 1:]
    segs[at] = bad
    n = 7 * 599
    for new, ctx in ((n, n), (1, n), (1500, n + 3)):
        batch, table, count, out = make([segs, good], [new, new], [ctx, ctx])
        err = dev([0])
        pkv.pkv_axis_positions(batch, table, count, out, err=err)
        want = positions_of(good, ctx)[:, ctx - new:]  # it counts as empty
        assert np.array_equal(out[:, :2 * new].cpu().numpy(), np.tile(want, 2))
        assert err.item() == pkv.PKV_DEVERR_SEGMENT


@pytest.mark.parametrize("bad", [(4, 0, 0, -1), (1, 0, 0, -2 ** 31), (-3, 0, 0, -3)])
def test_text_with_a_negative_step_counts_as_empty(bad):
    """A segment with negative numbers is bad, whether the number would matter or not."""
    segs, good = [(3, 0, 0, 1), bad, (1, 2, 2, 0), (2, 0, 0, 0)], [(3, 0, 0, 1), (1, 2, 2, 0), (2, 0, 0, 0)]
    batch, table, count, out = make([segs, good], [11, 11], [11, 11])
    err = dev([0])
    pkv.pkv_axis_positions(batch, table, count, out, err=err)
    assert np.array_equal(out[:, :22].cpu().numpy(), np.tile(positions_of(good, 11), 2))
    assert err.item() == pkv.PKV_DEVERR_SEGMENT
    batch, table, count, out = make([good], [11], [11])
    err.zero_()
    pkv.pkv_axis_positions(batch, table, count, out, err=err)
    assert np.array_equal(out[:, :11].cpu().numpy(), positions_of(good, 11)) and err.item() == 0
