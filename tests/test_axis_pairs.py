"""Host parts of positions on several axes and of the GPU's pools."""

from types import SimpleNamespace

import pytest
import torch

from paged_kv_cache_56_gb300.runtime import AxisPositions, axis_pairs


def test_axis_pairs():
    assert axis_pairs((2, 1, 3)) == [0, 0, 1, 2, 2, 2]
    assert axis_pairs((2, 1, 3), in_turn=True) == [0, 1, 2, 0, 2, 2]
    assert axis_pairs([24, 20, 20], in_turn=True) == [0, 1, 2] * 20 + [0] * 4
    assert axis_pairs((0, 2)) == [1, 1] and axis_pairs((4,)) == [0] * 4 and axis_pairs((1, 1, 1, 1), True) == [0, 1, 2, 3]
    for bad in ((), (1, 1, 1, 1, 1), (2, -1)):
        with pytest.raises(ValueError):
            axis_pairs(bad)


def test_segments_are_checked():
    cache = SimpleNamespace(device="cpu", max_slots=3, seqs={5: SimpleNamespace(slot=2)})
    a = AxisPositions(cache, 10, 3)
    a.set(5, [(4, 0, 0, 1), (1, 2, 3, 1)])
    assert a.counts.tolist() == [0, 0, 2] and a.segments[2, :2].tolist() == [[4, 0, 0, 1], [1, 2, 3, 1]]
    a.set(5, [])
    assert a.counts.tolist() == [0, 0, 0]
    for bad in ([(1, 0, 0, 1)] * 4, [(-1, 0, 0, 1)], [(1, 2, 0, 1)], [(1, 0, 2, 1)], [(1, 1, 1, -1)], [(2 ** 31, 0, 0, 1)],
                [(2, 2 ** 16, 2 ** 15, 1)], [(3, 1, 1, 2 ** 30)]):
        with pytest.raises(ValueError):
            a.set(5, bad)
    assert a.positions.shape == (3, 10) and a.positions.dtype == torch.int32
