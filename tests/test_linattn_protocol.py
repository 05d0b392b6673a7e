"""The linear attention kernels' barrier hand-offs: none can deadlock, overrun or underrun, whatever the timing."""
import pytest

from linattn_protocol import state_protocol, tile_protocol

ITEMS = {
    "single": [[(1, False)]],
    "one segment": [[(j + 1, True)] for j in range(2)] * 3,
    "first segment, then others": [[(1, False)], [(2, False)], [(1, True)], [(2, True)], [(3, True)], [(4, True)]],
    "several z tiles": [[(2, True)] * 4, [(1, True)] * 4, [(1, False)] * 3, [(4, False)] * 2],
    "long": [[(1, True)]] * 9,
}


@pytest.mark.parametrize("items", ITEMS.values(), ids=ITEMS.keys())
@pytest.mark.parametrize("nslots,stages,nx", [(1, 10, 2), (1, 5, 2), (1, 4, 2), (2, 4, 1), (3, 3, 1), (4, 2, 1)])
def test_tile_kernel(items, nslots, stages, nx):
    assert tile_protocol(items, nslots, stages, nx).check() == []


def test_skipped_slots_are_rejected():
    """The earlier form: the warp of the scores skipped Z's slots, and could take the open phase of one for its next."""
    found = [tile_protocol(items, 4, 2, 1, z_relay=False).check() for items in ITEMS.values()]
    assert any(any("underrun" in p and "scores" in p for p in f) for f in found)


@pytest.mark.parametrize("stages,parts,accs", [(4, 2, 1), (6, 3, 2), (6, 2, 2)])
@pytest.mark.parametrize("segments", [[[1]], [[8, 8, 3]], [[4], [4], [1]], [[16, 16], [16, 5], [2]], [[1, 1, 1, 1]] * 3], ids=str)
@pytest.mark.parametrize("skip_last", [False, True])
def test_state_kernel(stages, parts, accs, segments, skip_last):
    assert state_protocol(segments, stages, parts, accs, skip_last).check() == []


def test_planted_defects_are_caught():
    # a ring of three stages: the two groups of weights would meet each other's phases
    assert state_protocol([[8, 8, 8]], 3, 2, 2).check()
