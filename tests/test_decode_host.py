"""Host bookkeeping of the decode layer (no GPU needed): pages by lane, ancestor masks."""
import pytest

from resident_expert_routed_gb300.decode import LanePages, tree_mask


def test_pages_are_handed_out_and_returned():
    p = LanePages(2, 5, 16, 4)
    p.reserve(0, 17)
    p.reserve(1, 1)
    assert len(p.pages[0]) == 2 and len(p.pages[1]) == 1 and len(p.free) == 2
    assert p.table[0, :2].tolist() == p.pages[0] and p.table[0, 2:].tolist() == [-1, -1]
    slots = p.slots(0, 17)
    assert len(set(slots)) == 17 and slots[16] == p.pages[0][1] * 16
    p.advance(0, 16)
    p.reserve(0, 16)                                  # the second page was there already
    assert len(p.pages[0]) == 2 and p.slots(0, 1) == [p.pages[0][1] * 16]
    p.reserve(0, 17)
    with pytest.raises(MemoryError):
        p.reserve(1, 40)
    with pytest.raises(ValueError):
        p.reserve(0, 60)
    p.release(0)
    assert len(p.free) == 4 and p.rows[0] == 0 and p.table[0].tolist() == [-1] * 4
    assert sorted(p.free + p.pages[1]) == list(range(5))


def test_ancestor_masks():
    assert tree_mask([]) == []
    assert tree_mask([-1, 0, 0, 2]) == [0b1, 0b11, 0b101, 0b1101]
    assert tree_mask([-1, -1]) == [0b1, 0b10]
    for bad in ([0], [-1, 1], [-2]):
        with pytest.raises(ValueError):
            tree_mask(bad)
