"""Layouts of a state that engram_state_copy takes at its C entry, on the host: with n = 0 nothing is
launched and no address is looked at."""
import pytest

eng = pytest.importorskip("hashed_gram_memory_tid2eid_amd")


def layout_status(planes, plane_pitch, rows, row_pitch, row_bytes):
    return eng._lib.engram_state_copy(1 << 20, planes, plane_pitch, rows, row_pitch, row_bytes, None, None, 0, None)


def overlaps(planes, plane_pitch, rows, row_pitch, row_bytes):
    seen = set()
    for q in range(planes):
        for r in range(rows):
            at = set(range(q * plane_pitch + r * row_pitch, q * plane_pitch + r * row_pitch + row_bytes))
            if at & seen:
                return True
            seen |= at
    return False


def test_layouts_whose_rows_overlap_are_refused():
    """Every small layout; those that nest in neither order are refused without overlapping, too."""
    refused = 0
    for planes in (1, 2, 3):
        for rows in (1, 2, 4):
            for row_bytes in (1, 3, 8):
                for row_pitch in range(row_bytes, 30):
                    for plane_pitch in range(0, 70):
                        status = layout_status(planes, plane_pitch, rows, row_pitch, row_bytes)
                        nested = (plane_pitch >= (rows - 1) * row_pitch + row_bytes or
                                  plane_pitch >= row_bytes and row_pitch >= (planes - 1) * plane_pitch + row_bytes)
                        if planes == 1 or nested:
                            assert status == 0
                            assert not overlaps(planes, plane_pitch, rows, row_pitch, row_bytes)
                        else:
                            assert status == eng.ENGRAM_E_ARG
                            refused += 1
    assert refused


@pytest.mark.parametrize("layout, good", [
    ((2, 1 << 62, 1 << 20, 1 << 40, 4096), True),             # (their end is past 2^62)
    ((2, (1 << 60) - 1, 1 << 20, 1 << 40, 4096), True),       # (a plane ends at 2^60 - 2^40 + 4096)
    ((2, (1 << 60) - (1 << 40) + 4096, 1 << 20, 1 << 40, 4096), True),
    ((2, (1 << 60) - (1 << 40) + 4095, 1 << 20, 1 << 40, 4096), False),
    ((2, 1 << 60, 1 << 20, 1 << 40, 4096), True),
    ((1 << 20, 1 << 62, 1 << 30, 1 << 62, 4096), False),      # products past 2^63
    ((1 << 23, 4096, 1 << 30, 1 << 35, 4096), True), ((1 << 23, 4096, 1 << 30, (1 << 35) - 1, 4096), False),
    ((3, 0, 2, 64, 64), False), ((3, 0, 0, 64, 64), True), ((1, 0, 2, 64, 64), True), ((0, 0, 2, 64, 64), True),
    ((2, 63, 1, 64, 64), False), ((2, 64, 1, 64, 64), True),
])
def test_layouts_of_large_numbers(layout, good):
    assert layout_status(*layout) == (0 if good else eng.ENGRAM_E_ARG)
