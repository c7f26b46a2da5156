"""mrope_axes: every axis gets its pairs; a negative number of pairs is refused in both layouts (taking
axes in turn until none is left would never end)."""
import signal

import pytest

from asymmetric_kv_paged_gb300 import binding as B


@pytest.mark.parametrize("sections", [[8, 12, 12], [0, 5], [3, 0, 1, 2], [4], [0, 0]])
@pytest.mark.parametrize("in_turn", [False, True])
def test_every_axis_has_its_pairs(sections, in_turn):
    axes = B.mrope_axes(sections, in_turn=in_turn)
    assert [axes.count(a) for a in range(len(sections))] == sections


@pytest.mark.parametrize("sections", [[-1], [4, -2, 3], [3, -1]])
@pytest.mark.parametrize("in_turn", [False, True])
def test_negative_numbers_of_pairs_are_refused(sections, in_turn):
    def stop(*_):
        raise TimeoutError("mrope_axes does not end")

    before = signal.signal(signal.SIGALRM, stop)
    signal.alarm(2)
    try:
        with pytest.raises(ValueError):
            B.mrope_axes(sections, in_turn=in_turn)
    finally:
        signal.alarm(0)
        signal.signal(signal.SIGALRM, before)
