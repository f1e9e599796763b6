"""Numbers that the C structs' 32 bits do not hold (no GPU needed)."""

import pytest


@pytest.fixture
def limits():
    from recurrent_associative_memory_gb300 import attention
    return attention._limits


def test_a_window_wider_than_every_position_is_the_widest(limits):
    for window in (2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1):
        assert limits(window, 4, 7) == (2 ** 31 - 1, 4, 7)
    assert limits(1, 0) == (1, 0, 0) and limits(0, -1) == (0, -1, 0)   # refused by the call itself


@pytest.mark.parametrize("args", [(-2 ** 32 + 5, 0, 0), (8, 2 ** 32 + 4, 0), (8, -2 ** 32 + 4, 0),
                                  (8, 0, 2 ** 32), (8, 0, -2 ** 32 + 1)])
def test_others_are_refused(limits, args):
    with pytest.raises(ValueError, match="32 bits"):
        limits(*args)
