"""Slots of one sealing call that share pools: what the host can see to write one place twice is refused
(no device needed: validation precedes launches)."""
import pytest

import invariant_sequence_decode_gb300 as luce
from test_q8kv_refusals import E, M, P, lib, seal, slot  # noqa: F401


def two(first, second):
    """Two slots of the same pools with tails of their own."""
    return [slot(**first), slot(k=P + 8 * M, v=P + 9 * M, **second)]


@pytest.mark.parametrize("first,second", [
    (dict(), dict()),
    (dict(sealed=0, length=64), dict(sealed=32)),                                  # 0 .. 63 and 32 .. 63
    (dict(sealed=96), dict(sealed=64, length=64)),
    (dict(sealed=0, length=63), dict(sealed=0, length=35)),
    (dict(table=P + 10 * M), dict(table=P + 10 * M)),                              # one table for both
    (dict(), dict(vc=P + 11 * M, sc=P + 12 * M)),                                  # K's pool alone
    (dict(), dict(kc=P + 11 * M, sc=P + 12 * M)),
    (dict(), dict(kc=P + 11 * M, vc=P + 12 * M)),
])
def test_slots_that_would_write_the_same_blocks(lib, first, second):  # noqa: F811
    for slots in (two(first, second), two(second, first)):
        assert seal(lib, slots) == E and b"the same blocks" in lib.luce_last_error()


def test_slots_that_write_other_blocks_pass(lib):  # noqa: F811
    """(nothing is sealed where no slot has a whole block; what passes otherwise meets the check of a later slot)"""
    bad = slot(k=P + 13 * M, v=P + 14 * M, length=65)
    for first, second in ((dict(sealed=0), dict(sealed=32)), (dict(sealed=64), dict(sealed=0, length=64)),
                          (dict(), dict(length=31)), (dict(length=31), dict()), (dict(), dict(table=P + 10 * M)),
                          (dict(table=P + 10 * M), dict(table=P + 11 * M))):
        assert seal(lib, two(first, second) + [bad]) == E and b"slot 2 len=65" in lib.luce_last_error()
    assert seal(lib, two(dict(length=31), dict(length=31))) == luce.LUCE_OK
