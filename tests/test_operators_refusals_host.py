"""Refusals of the operators around retention beyond test_operators_host.py: nothing is launched."""
from tests.test_operators_host import ALIGN, BASE, _rot, lib  # noqa: F401 - lib is a fixture


def test_rotary_tables_must_be_aligned(lib):
    for bad in (dict(freqs=3 * BASE + 4), dict(freqs=3 * BASE + 1), dict(positions=4 * BASE + 4),
                dict(starts=5 * BASE + 2)):
        assert _rot(lib, **bad) == ALIGN, bad
