"""More refusals of the windowed / paged calls and of the page calls, found on
the host before anything is enqueued (no GPU, device pointers that nothing reads)."""

import ctypes

import pytest

from test_view_refusals import INVALID, WS, ALIGNMENT, B, _pool, _table  # noqa: F401  (B is the fixture)


def test_granted_must_not_meet_lengths_or_add(B):
    L = B.load()
    a = B.tq_pages_reserve_args(_pool(B), _table(B), 0x5000, 0x6000, 0, None, 0x7000)
    for at, status in ((0x5008, INVALID), (0x5ff8, INVALID), (0x6002, ALIGNMENT)):
        a.granted = at
        assert L.tq_pages_reserve(ctypes.byref(a), WS, 1 << 40, None) == status
