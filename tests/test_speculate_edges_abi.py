"""CPU checks of the speculative step's C ABI: what a fork's output rows may share with the table."""
import ctypes
import random

import pytest
import torch

from tests.test_speculate_abi import F, INVALID, SPACE, WORKSPACE, lib  # noqa: F401

# Calls that are not refused go on to the device: with addresses that nobody owns, there must be none.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses, for machines without a device")


def _fork(lib, at, pitch, rows, width, P=8, B=4, M=6, table_pitch=6, space=F):  # noqa: F811
    """Output rows `at` entries behind the table's start."""
    base = 0x100000
    return lib.ets_pages_fork(F, P, ctypes.c_void_p(base), table_pitch, B, M, F, 8, F, rows, ctypes.c_void_p(base + 4 * at), pitch, width,
                              F, None, 0, space, SPACE, None)


def test_fork_refuses_rows_of_the_table(lib):  # noqa: F811
    meets = [dict(at=0, pitch=6, rows=4, width=6), dict(at=0, pitch=6, rows=1, width=1), dict(at=23, pitch=6, rows=2, width=6),
             dict(at=18, pitch=6, rows=3, width=6), dict(at=-5, pitch=6, rows=1, width=6), dict(at=-100, pitch=50, rows=9, width=6),
             dict(at=5, pitch=10, rows=2, width=2, table_pitch=10), dict(at=9, pitch=10, rows=3, width=3, table_pitch=10),
             dict(at=30, pitch=7, rows=2, width=4, table_pitch=20, B=3), dict(at=17, pitch=1000, rows=1, width=4, table_pitch=20)]
    apart = [dict(at=24, pitch=6, rows=4, width=6), dict(at=-12, pitch=6, rows=2, width=6), dict(at=6, pitch=12, rows=4, width=6, table_pitch=12),
             dict(at=6, pitch=10, rows=3, width=4, table_pitch=10), dict(at=7, pitch=30, rows=2, width=8, table_pitch=15),
             dict(at=-6, pitch=24, rows=3, width=6, table_pitch=12, B=1), dict(at=-6, pitch=12, rows=40, width=6, table_pitch=24, B=9),
             dict(at=0, pitch=6, rows=4, width=0), dict(at=0, pitch=6, rows=4, width=6, B=0), dict(at=0, pitch=6, rows=4, width=6, M=0)]
    for case in meets:
        assert _brute(**case), case
        assert _fork(lib, **case) == INVALID, case
    for case in apart:  # past the checks of arguments; there is no device here
        assert not _brute(**case), case
        assert _fork(lib, **case) not in (0, INVALID, WORKSPACE), case
    assert _fork(lib, 0, 6, 0, 6) == 0 and _fork(lib, 0, 6, 4, 6, space=None) == WORKSPACE


def _brute(at, pitch, rows, width, B=4, M=6, table_pitch=6):
    mine = {b * table_pitch + j for b in range(B) for j in range(M)}
    return any(at + i * pitch + j in mine for i in range(rows) for j in range(width))


def test_fork_overlap_follows_the_entries(lib):  # noqa: F811
    r = random.Random(5)
    seen = set()
    for _ in range(3000):
        case = dict(at=r.randint(-60, 80), rows=r.randint(1, 6), width=r.randint(1, 8), B=r.randint(1, 6), M=r.randint(1, 8))
        case.update(pitch=case["width"] + r.randint(0, 12), table_pitch=case["M"] + r.randint(0, 12))
        meets = _brute(**case)
        assert (_fork(lib, **case) == INVALID) == meets, case
        seen.add(meets)
    assert seen == {True, False}
