"""Lengths beyond what the kernels number in 32 bits are refused (CPU: nothing is enqueued)."""
import ctypes
import re

from tests.test_decode_abi import HEADER, INVALID, _scores, lib  # noqa: F401

MAX_LENGTH = 0x7FFFF000


def test_lengths_beyond_the_limit_are_refused(lib):  # noqa: F811
    from exact_top_selection_amd import _decode
    assert int(re.search(r"#define ETS_MAX_LENGTH (0x[0-9a-f]+)", open(HEADER).read()).group(1), 16) == MAX_LENGTH == _decode.MAX_LENGTH
    need = ctypes.c_size_t(0)
    good = dict(B=1, T=1, Hq=4, Hkv=2, D=64, Dv=64, dtype=0, K=8, L=8, page_size=1 << 30, S=16)
    for L in (MAX_LENGTH + 1, 0x7FFFFFFF):
        assert _scores(lib, B=1, page=1 << 30, L=L, stride=L) == INVALID
        for form in (dict(L=L), dict(K=L, slots=0x1000)):
            args = _decode._AttendArgs(**{**good, **form})
            assert lib.ets_attend_workspace_size(ctypes.byref(args), ctypes.byref(need)) == INVALID, form
