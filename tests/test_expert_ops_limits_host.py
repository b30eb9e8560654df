"""Host-only checks of the separate expert operators at the ends of their
ranges: offsets, sizes and tensors that do not fit are cut or refused before a
kernel sees them (no GPU needed)."""
import ctypes
import itertools
import os

import pytest

from mixture_experts_layer_34_amd import mok

MIN, MAX = -2 ** 31, 2 ** 31 - 1


def _diag():
    return ctypes.CDLL(os.path.join(os.path.dirname(mok.LIB_PATH), "libmok_diag.so"))


@pytest.mark.parametrize("rows", [0, 1, 30, 1 << 24])
def test_offsets_are_cut_at_both_ends(rows):
    """Any two offsets give 0 <= begin <= end <= rows: the rows r with
    begin <= r < end of the offsets that lie in the buffer, none for a range
    that ends before it begins, however far apart the two are."""
    f, got = _diag().mok_diag_expert_rows, (ctypes.c_int32 * 2)()
    f.argtypes = [ctypes.c_int32] * 3 + [ctypes.c_void_p]
    ends = [MIN, MIN + 1, -(1 << 30), -50, -1, 0, 1, 2, 5, 29, 30, 31, rows - 1, rows, rows + 1, 1 << 30, MAX - 1, MAX]
    for lo, hi in itertools.product(ends, ends):
        assert f(lo, hi, rows, got) == 0
        begin, end = got
        assert 0 <= begin <= end <= rows
        want = (max(lo, 0), min(hi, rows))
        assert (begin, end) == want if want[0] < want[1] else begin == end, (lo, hi)
    assert f(0, 1, rows, None) == 1
