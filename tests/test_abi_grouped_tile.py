"""The control of the grouped products' tiles refuses what there is no kernel for, on the host."""
import ctypes

import pytest

OK, INVALID = 0, 1


@pytest.fixture()
def control():
    import __graft_entry__
    f = ctypes.CDLL(__graft_entry__._build_module().build()).gdn_debug_set_grouped_tile
    f.argtypes = [ctypes.c_int32, ctypes.c_int32]
    yield f
    assert f(0, -1) == OK


@pytest.mark.parametrize("want,rows,cut", [(OK, 0, -1), (OK, 16, -1), (OK, 16, 3), (OK, 32, 0), (OK, 64, 2), (OK, 128, 3), (OK, 256, 0),
                                           (OK, 256, -1), (INVALID, 256, 1), (INVALID, 0, 0), (INVALID, 8, 0), (INVALID, 100, -1),
                                           (INVALID, 16, 4), (INVALID, 16, -2), (INVALID, -16, 0), (INVALID, 65552, 0)])
def test_tiles(control, want, rows, cut):
    assert control(rows, cut) == want
