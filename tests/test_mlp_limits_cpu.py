"""Largest sizes of rows in 8 bits, on the host alone: whatever trellis_swiglu keeps,
trellis_restore takes back. A call whose sizes are right fails at its null pointers."""
import ctypes as C

import pytest

from test_mlp_cpu import T  # noqa: F401 (the fixture)

WIDTH = 16384


def statuses(T, rows, width):
    none, stream = C.c_void_p(0), C.c_void_p(0)
    raw = T.raw()
    return {"keep": raw.trellis_keep(none, rows, width, None, stream),
            "restore": raw.trellis_restore(None, rows, width, none, stream),
            "swiglu": raw.trellis_swiglu(none, rows // 2, width, none, None, stream),
            "gradient": raw.trellis_swiglu_backward(none, none, None, rows // 2, width, none, none, stream)}


@pytest.mark.parametrize("rows,width", [((1 << 35) // WIDTH, WIDTH), ((1 << 35) // 131072, 131072 - 31),
                                        (1 << 22, 8192), (1 << 22, 8161), (131072, 1 << 18)])
def test_what_is_kept_can_be_restored(T, rows, width):  # noqa: F811
    assert set(statuses(T, rows, width).values()) == {T.ERR_NULL}


@pytest.mark.parametrize("rows,width", [((1 << 35) // WIDTH + 2, WIDTH), ((1 << 35) // 131072, 131072 + 1),
                                        (1 << 22, 8193), ((1 << 22) + 2, 32), (131074, 1 << 18)])
def test_beyond_is_refused(T, rows, width):  # noqa: F811
    assert set(statuses(T, rows, width).values()) == {T.ERR_GEOMETRY}
