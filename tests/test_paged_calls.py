"""Refusals of the calls of rotary positions and the 8-bit paged cache that
depend on how several arguments go together, and sizes the host computes: no GPU
is needed."""
import ctypes

import pytest

from test_paged_refusals import BASE, INVALID, append, attend, lib, pages  # noqa: F401


# ------------------------------------------------------------- table slices
def append_cols(lib, stride, width, n=4):
    return lib.pcd_k_kv_append_cols(ctypes.byref(pages()), BASE, BASE, 3, 128, 64, 128, 64, BASE, BASE, BASE, 2, n, stride, width,
                                    BASE, 64, 0, 1.0, None, None, None)


def attend_cols(lib, stride, width, n=4):
    return lib.pcd_k_paged_attention_cols(ctypes.byref(pages()), BASE, 2 * BASE, None, 3, 4, 256, 64, 256, 64, BASE, BASE, BASE,
                                          2, n, stride, width, 64, 1, 0.125, None, 0, None, None)


@pytest.mark.parametrize("stride,width", [(4, 5), (4, -1), (-1, -1), (0, 1), (-4, 0)])
def test_table_slices_refused(lib, stride, width):  # noqa: F811
    for call in (append_cols, attend_cols):
        assert call(lib, stride, width) == INVALID and lib.pcd_last_error()
        assert call(lib, 4, 3, n=0) == 0
