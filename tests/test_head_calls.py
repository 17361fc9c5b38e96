"""How the int8 decode head is called and built, where no GPU is needed: host
checks of its entry points, the bindings and the call module."""
import ctypes

import pytest

from quantized_moe_decode_luce_gb300 import build as B

vp, ci, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(B.build())


def test_mask_rows_without_masks(lib):
    f = lib.luce_logits_process
    f.argtypes = [vp, ci, ci, i64, i64, vp, i64, vp, vp, vp, vp, vp, vp, vp, ci, vp, ci, i64, vp, vp, i64, vp]

    def call(mask, n_masks, mask_rows):  # (no rows: nothing is launched)
        return f(None, 0, 0, 64, 64, None, 0, None, None, None, None, None, None, None, 0, mask, n_masks, 2, mask_rows,
                 None, 64, None)
    assert call(None, 0, 0x10000) == 0 and call(None, 0, None) == 0
    assert call(None, 2, 0x10000) == 1  # masks that are not there
    assert call(0x20000, 0, 0x10000) == 1 and call(0x20000, 2, 0x10000) == 0
