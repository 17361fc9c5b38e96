"""How the int8 decode head is called and built, where no GPU is needed: host
checks of its entry points, the bindings and the call module."""
import ctypes

import pytest
import torch

from oracle import head as O
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


# ----------------------------------------------------------------------------- definitions
def test_a_row_of_zeros_has_scale_zero_without_an_epsilon():
    x = torch.zeros((2, 8))
    x[1, 3] = 4.0
    q, s, _ = O.rows_i8(x, torch.ones(8), 0.0)
    assert s[0] == 0 and torch.all(q[0] == 0) and q[1, 3] == 127
    assert abs(float(s[1]) * 127 - 8 ** 0.5) < 1e-6  # 4 / sqrt(16 / 8)
    q, s, _ = O.rows_i8(x, torch.zeros(8), 0.0)
    assert torch.all(s == 0) and torch.all(q == 0)
