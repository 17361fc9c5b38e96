"""The build stops where a kernel whose warpgroups trade registers got fewer than they share (no GPU needed)."""
import os

import pytest

from quantized_moe_decode_luce_gb300 import build as B

SRC = "linear_w4_tc.cu"
with open(os.path.join(B.CSRC, SRC)) as f:
    TEXT = f.read()


def log(*kernels):
    return "ptxas info    : 9 bytes gmem\n" + "".join(
        f"ptxas info    : Compiling entry function '{name}' for 'sm_103a'\nptxas info    : Function properties for {name}\n"
        f"    0 bytes stack frame\nptxas info    : Used {regs} registers, used 2 barriers\n" for name, regs in kernels)


def kernel(mode):
    return f"_ZN48_GLOBAL__N__b6e132bf_15_linear_w4_tc_cu_1dd6e08c14k_linear_w4_tcILi{mode}ELi2ELi1EEEvNS_6TcArgsE"


def test_enough_registers():
    B.check_registers(SRC, TEXT, log((kernel(0), 72), (kernel(1), 80), ("_Z5other", 8), (kernel(2), 80), (kernel(3), 168)))


@pytest.mark.parametrize("mode,regs", [(0, 64), (1, 71), (2, 72), (3, 79)])
def test_too_few_registers(mode, regs):
    with pytest.raises(RuntimeError, match=f"has {regs} registers"):
        B.check_registers(SRC, TEXT, log((kernel(0), 72), (kernel(mode), regs)))


def test_registers_that_nothing_told():
    with pytest.raises(RuntimeError, match="told no kernel"):
        B.check_registers(SRC, TEXT, log(("_Z5other", 200)))
