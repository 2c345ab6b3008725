"""The 4-bit products' kernels as built, without a GPU: their loads in flight are
counted by hand (s_waitcnt vmcnt(n)), so none may spill a register, whose load or
store would be counted too; and the sources load nothing in inline assembly."""

import os
import re

from test_kernel_registers import CSRC, kernels  # noqa: F401


def test_no_4_bit_kernel_spills(kernels):  # noqa: F811
    names = [n for n in kernels if re.search(r"q4_\w+_kernel", n)]
    for kind in ("q4_quantise_kernel", "q4_dequantise_kernel", "q4_stream_kernel", "q4_tile_kernel", "q4_mid_kernel",
                 "q4_rows_stream_kernel", "q4_rows_tile_kernel", "q4_rows_mid_kernel"):
        assert any(kind in n for n in names), kind
    assert not [n for n in names if any(ins.startswith("scratch_") for ins in kernels[n])]


def test_no_inline_loads():
    loads = re.compile(r"\b(ds_read|ds_load|global_load|buffer_load|flat_load)")
    for name in sorted(os.listdir(CSRC)):
        if name.startswith("q4_"):
            for block in re.findall(r"asm volatile\((.*?)\);", open(os.path.join(CSRC, name)).read(), re.S):
                assert not loads.search(block), (name, block[:80])
