"""Registers that the kernels' hand-counted loads rely on, without a GPU: the
built library's device code, and the sources' inline assembly.

A load written in inline assembly gives the compiler its registers at once.  Where
the wait is not in the same block, the compiler may put an instruction on such a
register between the two; and where loads in flight are counted by hand
(s_waitcnt vmcnt(n)), a spilled register's load or store would be counted too."""

import os
import re
import shutil
import subprocess

import pytest

_lib = pytest.importorskip("newton_schulz_dmuon_amd")._lib
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "newton_schulz_dmuon_amd", "csrc")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{kernel: [instruction, ...]} of the library."""
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    tmp = str(tmp_path_factory.mktemp("code"))
    shutil.copy(_lib.LIB_PATH, os.path.join(tmp, "lib.so"))
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp, check=True, capture_output=True)
    out = {}
    for name in sorted(os.listdir(tmp)):
        if not name.endswith("gfx950"):
            continue
        text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", name], cwd=tmp, check=True, capture_output=True,
                              text=True).stdout
        body = None
        for line in text.splitlines():
            head = re.match(r"^[0-9a-f]+ <(\S+)>:", line)
            if head:
                body = out.setdefault(head.group(1), [])
            elif body is not None and line.startswith("\t"):
                body.append(line.split("//")[0].strip())
    assert any("q8_wgrad_kernel" in k for k in out) and any("ns_gemm_kernel" in k for k in out)
    return out


def vector_registers(text):
    regs = set()
    for lo, hi, one in re.findall(r"\bv(?:\[(\d+):(\d+)\]|(\d+)\b)", text):
        regs.update(range(int(lo), int(hi) + 1) if lo else [int(one)])
    return regs


def test_no_register_is_touched_before_its_read_has_landed(kernels):
    reads = 0
    for name, body in kernels.items():
        pending = set()
        for i, ins in enumerate(body):
            op, _, operands = ins.partition(" ")
            if op == "s_waitcnt" and "lgkmcnt(0)" in operands:
                pending.clear()
                continue
            assert not pending or not op.startswith(("s_cbranch", "s_branch", "s_endpgm", "s_setpc")), (name, i, ins)
            assert not vector_registers(operands) & pending, (name, i, ins, body[i - 8:i])
            if op == "ds_read_b64_tr_b16":
                pending |= vector_registers(operands.split(",")[0])
                reads += 1
    assert reads > 0


def test_no_kernel_spills(kernels):
    spilled = {name for name, body in kernels.items() if any(ins.startswith("scratch_") for ins in body)}
    assert not spilled


def test_inline_loads_of_the_8_bit_products_wait_in_their_block():
    loads = re.compile(r"\b(ds_read|ds_load|global_load|buffer_load|flat_load)\w*\s+%\d")
    seen = 0
    for name in sorted(os.listdir(CSRC)):
        if not name.startswith("q8_"):
            continue
        source = open(os.path.join(CSRC, name)).read()
        for block in re.findall(r"asm volatile\((.*?)\);", source, re.S):
            if loads.search(block):
                seen += 1
                assert re.search(r"s_waitcnt (lgkmcnt|vmcnt)\(0\)", block), (name, block[:80])
                assert '"=v"' not in block, (name, "an output may share an address's register")
    assert seen == 2
