"""The grouped and 4-bit kernels in gfx950 assembly, as test_asm_m0.py and test_asm_scratch.py look
at the others: nothing but the asm statements uses M0, each write of it waits one state before the
LDS load that reads it (16 bytes a lane, or the 4 of a scale), and no kernel spills to scratch
memory.

CPU only: hipcc cross-compiles for gfx950 without a GPU."""
import os
import re
import shutil
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_asm_m0 import IMPLICIT_M0, NAMES_M0, ROOT, assemble, instructions
from test_asm_scratch import kernels

sys.path.insert(0, os.path.join(ROOT, "swiglu_gemm_amd"))

# unit: its ring kernels, and whether it has the scales' loads
UNITS = {"inst_grouped_bf16.hip": ("grouped_dma_kernel", 26, False),
         "inst_grouped_f16.hip": ("grouped_dma_kernel", 26, False),
         "inst_grouped_e4m3.hip": ("grouped_dma_kernel", 9, False),
         "inst_mx4.hip": ("mx_dma_kernel", 20, True)}
LDS_LOAD = re.compile(r"global_load_lds_dword(x4)? v\d+, s\[\d+:\d+\]$")


@pytest.fixture(scope="module")
def asm_files(tmp_path_factory):
    import build
    if shutil.which(build.hipcc()) is None and not os.path.exists(build.hipcc()):
        pytest.skip("hipcc not available")
    d = str(tmp_path_factory.mktemp("asm_experts"))
    with ThreadPoolExecutor(len(UNITS)) as ex:
        return dict(zip(UNITS, ex.map(lambda u: assemble(build, u, d), UNITS)))


@pytest.mark.parametrize("unit", sorted(UNITS))
def test_compiler_never_uses_m0(asm_files, unit):
    bad = [s for inside, s in instructions(asm_files[unit])
           if not inside and (NAMES_M0.search(s) or IMPLICIT_M0.match(s))]
    assert not bad, "%s: compiler-generated M0 use: %s" % (unit, bad[:5])


@pytest.mark.parametrize("unit", sorted(UNITS))
def test_each_m0_write_waits_one_state_before_the_load(asm_files, unit):
    ins = list(instructions(asm_files[unit]))
    widths = {"": 0, "x4": 0}
    for i, (inside, s) in enumerate(ins):
        if inside and NAMES_M0.search(s):
            assert re.match(r"s_mov_b32 m0, s\d+$", s), s
            assert ins[i + 1] == (True, "s_nop 0"), ins[i + 1]
            m = LDS_LOAD.match(ins[i + 2][1])
            assert ins[i + 2][0] and m, ins[i + 2]
            widths[m.group(1) or ""] += 1
    assert widths["x4"] > 100
    assert (widths[""] > 20) == UNITS[unit][2], widths


@pytest.mark.parametrize("unit", sorted(UNITS))
def test_kernels_do_not_spill(asm_files, unit):
    kind, count, _ = UNITS[unit]
    found = list(kernels(asm_files[unit]))
    assert sum(kind in name for name, _ in found) == count
    bad = [(name, size) for name, size in found if size]
    assert not bad, "scratch: %s" % bad[:3]
