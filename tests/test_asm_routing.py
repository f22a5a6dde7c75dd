"""The kernels of the routing to experts and of 4-bit integer weights in gfx950 assembly: none spills
to scratch memory, and none uses the packed fp32 instructions that the build turns off.

CPU only: hipcc cross-compiles for gfx950 without a GPU."""
import os
import shutil
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_asm_scratch import ROOT, assemble, kernels

sys.path.insert(0, os.path.join(ROOT, "swiglu_gemm_amd"))

UNITS = ["api_routing.hip", "api_int4.hip"] + \
    ["inst_int4_%s_%s.hip" % (d, z) for d in ("f16", "bf16") for z in ("zeros", "sym")]


@pytest.fixture(scope="module")
def asm_files(tmp_path_factory):
    import build
    if shutil.which(build.hipcc()) is None and not os.path.exists(build.hipcc()):
        pytest.skip("hipcc not available")
    d = str(tmp_path_factory.mktemp("asm_routing"))
    with ThreadPoolExecutor(len(UNITS)) as ex:
        return dict(zip(UNITS, ex.map(lambda u: assemble(build, u, d), UNITS)))


@pytest.mark.parametrize("unit", UNITS)
def test_kernels_do_not_spill(asm_files, unit):
    found = list(kernels(asm_files[unit]))
    assert len(found) >= 20, unit
    bad = [(name, size) for name, size in found if size]
    assert not bad, "scratch: %s" % bad[:3]


@pytest.mark.parametrize("unit", UNITS)
def test_no_packed_fp32(asm_files, unit):
    text = open(asm_files[unit]).read()
    assert not [op for op in ("add", "mul", "fma") if "v_pk_%s_f32" % op in text]
