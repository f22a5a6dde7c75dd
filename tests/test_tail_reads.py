"""What the grouped kernels load behind K: rows of no expert and gaps between the experts'
matrices are not theirs.  A host program includes the kernels' own header, asks its
tail_readable() for small problems and checks every element that the tile would load.

CPU only: the header's host side, built by hipcc."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "swiglu_gemm_amd"))


def test_a_whole_last_tile_stays_in_the_experts_rows_and_matrices(tmp_path):
    import build
    if shutil.which(build.hipcc()) is None and not os.path.exists(build.hipcc()):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "tail_driver")
    src = os.path.join(ROOT, "tests", "sanitize", "tail_driver.hip")
    r = subprocess.run([build.hipcc(), "--offload-host-only", "-O1", "-std=c++17", "-w", "-I",
                        build.INCLUDE, "-I", build.CSRC, src, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr
    print(r.stdout)
