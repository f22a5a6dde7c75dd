"""Host-side AddressSanitizer + UndefinedBehaviorSanitizer run of the grouped and 4-bit operators'
C ABI (swiglu_gemm_amd/csrc/api_experts.hip): argument checks, the choice of tiles and the sizes
of launches, which tests/sanitize/experts_driver.hip's stand-ins for the launchers look over.
CPU only: sanitizers on the host side of the compile, no kernel runs."""
import os

import pytest

from test_sanitizers import ENV, HIPCC, ROOT, SAN, run


def test_experts_abi_under_asan_ubsan(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    csrc = os.path.join(ROOT, "swiglu_gemm_amd", "csrc")
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-w",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-omit-frame-pointer",
             "-I", os.path.join(ROOT, "include"), "-I", csrc]
    objs = []
    for src in (os.path.join(csrc, "api_experts.hip"), os.path.join(SAN, "experts_driver.hip")):
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        run([HIPCC] + flags + ["-c", src, "-o", objs[-1]])
    exe = str(tmp_path / "experts_san")
    run([HIPCC, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address",
         "-Xarch_host", "-fsanitize=undefined"] + objs + ["-o", exe])
    r = run([exe], env=ENV, timeout=300)
    assert r.stdout.startswith("ok")
