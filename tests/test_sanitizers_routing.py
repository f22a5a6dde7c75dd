"""Host-side AddressSanitizer + UndefinedBehaviorSanitizer run of the C ABI of the routing to experts
and of 4-bit integer weights (swiglu_gemm_amd/csrc/api_routing.hip, api_int4.hip): argument checks,
limits of launches, the choice of tiles and their number, which tests/sanitize/routing_driver.hip's
stand-in for the launcher looks over.  CPU only: sanitizers on the host side of the compile, no
kernel runs."""
import os

import pytest

from test_sanitizers import ENV, HIPCC, ROOT, SAN, run


def test_routing_and_int4_abi_under_asan_ubsan(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    csrc = os.path.join(ROOT, "swiglu_gemm_amd", "csrc")
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-w",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-omit-frame-pointer",
             "-I", os.path.join(ROOT, "include"), "-I", csrc]
    objs = []
    for src in (os.path.join(csrc, "api_routing.hip"), os.path.join(csrc, "api_int4.hip"),
                os.path.join(SAN, "routing_driver.hip")):
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        run([HIPCC] + flags + ["-c", src, "-o", objs[-1]])
    exe = str(tmp_path / "routing_san")
    run([HIPCC, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address",
         "-Xarch_host", "-fsanitize=undefined"] + objs + ["-o", exe])
    env = {k: v for k, v in ENV.items() if k != "SG_FORCE_INT4"}
    assert run([exe], env=env, timeout=300).stdout.startswith("ok")
