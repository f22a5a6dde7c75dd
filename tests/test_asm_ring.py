"""A stage of the direct-to-LDS ring is written again by the loads that any wave issues behind
the barrier at the end of its tile, and the barrier does not wait for LDS reads.  So a wave may
come to a barrier only with none of its own reads in flight: this test builds the library's
ring kernels to gfx950 assembly and follows every path to every s_barrier, counting the LDS
operations that no s_waitcnt lgkmcnt has covered.

CPU only: hipcc cross-compiles for gfx950 without a GPU."""
import os
import re
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "swiglu_gemm_amd"))

# every kind of ring: tile kernels of both operand sizes (split-weight ones among them, which
# are in the NN units), few-row kernels, grouped and 4-bit kernels
UNITS = {"inst_bf16_nn.hip": 50, "inst_e4m3_nn.hip": 20, "inst_decode_bf16.hip": 4,
         "inst_grouped_bf16.hip": 10, "inst_grouped_e4m3.hip": 4, "inst_mx4.hip": 12}
MANY = 99
DS = re.compile(r"ds_(?!nop)")
WAIT = re.compile(r"s_waitcnt\b(.*)")
LABEL = re.compile(r"^(\.L\w+|\w+):")
JUMP = re.compile(r"s_(c?branch)\w*\s+(\.L\w+)")


def reads_in_flight(lines):
    """The s_barriers of one kernel (a list of assembly lines) that a path reaches with LDS
    operations in flight, and how many s_barriers there are.  Blocks are walked with the most
    operations that can be in flight at their start, until nothing changes; LDS operations end
    in order, so lgkmcnt(n) leaves at most n of them."""
    label, code = {}, []
    for line in lines:
        s = line.split(";")[0].strip()
        m = LABEL.match(s)
        if m:
            label[m.group(1)] = len(code)
        elif s and not s.startswith("."):
            code.append(s)
    seen, todo, bad, barriers = {}, [(0, 0)], set(), set()
    while todo:
        i, n = todo.pop()
        while i < len(code):
            if seen.get(i, -1) >= n:
                break
            seen[i] = n
            s = code[i]
            if DS.match(s):
                n = min(n + 1, MANY)
            w = WAIT.match(s)
            if w:
                c = re.search(r"lgkmcnt\((\d+)\)", w.group(1))
                if c:
                    n = min(n, int(c.group(1)))
                elif w.group(1).strip().isdigit():
                    n = min(n, (int(w.group(1)) >> 8) & 15)
            if s.startswith("s_barrier"):
                barriers.add(i)
                if n:
                    bad.add(i)
            j = JUMP.match(s)
            if j:
                todo.append((label[j.group(2)], n))
                if j.group(1) == "branch":
                    break
            if s.startswith(("s_endpgm", "s_setpc")):
                break
            i += 1
    return bad, len(barriers)


def kernels(text):
    for m in re.finditer(r"^(\w+):\s*; @\1\n(.*?)^\.Lfunc_end\d+:", text, re.S | re.M):
        yield m.group(1), m.group(2).splitlines()


def assemble(build, src, out_dir):
    out = os.path.join(out_dir, src.replace(".hip", ".s"))
    cmd = [build.hipcc()] + build._flags() + ["-S", "--offload-device-only", "-w",
                                               os.path.join(build.CSRC, src), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return out


@pytest.fixture(scope="module")
def asm_files(tmp_path_factory):
    import build
    if shutil.which(build.hipcc()) is None and not os.path.exists(build.hipcc()):
        pytest.skip("hipcc not available")
    d = str(tmp_path_factory.mktemp("asm_ring"))
    with ThreadPoolExecutor(4) as ex:
        return dict(zip(UNITS, ex.map(lambda u: assemble(build, u, d), UNITS)))


def test_the_walk_itself():
    loop = """s_mov_b32 s0, 0
.LBB0_1:
ds_read_b128 v[0:3], v9
v_mfma_f32_32x32x16_bf16 a[0:15], v[4:7], v[4:7], a[0:15]
s_waitcnt vmcnt(0)%s
s_barrier
v_mfma_f32_32x32x16_bf16 a[0:15], v[0:3], v[0:3], a[0:15]
s_cbranch_scc1 .LBB0_1
s_endpgm"""
    assert reads_in_flight((loop % "").splitlines()) == ({4}, 1)
    assert reads_in_flight((loop % " lgkmcnt(1)").splitlines()) == ({4}, 1)
    assert reads_in_flight((loop % " lgkmcnt(0)").splitlines()) == (set(), 1)
    carried = "s_barrier\n.LBB0_1:\ns_waitcnt lgkmcnt(0)\ns_barrier\nds_read_b32 v0, v1\n" \
              "s_branch .LBB0_1"
    assert reads_in_flight(carried.splitlines()) == (set(), 2)
    assert reads_in_flight(carried.replace("lgkmcnt(0)", "vmcnt(0)").splitlines()) == ({2}, 2)


@pytest.mark.parametrize("unit", sorted(UNITS))
def test_no_wave_meets_a_barrier_with_lds_reads_in_flight(asm_files, unit):
    seen = 0
    for name, lines in kernels(open(asm_files[unit]).read()):
        if not any("global_load_lds" in s for s in lines):
            continue
        bad, barriers = reads_in_flight(lines)
        assert barriers > 0, name
        assert not bad, "%s: %d of %d barriers with LDS reads in flight" % (name, len(bad), barriers)
        seen += 1
    assert seen >= UNITS[unit], "expected the ring kernels, found %d" % seen
