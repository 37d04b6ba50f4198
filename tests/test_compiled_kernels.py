"""The compiled kernels: nothing that works lane by lane stands between the end
of a branch or loop that only some lanes of a wave took and the instruction that turns
the others on again.  The compiler has placed copies of live registers there
(v_accvgpr_write, under register pressure); the lanes that were off lose what
was copied, thread numbers and addresses among it."""
import concurrent.futures
import os
import re
import shutil
import subprocess

import pytest

import group_wise_affine_aq_amd as aq

OBJDUMP = shutil.which("llvm-objdump", path="/opt/rocm/llvm/bin:" + os.environ.get("PATH", ""))

# what ignores the lanes that are off, or only reads them
SCALAR = re.compile(r"s_|v_(readlane|writelane|readfirstlane|nop)")
RESTORES = re.compile(r"s_(or_b64 exec, exec|mov_b64 exec|or_saveexec_b64)")
LEAVES = re.compile(r"s_(cbranch|branch|endpgm|setpc|swappc)")


def misplaced(lines):
    """(kernel, label, instructions) of every such place in a disassembly."""
    kernel, labels, ends = None, {}, []
    for i, line in enumerate(lines):
        if "s_cbranch_execz" in line:
            ends.append((kernel, re.search(r"s_cbranch_execz\s+(\.?L\w+)", line).group(1)))
        elif "s_cbranch_execnz" in line:  # what follows runs when no lane goes back
            labels[kernel, i] = i
            ends.append((kernel, i))
        elif line and line[0] in "<.L_":
            name = re.match(r"<?(\.?\w+)>?:", line)
            if name and name.group(1).startswith("_Z"):
                kernel = name.group(1)
            elif name:
                labels[kernel, name.group(1)] = i
    found = []
    for kernel, label in dict.fromkeys(ends):
        lane_wise = []
        for i in range(labels[kernel, label] + 1, len(lines)):
            op = lines[i].split("//")[0].split(";")[0].strip()
            if not op:
                continue
            if RESTORES.match(op):
                if lane_wise:
                    found.append((kernel, label, lane_wise))
                break
            if LEAVES.match(op) or op.endswith(":"):
                break
            if not SCALAR.match(op):
                lane_wise.append(op)
    return found


def test_the_scan_finds_them():
    text = """
_Z6kernel:
	s_and_saveexec_b64 s[2:3], vcc
	s_cbranch_execz .LBB0_2
	global_load_dword v1, v[2:3], off
.LBB0_2:                                ; in Loop
	v_writelane_b32 v255, s68, 8
	%s
	s_or_b64 exec, exec, s[2:3]
	v_and_b32_e32 v0, 32, v12
	s_endpgm
"""
    assert misplaced((text % "v_accvgpr_write_b32 a167, v167").split("\n")) == [
        ("_Z6kernel", ".LBB0_2", ["v_accvgpr_write_b32 a167, v167"])]
    assert not misplaced((text % "s_mov_b32 s97, s5").split("\n"))
    text = """
_Z6kernel:
.LBB0_1:                                ; Loop
	v_cmp_gt_i32_e32 vcc, 4, v1
	s_andn2_b64 exec, exec, vcc
	s_cbranch_execnz .LBB0_1
	%s
	s_or_b64 exec, exec, s[2:3]
	s_endpgm
"""
    assert [x[2] for x in misplaced((text % "v_mov_b32_e32 v1, v2").split("\n"))] == [
        ["v_mov_b32_e32 v1, v2"]]
    assert not misplaced((text % "s_nop 0").split("\n"))


@pytest.mark.skipif(OBJDUMP is None, reason="no llvm-objdump")
def test_no_lane_loses_what_it_holds(tmp_path):
    lib = os.path.join(os.path.dirname(aq.__file__), "libaq.so")
    if not os.path.exists(lib):
        pytest.skip("nothing is built")
    shutil.copy(lib, tmp_path / "libaq.so")
    subprocess.run([OBJDUMP, "--offloading", "libaq.so"], cwd=tmp_path, check=True,
                   capture_output=True)
    objects = [p for p in tmp_path.iterdir() if "gfx950" in p.name]
    assert objects
    kernels, found = 0, []
    with concurrent.futures.ThreadPoolExecutor(4) as pool:
        for text in pool.map(lambda obj: subprocess.run(
                [OBJDUMP, "-d", "--symbolize-operands", "--no-show-raw-insn", "--no-leading-addr",
                 obj.name], cwd=tmp_path, check=True, capture_output=True, text=True).stdout, objects):
            lines = text.split("\n")
            kernels += sum(line.startswith("<_Z") for line in lines)
            found += misplaced(lines)
    assert kernels > 100
    assert found == []
