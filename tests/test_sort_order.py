"""The sort's waves hand LDS counters from lane to lane without a barrier, which the
hardware's order of a wave's accesses allows and the compiler has to be told: in the
compiled kernel a wavefront fence stands between each write of a counter and the
accesses of other lanes before and after it."""

import os
import re
import shutil
import subprocess

import pytest

from fp8_block_scaled_quant_amd import build


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not found")
    out = str(tmp_path_factory.mktemp("sort") / "expert_sort.ll")
    cmd = [hipcc, *build.HIP_FLAGS, "--cuda-device-only", "-S", "-emit-llvm", "-I", build.INCLUDE, "-I", build.CSRC, "-x", "hip",
           os.path.join(build.CSRC, "expert_sort.hip"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    with open(out) as f:
        return re.findall(r"^define [^\n]*?(sort_\w+?_kernel)\w*\([^\n]*\n(.*?)^}", f.read(), re.M | re.S)


def test_counters_are_written_between_fences(kernels):
    placing = [body for name, body in kernels if "sort_place" in name]
    assert len(placing) == 2   # int32 and int64 numbers
    for body in placing:
        # the accesses after the last barrier: handing out rows
        lines = [l.strip() for l in body[body.rindex("amdgcn.s.barrier"):].splitlines()]
        marks = "".join("f" if l.startswith("fence syncscope(\"wavefront\")") else "w" if re.match(r"store i32 .*addrspace\(3\)", l) else "" for l in lines)
        assert marks.count("w") >= 2                 # the first rounds and the others
        assert "ww" not in marks and re.fullmatch(r"f*(fwf+)+", marks), marks
