"""The GPU tests' sizes still choose the kernels of the experts' products that they are
there for: the choice goes by a model of measured times, and a change of that moves
sizes from one kernel to another.  The rule is asked of the source itself, compiled for
the host."""

import os
import re
import shutil
import subprocess

import pytest

from fp8_block_scaled_quant_amd import build
from tests import test_gpu_expert_shapes as shapes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUS = 256


def _hipcc():
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not found")
    return hipcc


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plans") / "expert_plans")
    # host code only: the device image that its kernels' stubs name stays unresolved
    cmd = [_hipcc(), "--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17", "-Wl,--unresolved-symbols=ignore-all",
           "-I", build.INCLUDE, "-I", build.CSRC, "-x", "hip", os.path.join(ROOT, "tests", "expert_plans.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1")

    def ask(text, *args):
        r = subprocess.run([exe, *args], input=text, capture_output=True, text=True, env=env, timeout=120)
        assert r.returncode == 0, r.stderr
        return r.stdout.splitlines()
    return ask


@pytest.fixture(scope="module")
def kernels(plans):
    return lambda cases: plans("".join("%d %d %d %d %d\n" % (gated, sum(counts) + behind, len(counts), n, k)
                                       for gated, counts, behind, n, k in cases))


def test_sizes_take_the_kernels_they_are_there_for(kernels):
    assert kernels(shapes.CASES) == list(shapes.SIZES.values())
    # every kernel that there is
    assert {(shape, case[0]) for case, shape in shapes.SIZES.items()} == \
        {(shape, gated) for shape in ("many by four", "many", "some", "few", "long32", "long64") for gated in (False, True)}


def test_few_tiles_are_more_than_the_workgroups():
    """... of each kind, with two steps of four K blocks a tile and with more."""
    steps = {}
    for (gated, counts, _, n, k), shape in shapes.SIZES.items():
        if shape.startswith("long"):
            features = int(shape[4:]) // (2 if gated else 1)
            assert sum(-(-c // 16) for c in counts) * -(-n // features) > CUS
            steps.setdefault((shape, gated), set()).add(-(-k // 512))
    assert len(steps) == 4 and all(min(s) == 2 and max(s) > 2 for (shape, _), s in steps.items() if shape == "long32")
    assert all(min(s) == 3 and max(s) > 3 for (shape, _), s in steps.items() if shape == "long64")   # from 12 blocks on


def test_two_workgroups_share_a_compute_unit(plans, tmp_path):
    """... of the kernels whose grid and whose times are of two, with every number of
    experts: by the LDS that a launch asks for, and the kernel's own."""
    out = str(tmp_path / "expert_gemm.s")
    r = subprocess.run([_hipcc(), *build.HIP_FLAGS, "--cuda-device-only", "-S", "-I", build.INCLUDE, "-I", build.CSRC, "-x", "hip",
                        os.path.join(build.CSRC, "expert_gemm.hip"), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    with open(out) as f:
        own = re.findall(r"group_segment_fixed_size: (\d+)\n *\.kernarg[^\0]*?\.name: +(\S+)", f.read())
    own = [(size, re.search(r"ELi(\d+)E", name)[1]) for size, name in own if "product_stream_kernel" in name]
    assert sorted(rows for _, rows in own) == ["16", "16", "64", "64"]
    asked = dict(zip(("16", "64"), map(int, plans("", "1024")[0].split())))
    for size, rows in own:
        assert 2 * (asked[rows] + int(size)) <= 160 * 1024, (size, rows)
