"""The GPU tests' sizes still choose the kernels of the experts' products that they are
there for: the choice goes by a model of measured times, and a change of that moves
sizes from one kernel to another.  The rule is asked of the source itself, compiled for
the host."""

import os
import shutil
import subprocess

import pytest

from tests import test_gpu_expert_shapes as shapes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUS = 256


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not found")
    exe = str(tmp_path_factory.mktemp("plans") / "expert_plans")
    # host code only: the device image that its kernels' stubs name stays unresolved
    cmd = [hipcc, "--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17", "-Wl,--unresolved-symbols=ignore-all",
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "fp8_block_scaled_quant_amd", "csrc"),
           "-x", "hip", os.path.join(ROOT, "tests", "expert_plans.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1")

    def ask(cases):
        text = "".join("%d %d %d %d %d\n" % (gated, sum(counts) + behind, len(counts), n, k) for gated, counts, behind, n, k in cases)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, env=env, timeout=120)
        assert r.returncode == 0, r.stderr
        return r.stdout.splitlines()
    return ask


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
