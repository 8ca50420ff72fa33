"""The GPU tests' sizes still take the launches that they are there for: the
backward pass plans its products by measured times, and a change of those moves
sizes from one launch to another.  The plans are asked of the source itself,
compiled for the host."""

import os
import shutil
import subprocess

import pytest

from tests import test_gpu_gated_ffn_backward_paths as paths

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not found")
    exe = str(tmp_path_factory.mktemp("plans") / "backward_plans")
    # host code only: the device image that its kernels' stubs name stays unresolved
    cmd = [hipcc, "--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17", "-Wl,--unresolved-symbols=ignore-all",
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "fp8_block_scaled_quant_amd", "csrc"),
           "-x", "hip", os.path.join(ROOT, "tests", "backward_plans.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    # no device: the plans are those of 256 compute units
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1")

    def ask(sizes):
        text = "".join("%d %d %d\n" % s for s in sizes)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, env=env, timeout=120)
        assert r.returncode == 0, r.stderr
        return [line.split() for line in r.stdout.splitlines()]
    return ask


def test_sizes_take_the_launches_they_are_there_for(plans):
    for (dx, dw, paired, _), want in zip(plans(paths.TOGETHER), paths.TOGETHER.values()):
        assert (dx, dw) == want and paired == ("1" if (dx == "big") == (dw == "big") else "0")
    assert set(paths.TOGETHER.values()) == {(dx, dw) for dx in ("big", "mid", "split") for dw in ("big", "mid", "split")}
    for (dx, dw, paired, alone), want in zip(plans(paths.JOINED), paths.JOINED.values()):
        assert (dx, dw, paired, alone) == (*want, "1", "big")
    assert plans([paths.LARGE])[0][:2] == ["big", "big"]


def test_plans_without_tokens(plans):
    """Nothing to multiply: no parts, so no partials in a workspace."""
    assert all("split" not in p for p in plans([(0, 128, 128), (0, 18432, 7168)]))
