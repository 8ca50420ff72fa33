"""A library that lacks a launcher does not link: without this, a source left out of the
build, or a signature that drifted, would become a call through null."""

import os
import subprocess

import pytest

from fp8_block_scaled_quant_amd import build


@pytest.fixture(scope="module")
def layer(tmp_path_factory):
    if not os.path.exists(build.LIB_PATH):
        build.build()
    obj = str(tmp_path_factory.mktemp("layer") / "ffn_abi.o")
    r = subprocess.run(build._compile_command(build.hipcc(), "ffn_abi.cpp", obj), capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return obj


def test_the_layer_needs_every_launcher(layer):
    r = subprocess.run(["nm", layer], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    kinds = {line.split()[-1]: line.split()[-2] for line in r.stdout.splitlines() if "fp8bsq" in line and "launch_" in line}
    assert len(kinds) == 11 and set(kinds.values()) == {"U"}, kinds   # five of the feed-forward operators, six of the experts'


def test_a_library_without_its_launchers_does_not_link(layer, tmp_path):
    out = str(tmp_path / "libwithout.so")
    with pytest.raises(RuntimeError, match="launch_expert_product"):
        build._link(build.hipcc(), [layer], build._ffn_link(), out, False)
    assert not os.path.exists(out)
