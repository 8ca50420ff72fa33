"""Building the C libraries takes hipcc and nothing else: the build runs with a
stand-in for the compilers that records its commands, into a folder of its own."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

COMPILER = """#!{python}
import os, sys
args = sys.argv[1:]
open(args[args.index("-o") + 1], "w").close()
open({log!r}, "a").write(os.path.basename(sys.argv[0]) + " " + " ".join(args) + "\\n")
"""

# build.py as a script sees it: without the package, which imports torch
RUN = """
import importlib.util, os, sys
if sys.argv[3] == "no":
    sys.modules["torch"] = None
spec = importlib.util.spec_from_file_location("build", sys.argv[1])
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b.PKG_DIR = sys.argv[2]
for name in ("LIB_PATH", "FFN_LIB_PATH", "BINDING_PATH"):
    setattr(b, name, os.path.join(sys.argv[2], os.path.basename(getattr(b, name))))
print(b.build())
"""


def _build(tmp_path, tools, torch="yes"):
    bin_dir, out, log = tmp_path / "bin", tmp_path / "out", tmp_path / "log"
    bin_dir.mkdir()
    out.mkdir()
    for tool in tools:
        (bin_dir / tool).write_text(COMPILER.format(python=sys.executable, log=str(log)))
        (bin_dir / tool).chmod(0o755)
    r = subprocess.run([sys.executable, "-c", RUN, os.path.join(ROOT, "fp8_block_scaled_quant_amd", "build.py"), str(out), torch],
                       capture_output=True, text=True, env=dict(os.environ, PATH=str(bin_dir)), timeout=300)
    return r, {p.name for p in out.iterdir() if p.suffix == ".so"}, log.read_text() if log.exists() else ""


@pytest.mark.parametrize("tools,torch,missing", [(["hipcc", "g++"], "no", "torch"), (["hipcc"], "yes", "g++"), (["hipcc"], "no", "torch")])
def test_libraries_without_torch_or_gxx(tmp_path, tools, torch, missing):
    r, built, log = _build(tmp_path, tools, torch)
    assert r.returncode == 0, r.stderr
    assert built == {"libfp8bsq.so", "libfp8bsq_ffn.so"} and f"{missing} not found" in r.stderr
    assert "g++ " not in log and log.count("--offload-arch=gfx950") == len(log.splitlines())


def test_binding_too_where_both_are_there(tmp_path):
    r, built, log = _build(tmp_path, ["hipcc", "g++"])
    assert r.returncode == 0, r.stderr
    assert built == {"libfp8bsq.so", "libfp8bsq_ffn.so", "_ffn_ext.so"} and "not found" not in r.stderr
    assert sum(line.startswith("g++ ") for line in log.splitlines()) == 1
    # packed FP32 instructions stay off in every HIP source
    hip = [line for line in log.splitlines() if " -c " in line and line.startswith("hipcc")]
    assert len(hip) >= 9 and all("-packed-fp32-ops" in line for line in hip)
