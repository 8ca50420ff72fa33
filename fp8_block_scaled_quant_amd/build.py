"""Compile the HIP sources into the in-tree shared libraries ``libfp8bsq.so`` (the
quantizers and the block-scaled GEMM) and ``libfp8bsq_ffn.so`` (the feed-forward
operators, which call the first), and the latter's Python binding ``_ffn_ext.so``
(host code over torch's headers, by g++).  The libraries need hipcc alone: run as
a script where there is no torch or no g++, this file builds them and leaves the
binding out.

gfx950 only.  Packed-FP32 instruction selection is switched off for every HIP
source, floating-point contraction is off unless a kernel asks for a fused
multiply-add explicitly, and no fast-math flag is used (the quantizer relies on
IEEE division and exact fused multiply-adds).
"""

import importlib.util
import os
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libfp8bsq.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)

FFN_LIB_NAME = "libfp8bsq_ffn.so"
FFN_LIB_PATH = os.path.join(PKG_DIR, FFN_LIB_NAME)

SOURCES = ["abi.cpp", "act_quant.hip", "weight_dequant.hip", "weight_quant.hip", "block_gemm.hip"]
FFN_SOURCES = ["ffn_abi.cpp", "gated_ffn.hip", "gated_ffn_backward.hip", "fp4.hip", "grad_clip.hip"]
BINDING_SOURCE = "ffn_binding.cpp"
BINDING_PATH = os.path.join(PKG_DIR, "_ffn_ext.so")

HIP_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-fvisibility=hidden",
    "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found: the HIP toolchain is required to build libfp8bsq")
    return path


def build(verbose: bool = False, jobs: int = 4) -> str:
    """Compile every source for gfx950 and link both libraries and, with torch and g++, the binding.

    Returns ``libfp8bsq.so``'s path.
    """
    objdir = os.path.join(PKG_DIR, "_build")
    os.makedirs(objdir, exist_ok=True)
    cc = hipcc()
    missing = "torch" if importlib.util.find_spec("torch") is None else None if shutil.which("g++") else "g++"
    if not missing:
        binding = (BINDING_SOURCE, subprocess.Popen(_binding_command(objdir, verbose), stdout=subprocess.PIPE,
                                                    stderr=subprocess.STDOUT))
    procs = []
    objs = {src: os.path.join(objdir, src + ".o") for src in SOURCES + FFN_SOURCES}
    # the slowest source first, so that the others compile beside it
    for src in sorted(objs, key=lambda s: s != "block_gemm.hip"):
        lang = ["-x", "hip"] if src.endswith(".hip") else []
        cmd = [cc, *HIP_FLAGS, "-I", INCLUDE, "-I", CSRC, *lang, "-c",
               os.path.join(CSRC, src), "-o", objs[src]]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        if len(procs) >= jobs:
            _drain(procs[:1])
            procs = procs[1:]
    _drain(procs)
    _link(cc, [objs[s] for s in SOURCES], [], LIB_PATH, verbose)
    # found beside it at run time
    _link(cc, [objs[s] for s in FFN_SOURCES], ["-L", PKG_DIR, "-lfp8bsq", "-Wl,-rpath,$ORIGIN"], FFN_LIB_PATH, verbose)
    if missing:
        print(f"{missing} not found: the Python binding, {os.path.basename(BINDING_PATH)}, is not built", file=sys.stderr)
        return LIB_PATH
    _drain([binding])
    from torch.utils import cpp_extension
    dirs = [arg for d in cpp_extension.library_paths() for arg in ("-L", d, "-Wl,-rpath," + d)]
    _link(cc, [os.path.join(objdir, BINDING_SOURCE + ".o")],
          ["-L", PKG_DIR, "-lfp8bsq_ffn", "-Wl,-rpath,$ORIGIN", *dirs, "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_hip"], BINDING_PATH, verbose)
    return LIB_PATH


def _binding_command(objdir, verbose):
    """The binding's compile command: host code only, torch's own compile-time definitions."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    cmd = [shutil.which("g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__",
           "-DUSE_ROCM", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"],
           *[arg for d in cpp_extension.include_paths("cuda") for arg in ("-isystem", d)],
           "-c", os.path.join(CSRC, BINDING_SOURCE), "-o", os.path.join(objdir, BINDING_SOURCE + ".o")]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    return cmd


def _link(cc, objs, libs, path, verbose):
    tmp = path + ".tmp"
    link = [cc, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, *libs, "-o", tmp]
    if verbose:
        print(" ".join(link), file=sys.stderr)
    out = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if out.returncode != 0:
        raise RuntimeError("link failed:\n" + out.stdout.decode(errors="replace"))
    os.replace(tmp, path)


def _drain(procs):
    for src, p in procs:
        text, _ = p.communicate()
        if p.returncode != 0:
            raise RuntimeError(f"hipcc failed on {src}:\n" + text.decode(errors="replace"))


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
