"""Builds libringsim.so, and the operators' Python extension on top of it,
in-tree with hipcc for gfx950.

Usage: python -m ring_all_reduce_allreduce_amd.build [--verbose]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libringsim.so")
BINDING = os.path.join(PKG, "_ops_binding.so")
# Results of matrix instructions in ordinary vector registers: in accumulation
# registers, which only those instructions and moves reach, every rescaling of
# them copies them over and back.
MATRIX_FLAGS = ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]
# (source, object name, extra defines): the line kernel's instantiation unit
# is compiled once per line mode, the attention's once per head size.
SOURCES = [
    ("ringsim_api.hip", "ringsim_api", []),
    ("ring_bulk.hip", "ring_bulk", []),
    ("ring_lines_inst.hip", "ring_lines_half", ["-DRINGSIM_LINE_MODE=kLinesHalf", "-DRINGSIM_LINE_NAME=half"]),
    ("ring_lines_inst.hip", "ring_lines_one", ["-DRINGSIM_LINE_MODE=kLinesOne", "-DRINGSIM_LINE_NAME=one"]),
    ("ring_lines_inst.hip", "ring_lines_multi", ["-DRINGSIM_LINE_MODE=kLinesMulti", "-DRINGSIM_LINE_NAME=multi"]),
    ("tree.hip", "tree", []),
    ("copy.hip", "copy", []),
    ("ringsim_ops.hip", "ringsim_ops", []),
    ("rms_norm.hip", "rms_norm", []),
    ("rms_norm_backward.hip", "rms_norm_backward", []),
    ("grad_norm.hip", "grad_norm", []),
    ("ringsim_attention.hip", "ringsim_attention", []),
    ("rotary.hip", "rotary", []),
    ("kv_cache.hip", "kv_cache", []),
    ("attention.hip", "attention", []),
    *(("attention_inst.hip", f"attention_{d}", [f"-DRINGSIM_HEAD_DIM={d}", *MATRIX_FLAGS])
      for d in (64, 96, 128, 192, 256)),
]
# The Python extension's sources: host code only.
BINDING_SOURCES = ["ops_binding", "attention_binding"]
ARCH = "gfx950"

# -packed-fp32-ops: keep the compiler from forming packed fp32 instructions.
# -ffp-contract=off: every hop is one rounded add or multiply, never fused.
HIP_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-ffp-contract=off",
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-function",
    f"-I{os.path.join(ROOT, 'include')}",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the ROCm toolchain is required to build libringsim")


def binding_flags() -> list[str]:
    """Host code only: where torch's and Python's headers are."""
    import sysconfig

    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    return ["-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f"-I{inc}", f"-I{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}",
            f"-I{sysconfig.get_paths()['include']}"]


def torch_lib_dir() -> str:
    import torch

    return os.path.join(os.path.dirname(torch.__file__), "lib")


def build(verbose: bool = False) -> str:
    """Compiles every source to an object, links libringsim.so and the
    operators' Python extension, returns the library's path."""
    cc = hipcc()
    with tempfile.TemporaryDirectory(prefix="ringsim_build_") as tmp:
        objs, binding_objs = [], []
        procs = []
        jobs = [(name, [cc, *HIP_FLAGS, *defines, "-c", os.path.join(CSRC, src), "-o", os.path.join(tmp, name + ".o")])
                for src, name, defines in SOURCES]
        jobs += [(name, [cc, *binding_flags(), "-c", os.path.join(CSRC, name + ".cpp"), "-o",
                         os.path.join(tmp, name + ".o")]) for name in BINDING_SOURCES]
        for name, cmd in jobs:
            obj = cmd[-1]
            if verbose:
                print(" ".join(cmd), flush=True)
            procs.append((name, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
            (binding_objs if name in BINDING_SOURCES else objs).append(obj)
        failed = []
        for src, p in procs:
            out, _ = p.communicate()
            if out and (verbose or p.returncode):
                sys.stderr.write(out)
            if p.returncode:
                failed.append(src)
        if failed:
            raise RuntimeError(f"hipcc failed for {failed}")
        tmp_lib = LIB + ".tmp"
        cmd = [cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp_lib, *objs]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp_lib, LIB)
        # Loaded by Python, so Python's symbols stay open; libringsim.so is found beside it.
        cmd = [cc, "-shared", "-fPIC", "-o", BINDING + ".tmp", *binding_objs, f"-L{torch_lib_dir()}", "-lc10",
               "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python", f"-L{PKG}", "-l:libringsim.so", "-Wl,-rpath,$ORIGIN"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(BINDING + ".tmp", BINDING)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv))
