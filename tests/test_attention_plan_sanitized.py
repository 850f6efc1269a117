"""How attention calls are cut (attention_plan.h), built into a host driver with
AddressSanitizer and UndefinedBehaviorSanitizer (g++, CPU only)."""
import os
import shutil
import subprocess

import pytest

from ring_all_reduce_allreduce_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_which_kernel_a_call_takes(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not installed")
    exe = str(tmp_path / "attention_plan_check")
    subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-Wall", "-Werror", "-I", os.path.join(build.PKG, "csrc"),
                    os.path.join(HERE, "attention_plan_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert out.stdout.strip() == "ok" and out.returncode == 0, out.stdout + out.stderr[-3000:]
