"""The C ABI from a plain C99 program: include/qmoe.h compiles with gcc -std=c99
-Wall -Werror, links against libqmoe.so, and the host-only calls behave as the
header states (no GPU needed)."""

import os
import shutil
import subprocess

import pytest

from quantized_moe_grouped_route_gb300 import qmoe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_header_compiles_as_c99_and_host_calls_work(tmp_path):
    qmoe.lib()  # built in-tree
    libdir = os.path.dirname(qmoe.LIB_PATH)
    exe = str(tmp_path / "abi_from_c")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "c", "abi_from_c.c"),
                    "-o", exe, "-L", libdir, "-lqmoe", "-Wl,-rpath," + libdir, "-lm"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "ok: 0 failure(s)" in r.stdout


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists("/usr/local/cuda/include"),
                    reason="needs g++ and the CUDA headers")
def test_numbers_kept_per_device(tmp_path):
    exe = str(tmp_path / "per_device")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I/usr/local/cuda/include", "-I",
                    os.path.join(ROOT, "quantized_moe_grouped_route_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "c", "per_device.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
