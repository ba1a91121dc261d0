"""The rules by which the launchers choose a kernel (csrc/aa_rules.h), compiled
for the host and checked on the CPU: the launchers use the same functions."""
import os
import shutil
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "associative_algebra_block_amd", "csrc")
HERE = os.path.join(ROOT, "tests", "host_rules")


def compiled(tmp_path, name):
    cxx = shutil.which("g++") or shutil.which("clang++") or "/opt/rocm/llvm/bin/clang++"
    exe = str(tmp_path / name)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-I" + CSRC, "-I" + os.path.join(ROOT, "include"),
                        os.path.join(HERE, name + ".cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    return exe


def test_a_turned_append_fits_a_grid(tmp_path):
    r = subprocess.run([compiled(tmp_path, "append_driver")], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "append rule holds" in r.stdout, (r.stdout, r.stderr)
