"""The host code of the LayerNorm, paged-attention and mixture-of-experts entry
points under AddressSanitizer and UndefinedBehaviorSanitizer, with stand-in
launchers (tests/host_sanitize/ops_driver.cpp).  CPU only: no HIP runtime call
is made."""
import os
import subprocess

import pytest

from tests.test_host_sanitizers import CLANG, CSRC, HERE, ROOT


def test_ops_host_code_under_asan_and_ubsan(tmp_path):
    if not os.path.exists(CLANG):
        pytest.skip("clang++ of the ROCm toolchain not found")
    flags = ["-std=c++17", "-g", "-O1", "-D__HIP_PLATFORM_AMD__", "-fsanitize=address,undefined",
             "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-w",
             "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]
    srcs = [os.path.join(CSRC, "aa_plan.cpp"), os.path.join(CSRC, "aa_api_ops.cpp"),
            os.path.join(HERE, "ops_stub_launch.cpp"), os.path.join(HERE, "ops_driver.cpp")]
    exe = str(tmp_path / "aa_ops_host_san")
    r = subprocess.run([CLANG, *flags, *srcs, "-o", exe, "-lpthread"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    env.pop("LD_PRELOAD", None)
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-4000:])
    assert "host checks passed" in r.stdout


def test_in_place_operands_do_not_hang_on_merged_literals(tmp_path):
    """The same calls from a build in which equal string literals are objects of
    their own (which the language leaves open): the in-place forms are accepted
    all the same."""
    if not os.path.exists(CLANG):
        pytest.skip("clang++ of the ROCm toolchain not found")
    flags = ["-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-fwritable-strings", "-w",
             "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]
    srcs = [os.path.join(CSRC, "aa_plan.cpp"), os.path.join(CSRC, "aa_api_ops.cpp"),
            os.path.join(HERE, "ops_stub_launch.cpp"), os.path.join(HERE, "in_place_driver.cpp")]
    exe = str(tmp_path / "aa_ops_literals")
    r = subprocess.run([CLANG, *flags, *srcs, "-o", exe, "-lpthread"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "in-place calls passed" in r.stdout, (r.stdout, r.stderr)
